"""What the kernels' sources may not hold."""
import glob
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_05_gb300", "csrc")


def test_no_cluster_multicast():
    """The same kernels run on every rank of a run over several GPUs, where loads with cluster multicast stay out."""
    sources = glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    assert len(sources) > 10
    for path in sources:
        assert "multicast::" not in open(path).read(), path
