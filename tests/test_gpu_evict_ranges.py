"""GPU: msa_evict_paged at the ends of its ranges."""
import pytest
import torch

from test_gpu_evict import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_05_gb300 as m
    torch.cuda.set_device(0)
    return m


@pytest.mark.parametrize("lens", [[5], [0], [70000]])
@pytest.mark.parametrize("below", [0, 1, 1023, 1024, 8192])
def test_budgets_next_to_2_31(msa, lens, below):
    """The tail of `kept`, behind the kept slots, is -1 up to its end and not a word further (70,000 keys: a cluster)."""
    budget = 2 ** 31 - 1 - below
    c = Cache(msa, lens, 1, budget, 0)
    space = torch.full((budget + 4096,), 7, dtype=torch.int32, device="cuda")
    kept = space[2048:2048 + budget].view(1, 1, budget)
    new_weight = torch.zeros(1, 1, max(1, lens[0]), device="cuda")
    ws = c.ws(msa)
    _, _, cu = c.call(msa, kept=kept, new_weight=new_weight, ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    n = lens[0]
    assert cu.tolist() == [0, n]
    assert torch.equal(kept[0, 0, :n], torch.arange(n, dtype=torch.int32, device="cuda"))
    assert int(kept[0, 0, n:].max()) == -1 and int(kept[0, 0, n:].min()) == -1
    assert (space[:2048] == 7).all() and (space[2048 + budget:] == 7).all()
    assert torch.equal(new_weight[0, 0, :n], c.weight[0, 0, :n])
