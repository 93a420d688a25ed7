"""Queries and outputs of more than 2^31 values: the first, the last and some sequences between against 64 bits."""
import pytest
import torch

from test_gpu_prompt_attn import Batch, check, msa, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["packed", "fp8"])
def test_many_rows(msa, layout):
    seqs = 2800
    q = [90 + s % 21 for s in range(seqs)]
    kv = [n + (300 if s % 97 == 0 else 0) for s, n in enumerate(q)]
    b = Batch(msa, q, kv, 64, 4, layout, seed=83)
    assert b.q.numel() > 2 ** 31
    ws = msa.workspace(b.prob, b.op())
    o, lse = b.run(ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    for s in (0, 1, 97, 1400, 2716, 2798, 2799):
        at = sum(q[:s])
        part = slice(at, at + q[s])
        check((o[part], lse[part]), reference([q[s]], [kv[s]], [b.rows[s]], b.q[part], b.k, b.v, b.ks, b.vs, 0.0, None), f"sequence {s}")
