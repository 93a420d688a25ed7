"""Prompt and tree attention over E4M3 pages where logits or page scales are far from ordinary.

Bounds: where an fp32 logit's own last place is many nats the weights of keys that are about as large are anybody's, but they
are weights: o lies between the least and the largest value among the keys whose logit, with its error, can be among the
largest (all others together count less than n e^-60), up to the weights' and the output's roundings (2^-11 and 2^-8 of the
largest such value); lse is off by at most the largest logit's error and ln n.  A logit's error is that of
test_gpu_prompt_attn plus its own rounding, twice (with V's scale and without): 2^-24 of its value each, and as much of the
reference.
"""
import math

import pytest
import torch

from paged_reference import DIM, U2, values
from test_gpu_prompt_attn import Batch, msa  # noqa: F401

pytestmark = pytest.mark.gpu


def check_large(b, got):
    """The bounds above for every row."""
    o, lse = got
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    hkv, at = b.k.shape[1], 0
    G = b.q.shape[1] // hkv
    scale = b.scale if b.scale else DIM ** -0.5
    for s, (ql, kl) in enumerate(zip(b.q_lens, b.kv_lens)):
        rows = b.rows[s].cuda()
        if b.visible is None:
            seen = torch.arange(kl, device="cuda")[None, :] <= kl - ql + torch.arange(ql, device="cuda")[:, None]
        else:
            seen = torch.ones(ql, kl, dtype=torch.bool, device="cuda")
            seen[:, kl - ql:] = b.visible[s].cuda()
        for h in range(b.q.shape[1]):
            kd, vd = values(b.k, b.ks, rows, h // G), values(b.v, b.vs, rows, h // G)
            qd = b.q[at:at + ql, h].double()
            logits = (qd @ kd.T * scale).masked_fill(~seen, -math.inf)
            err = 130 * U2 * scale * (qd.abs() @ kd.abs().T)
            err += 2.0 ** -17 * scale * qd.abs().amax(dim=1)[:, None] * kd.abs().sum(dim=1)[None, :]
            top, most = logits.amax(dim=1, keepdim=True), logits.masked_fill(~seen, 0).abs().amax(dim=1, keepdim=True)
            err = err + 4 * U2 * most + 1
            worst = err.masked_fill(~seen, 0).amax(dim=1, keepdim=True)
            assert ((lse[at:at + ql, h, None].double() - top).abs() <= 2 * worst + math.log(kl)).all()
            near = seen & (logits + 2 * err + 60 >= (logits - 2 * err).amax(dim=1, keepdim=True))
            for i in range(ql):
                v = vd[near[i]]
                slack = (2.0 ** -8 + 2.0 ** -10) * v.abs().amax(dim=0) + 2.0 ** -50 * vd.abs().amax()
                x = o[at + i, h].double()
                assert (x >= v.amin(dim=0) - slack).all() and (x <= v.amax(dim=0) + slack).all(), (s, h, i)
        at += ql


@pytest.mark.parametrize("lens", [([40, 3], [300, 700]), ([9], [6000])])   # whole, and cut into runs
@pytest.mark.parametrize("v_gain", [0.6, 400.0, 3e4, 2.0 ** 40])   # V's scales below and above 1
@pytest.mark.parametrize("q_gain,k_up", [(1e6, 0), (1e8, 0), (1e10, 0), (2.0, 24), (2.0, 27), (2.0, 31), (2.0, 45), (2.0, 60)])
def test_large_finite_logits(msa, lens, v_gain, q_gain, k_up):
    b = Batch(msa, *lens, 8, 2, "fp8", seed=61, q_gain=q_gain, tree=k_up == 27)
    b.vs *= v_gain
    b.ks *= 2.0 ** k_up
    ws = msa.workspace(b.prob, b.op())
    got = b.run(ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    check_large(b, got)
