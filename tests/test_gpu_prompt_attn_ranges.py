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

from paged_reference import DIM, U2, blocks, values
from test_gpu_prompt_attn import Batch, check, msa, reference  # noqa: F401

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


# ------------------------------------------------------------------------------------------------ V's page scales
# log2 of a scale is at most 2^8; it is added to a logit, to a reference and to their difference once a block, each sum rounded to
# 2^-24 of its value: 2^-14 a block in all is more than these weights and sums are off by beside test_gpu_prompt_attn's bounds.
def with_scales(b):
    o, lse, to, tl = b.want()
    extra = 2.0 ** -14 * (blocks(max(b.kv_lens)) + 1)
    return o, lse, to + extra * spread(b), tl + extra


def spread(b):
    """sum_j p_j |v_j| of every row: what a relative error of the weights counts with."""
    return reference(b.q_lens, b.kv_lens, b.rows, b.q, b.k, b.v & 0x7F, b.ks, b.vs, b.scale, b.visible)[0]


SHAPES = [([40, 3], [300, 700], False), ([9], [6000], False), ([9, 30], [400, 3000], True), ([1], [20000], True)]


@pytest.mark.parametrize("q,kv,tree", SHAPES)
@pytest.mark.parametrize("up", [-122, -119, -90, -60, 60, 90, 110])
def test_every_scale_of_v(msa, q, kv, tree, up):
    """All pages' scales 2^up times what they were: so are the results."""
    b = Batch(msa, q, kv, 8, 2, "fp8", seed=67, tree=tree)
    b.vs = b.vs * 2.0 ** up   # (rounded where that is below the normal numbers)
    ws = msa.workspace(b.prob, b.op())
    o, lse = b.run(ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    b.vs = b.vs.double() * 2.0 ** -up
    ro, rl, to, tl = with_scales(b)
    to = to + 2.0 ** (-133 - up)   # bf16's smallest step
    assert ((o.double() * 2.0 ** -up - ro).abs() <= to).all()
    assert ((lse.double() - rl).abs() <= tl).all()


@pytest.mark.parametrize("q,kv,tree", SHAPES)
@pytest.mark.parametrize("lo,hi", [(-119, 0), (-40, 100), (-119, 110)])
@pytest.mark.parametrize("gain", [2.0, 40.0])
def test_pages_of_any_scale_side_by_side(msa, q, kv, tree, lo, hi, gain):
    """Pages with every scale that rows can ask for in one sequence, a scale of 0 among them; large logits in either."""
    b = Batch(msa, q, kv, 8, 2, "fp8", seed=71, q_gain=gain, tree=tree)
    gen = torch.Generator(device="cuda").manual_seed(hi)
    b.vs *= 2.0 ** torch.randint(lo, hi + 1, b.vs.shape, generator=gen, device="cuda").float()
    b.vs[b.table[0, 1].long()] = 0
    ws = msa.workspace(b.prob, b.op())
    o, lse = b.run(ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    sv = b.vs
    b.vs = torch.where(sv == 0, 2.0 ** -200, sv.double())   # (the reference divides by a scale)
    check((o, lse), with_scales(b))


@pytest.mark.parametrize("up", [-117, -60, 100])
def test_pages_as_append_writes_them(msa, up):
    """The smallest and large rows that msa_append_paged_fp8 takes: the attention reads the pages that it makes."""
    b = Batch(msa, [300, 3], [300, 700], 8, 2, "fp8", seed=73)
    gen = torch.Generator(device="cuda").manual_seed(1)
    new = [torch.randn(1000, 2, DIM, device="cuda", generator=gen) for _ in range(2)]
    slots = torch.cat(b.rows).cuda()
    rows = [new[0].to(torch.bfloat16), (new[1] * 2.0 ** up).to(torch.bfloat16)]
    msa.msa_append_paged_fp8(*rows, slots, b.k, b.v, b.ks, b.vs, ws=msa.append_workspace(b.k.shape[0] // 128))
    assert (b.vs[b.table[1, :6].long()] * 2.0 ** -up).amax() < 1
    o, lse = b.run()
    b.vs = b.vs.double() * 2.0 ** -up
    ro, rl, to, tl = with_scales(b)
    assert ((o.double() * 2.0 ** -up - ro).abs() <= to + 2.0 ** (-133 - up)).all()
    assert ((lse.double() - rl).abs() <= tl).all()
