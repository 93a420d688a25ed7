"""GPU: what a CTA of the dense decode carries from unit to unit of a run (running maximum, sum, O's exponent) and from
segment to segment, for small, middle and large groups.

The number of KV heads leaves the batch one run or a few, so a CTA takes many units of a sequence; that follows from
the SM count, and the tests assert it."""
import math

import pytest
import torch

from paged_reference import DIM, PAGE, dense_reference, quantize_pages, rows_of
from test_gpu_dense_decode import LENS, Batch
from test_gpu_dense_heads_apart import one_run_heads

pytestmark = pytest.mark.gpu

GROUPS = [8, 24, 40, 128]  # one CTA of 16 heads, of 32, tcgen05 with idle rows, without


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_05_gb300 as m
    torch.cuda.set_device(0)
    return m


def units_per_run(lens, group, hkv):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    unit = 128 if group > 32 else 64
    units = sum(-(-n // unit) for n in lens)
    runs = max(1, min(sms * (2 if group <= 16 else 1) // hkv, max(1, 320 // hkv), units))
    return units // runs


def to_fp8(b):
    """Quantizes a bf16 batch; pages of nobody and rows past the sequences' ends hold the NaN code."""
    unused = b.k[:, 0, 0].isnan() | b.v[:, 0, 0].isnan()
    b.fp8 = True
    b.k, b.ks = quantize_pages(b.k.nan_to_num(0.0))
    b.v, b.vs = quantize_pages(b.v.nan_to_num(0.0))
    b.k[unused] = b.v[unused] = 0x7F


def follow(b, group, ramp, noise):
    """Every head of a group a little beside one direction, and keys along it: logits of about 45 nats a unit of `ramp`."""
    S = len(b.lens)
    q = b.q.float().view(S, -1, group, DIM)
    q = q[:, :, :1] + noise * q
    b.q = q.to(torch.bfloat16).view(S, -1, DIM)
    for s, n in enumerate(b.lens):
        rows = rows_of(b.host_table, s, n).cuda()
        b.k[rows] = (q[s, :, 0][None] * ramp(torch.arange(n, device="cuda"))[:, None, None]).to(torch.bfloat16)


RAMPS = {
    "up": lambda j: 4 * j / 2000 - 2,             # some 17 powers of two a unit of 128 keys
    "down": lambda j: 2 - 4 * j / 2000,
    "waves": lambda j: torch.sin(j * 0.007),      # up and down over a few units
    "steps": lambda j: (j // 384) * 0.5 - 1.5,    # a jump now and then
    "alternate": lambda j: (j // 128) % 2 * 2.0 - 1,  # the units of one parity far above those of the other
}


@pytest.mark.parametrize("ramp", list(RAMPS))
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", GROUPS)
def test_the_maximum_moves_inside_a_run(msa, group, fp8, ramp):
    hkv = one_run_heads(group)
    b = Batch(msa, [2000, 385, 130], group * hkv, hkv, False, True, seed=group)
    follow(b, group, RAMPS[ramp], 0.05)
    if fp8:
        to_fp8(b)
    assert units_per_run(b.lens, group, hkv) >= 8
    b.check(msa)


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("group", GROUPS)
def test_page_scales_move_inside_a_run(msa, group, order):
    """V scales from 2^-60 to 2^40 over the pages of a sequence, K scales over 2^12."""
    hkv = one_run_heads(group)
    b = Batch(msa, [2000, 385, 130], group * hkv, hkv, True, True, seed=group)
    n = b.vs.shape[0]
    at = torch.randperm(n, generator=torch.Generator().manual_seed(3))
    if order != "mixed":
        pages = [p for p in b.host_table.flatten().tolist() if p >= 0]
        at[torch.tensor(pages + sorted(set(range(n)) - set(pages)))] = torch.arange(n)
        if order == "down":
            at = n - 1 - at
    b.vs *= (2.0 ** torch.linspace(-60, 40, n))[at].cuda()[:, None]
    b.ks *= (2.0 ** torch.linspace(-12, 0, n)).cuda()[:, None]
    b.q *= torch.tensor([2.0 ** -30, 2.0 ** 8, 1.0], device="cuda").to(torch.bfloat16).view(3, 1, 1)
    assert units_per_run(b.lens, group, hkv) >= 8
    b.check(msa)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", GROUPS)
def test_first_units_without_weight(msa, group, fp8):
    """The first keys' logits are -inf: of whole units, of part of one, of all but the last key's.  In E4M3 the pages
    that do not count have V scales that are 2^60 times the others'."""
    hkv = one_run_heads(group)
    lens, none = [1700, 400, 257, 130], [900, 128, 256, 100]
    b = Batch(msa, lens, group * hkv, hkv, False, False, seed=group)
    if fp8:
        none = [n // PAGE * PAGE for n in none]  # whole pages: a scale that makes their codes pass fp32
    b.q[:, :, 0] = 16.0
    for s, n in enumerate(lens):
        b.k[rows_of(b.host_table, s, n).cuda(), :, 0] = -1.0
    if fp8:
        to_fp8(b)
        for s, m in enumerate(none):
            pages = b.host_table[s, :m // PAGE].cuda().long()
            rows = rows_of(b.host_table, s, m).cuda()
            b.k[rows] = 0x80  # -0
            b.k[rows, :, 0] = 0xFE  # -448
            b.ks[pages] = 1e38
            b.vs[pages] *= 2.0 ** 60
    else:
        for s, m in enumerate(none):
            b.k[rows_of(b.host_table, s, m).cuda(), :, 0] = -math.inf
    assert units_per_run(lens, group, hkv) >= 8
    ws = b.ws(msa)
    ws.fill_(0xFF)
    o, lse = b.call(msa, ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    # in 64 bits: the same batch without those keys (they are whole pages or the front of one: mask them by hand)
    for s, (n, m) in enumerate(zip(lens, none)):
        rows = rows_of(b.host_table, s, n)[m:].cuda()
        for g in range(0, hkv, 37):
            hs = slice(g * group, (g + 1) * group)
            if fp8:
                kd, vd = (x.view(torch.float8_e4m3fn)[rows, g].double() * sc[rows // PAGE, g].double()[:, None]
                          for x, sc in ((b.k, b.ks), (b.v, b.vs)))
            else:
                kd, vd = b.k[rows, g].double(), b.v[rows, g].double()
            qd, u2 = b.q[s, hs].double(), 2.0 ** -23
            logits = qd @ kd.T * DIM ** -0.5
            err = 130 * u2 * DIM ** -0.5 * (qd.abs() @ kd.abs().T)
            top = torch.logsumexp(logits, dim=1)
            p = torch.exp(logits - top[:, None])
            lse_tol = (p * err).sum(1) + u2 + (n + 16) * u2 + 4 * u2 * (top.abs() + logits.abs().amax(1))
            rel = err + lse_tol[:, None] + 4 * u2 * logits.abs() + (2.0 ** -11 if fp8 else 2.0 ** -16)
            want = p @ vd
            tol = 2.0 ** -8 * want.abs() + (p * rel) @ vd.abs() + (n + 16) * u2 * (p @ vd.abs())
            if fp8:
                tol += 2.0 ** -24 * n * p.amax(1)[:, None] * vd.abs().amax(0)[None]
            assert ((o[s, hs].double() - want).abs() <= tol).all(), (s, g)
            assert ((lse[s, hs].double() - top).abs() <= lse_tol).all(), (s, g)


@pytest.mark.parametrize("power", [8, 12, 16, 19, 20, 21, 24, 26, 31, 40, 60, 100])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", GROUPS)
def test_large_logits(msa, group, fp8, power):
    """All keys of one large logit, 3 * 2^power (exact in every step but the last product), and then a second level of
    keys at half of it: the weights are 1 / (number of the upper level's keys), whatever the size.

    Bounds: the weights' rounding 2^-16 (E4M3 2^-11), a sum over n keys (n + 16) 2^-23, the output's 2^-8; lse and the
    logits in log2 units are three fp32 roundings of the logit; the weights that are added up, G of them, each off
    by 2^-23 (16 + the rounding of logit and maximum, which are the same number)."""
    hkv = one_run_heads(group)
    lens = [1000, 300]
    b = Batch(msa, lens, group * hkv, hkv, False, True, seed=group, scale=1.0)
    b.q.zero_()
    b.q[:, :, 0] = 2.0 ** (power // 2)
    b.q[:, 1::2, 0] = 2.0 ** (power // 2) * 1.5   # heads of two sizes beside one another
    upper = [torch.ones(n, dtype=torch.bool) for n in lens]
    upper[0] = (torch.arange(lens[0]) * 7) % 3 != 1
    upper[0][:200] = False   # the upper level begins inside the run
    for s, n in enumerate(lens):
        rows = rows_of(b.host_table, s, n).cuda()
        b.k[rows] = 0
        b.k[rows, :, 0] = torch.where(upper[s], 3.0, 1.5).cuda().to(torch.bfloat16)[:, None] * 2.0 ** (power - power // 2)
    if fp8:
        to_fp8(b)
        pages = b.host_table.flatten()
        pages = pages[pages >= 0].cuda().long()
        b.ks[pages] = 2.0 ** (power - power // 2 - 7)   # codes 384 and 192 in every page
        for s, n in enumerate(lens):
            rows = rows_of(b.host_table, s, n).cuda()
            b.k[rows, :, 0] = torch.where(upper[s], 384.0, 192.0).cuda().to(torch.float8_e4m3fn).view(torch.uint8)[:, None]
        b.vs[pages] *= torch.rand(len(pages), 1, device="cuda") + 0.5
    assert units_per_run(lens, group, hkv) >= 8
    before = b.weight.clone()
    ws = b.ws(msa)
    o, lse = b.call(msa, ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    logit = b.q[..., 0].double() * 3.0 * 2.0 ** (power - power // 2)
    u2 = 2.0 ** -23
    for s, n in enumerate(lens):
        rows, count = rows_of(b.host_table, s, n)[upper[s]].cuda(), int(upper[s].sum())
        v = b.v[rows]
        v = v.view(torch.float8_e4m3fn).double() * b.vs[rows // PAGE].double()[..., None] if fp8 else v.double()
        want = v.mean(0)[:, None]                                     # [hkv, 1, 128]
        size = v.abs().mean(0)[:, None]
        small = 2.0 ** -24 * n / count * v.abs().amax(0)[:, None] if fp8 else 0.0
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 if fp8 else 2.0 ** -16) * size + (n + 16) * u2 * size + small
        got = o[s].double().view(hkv, group, DIM)
        assert torch.isfinite(got).all() and ((got - want).abs() <= tol).all(), float((got - want).abs().max())
        exact = logit[s] + math.log(count)
        assert ((lse[s].double() - exact).abs() <= 3 * u2 * exact.abs() + (n + 16) * u2).all()
        added = (b.weight[s, :, :n].double() - before[s, :, :n].double()).cpu()
        each = torch.where(upper[s], group / count, 0.0).double()
        wtol = each * (n + 32) * u2 + u2 * (before[s, :, :n].double().cpu() + each)
        # logits below 2^10 in log2 units are not rounded before the sum: the maximum's rounding, 2^-14, is in the weights
        assert ((added - each).abs() <= wtol + each * 2.0 ** -14).all()


@pytest.mark.parametrize("scale", [2e29, 1e-30, 1e-44])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [8, 128])
def test_softmax_scales_at_the_ends_of_the_range(msa, group, fp8, scale):
    """A query of zeros, or logits of next to nothing: uniform weights whatever the factor in front of the product."""
    b = Batch(msa, [300, 70], group, 1, fp8, True, seed=5, scale=scale)
    if scale > 1:
        b.q.zero_()
        b.q[0, :, 0] = 2.0 ** 100  # a factor past fp32 on products of zero
        b.k[rows_of(b.host_table, 0, 300).cuda()] = 0
    elif fp8:
        b.ks *= 1e-30
    b.weight.zero_()
    o, lse = b.call(msa)
    for s, n in enumerate(b.lens):
        v = b.v[rows_of(b.host_table, s, n).cuda(), 0]
        if fp8:
            v = v.view(torch.float8_e4m3fn).double() * b.vs[rows_of(b.host_table, s, n).cuda() // PAGE, 0].double()[:, None]
        v = v.double()
        tol = 2.0 ** -8 * v.mean(0).abs() + (2.0 ** -11 + (n + 16) * 2.0 ** -23) * v.abs().mean(0)
        tol = tol + (2.0 ** -24 * v.abs().amax(0) if fp8 else 0)
        assert ((o[s].double() - v.mean(0)).abs() <= tol).all()
        assert ((lse[s].double() - math.log(n)).abs() <= (n + 16) * 2.0 ** -23).all()
        assert ((b.weight[s, 0, :n].double() - group / n).abs() <= group / n * (n + 32) * 2.0 ** -23).all()


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("group", [8, 24, 128])
def test_a_scale_that_is_nan_shows(msa, group, which):
    """In its own sequence and KV head, and nowhere else."""
    b = Batch(msa, [700, 130], group * 2, 2, True, False, seed=6)
    clean_o, clean_lse = b.call(msa)
    getattr(b, which)[b.host_table[0, 3].item(), 1] = math.nan
    o, lse = b.call(msa)
    assert o[0, group:].isnan().all() and (which == "vs" or lse[0, group:].isnan().all())
    assert torch.equal(o[0, :group], clean_o[0, :group]) and torch.equal(o[1], clean_o[1])
    assert torch.equal(lse[0, :group], clean_lse[0, :group]) and torch.equal(lse[1], clean_lse[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(40, 1), (128, 1), (96, 2)])
@pytest.mark.parametrize("lens", ["127", "128", "129", "ragged", "trailing_empty", "all_empty", "long_and_short", "many_short"])
def test_lengths_large_groups(msa, lens, hq, hkv, fp8):
    Batch(msa, LENS[lens], hq, hkv, fp8, True, seed=len(lens)).check(msa)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,group", [
    ([(i * 53) % 400 for i in range(310)], 40),         # up to three units each, more sequences than runs
    ([(i * 53) % 400 for i in range(310)], 128),
    ([1 + (i * 29) % 128 for i in range(200)], 64),     # one unit each: both parities, Q for every one
    ([40000] + [(i * 31) % 300 for i in range(2000)], 48),
])
def test_many_segments_to_a_run_large_groups(msa, lens, group, fp8):
    Batch(msa, lens, group, 1, fp8, True, seed=group).check(msa)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [40, 128])
def test_a_run_of_many_segments(msa, group, fp8):
    """All sequences in one CTA per KV head, one after another: one, two and more units, empty ones between."""
    hkv = one_run_heads(group)
    lens = [1, 128, 0, 129, 256, 257, 0, 0, 5, 300, 384, 385, 64, 128, 128, 700, 2]
    assert units_per_run(lens, group, hkv) >= 20
    Batch(msa, lens, group * hkv, hkv, fp8, True, seed=group).check(msa)
