"""GPU: msa_add_rms_norm(_fp8) against 64 bits.

Bounds: the sum is one bf16 rounding (2^-8 of the value) of an fp32 sum.  y = h r gamma: r comes from an fp32 sum of
`width` squares in a fixed order (at most (width + 8) 2^-24 of its value, half of that after the root) and four fp32
roundings; bf16 adds 2^-8.  An E4M3 code is off by half a step: 2^-4 of the value, or 2^-10 (half the subnormal step) times
the scale.
"""
import math

import pytest
import torch

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


def _inputs(rows, width, seed, residual=True, gain=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16)
    x = rnd(rows, width) * gain
    return x, (rnd(rows, width) * 4 * gain if residual else None), 1 + rnd(width) / 8


def _reference(x, res, gamma, eps):
    h = x.double() + (res.double() if res is not None else 0)
    y = h / torch.sqrt((h * h).mean(dim=-1, keepdim=True) + eps) * gamma.double()
    return h, y


def _check(msa, x, res, gamma, eps=1e-6):
    width = x.shape[-1]
    h, y = _reference(x, res, gamma, eps)
    rel = (width / 2 + 16) * 2.0 ** -24
    total, got = msa.msa_add_rms_norm(x, gamma, residual=res, eps=eps)
    assert ((total.double() - h).abs() <= 2.0 ** -8 * h.abs() + 2.0 ** -24 * h.abs()).all()
    assert ((got.double() - y).abs() <= (2.0 ** -8 + 2 * rel) * y.abs() + 2.0 ** -130).all()
    total8, codes, scale = msa.msa_add_rms_norm_fp8(x, gamma, residual=res, eps=eps)
    assert torch.equal(total, total8)
    top = y.abs().amax(dim=-1)
    want = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert ((scale.double() - want).abs() <= 4 * rel * want).all()
    val = codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]
    assert ((val - y).abs() <= (2.0 ** -4 + 4 * rel) * y.abs() + 2.0 ** -10 * 1.01 * want[..., None]).all()


@pytest.mark.parametrize("width", [1, 2, 7, 8, 9, 31, 64, 100, 128, 1000, 1001, 1024, 2049, 4096, 5120, 8184, 8192,
                                   12345, 16384, 16385, 32768, 32776, 65535, 65536])
@pytest.mark.parametrize("residual", [True, False])
def test_widths(msa, width, residual):
    _check(msa, *_inputs(3, width, width, residual))


@pytest.mark.parametrize("rows", [1, 2, 151, 4097])
def test_rows(msa, rows):
    _check(msa, *_inputs(rows, 512, rows))
    _check(msa, *_inputs(rows, 513, rows))


def test_shapes_with_leading_dimensions(msa):
    x, res, gamma = _inputs(6, 256, 1)
    total, y = msa.msa_add_rms_norm(x.view(2, 3, 256), gamma, residual=res.view(2, 3, 256))
    flat = msa.msa_add_rms_norm(x, gamma, residual=res)
    assert total.shape == (2, 3, 256) and torch.equal(total.view(6, 256), flat[0]) and torch.equal(y.view(6, 256), flat[1])


def test_no_rows(msa):
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    assert msa.msa_add_rms_norm(x, gamma)[1].shape == (0, 128)
    assert msa.msa_add_rms_norm_fp8(x, gamma)[2].shape == (0,)


@pytest.mark.parametrize("width", [1000, 1001, 20001])
def test_in_place(msa, width):
    x, res, gamma = _inputs(5, width, 2)
    want = msa.msa_add_rms_norm(x, gamma, residual=res)
    want8 = msa.msa_add_rms_norm_fp8(x, gamma, residual=res)
    r2, x2 = res.clone(), x.clone()
    total, y = msa.msa_add_rms_norm(x2, gamma, residual=r2, sum_out=r2, y=x2)
    assert total is r2 and torch.equal(r2, want[0]) and torch.equal(x2, want[1])
    x3 = x.clone()
    got8 = msa.msa_add_rms_norm_fp8(x3, gamma, residual=res, sum_out=x3)
    assert torch.equal(x3, want8[0]) and torch.equal(got8[1], want8[1]) and torch.equal(got8[2], want8[2])


def test_zero_large_and_small_rows(msa):
    x, res, gamma = _inputs(4, 384, 3)
    x[0], res[0] = 0, 0
    x[1] *= 2.0 ** 50
    x[2], res[2] = x[2] * 2.0 ** -60, res[2] * 2.0 ** -60
    _check(msa, x, res, gamma)
    total, codes, scale = msa.msa_add_rms_norm_fp8(x, gamma, residual=res)
    assert scale[0] == 1 and (codes[0] == 0).all()


def test_nan_stays_in_its_row(msa):
    x, res, gamma = _inputs(3, 200, 4)
    clean = msa.msa_add_rms_norm(x, gamma, residual=res)
    x[1, 7] = math.nan
    total, y = msa.msa_add_rms_norm(x, gamma, residual=res)
    assert y[1].isnan().all() and torch.equal(y[0], clean[1][0]) and torch.equal(y[2], clean[1][2])
    codes = msa.msa_add_rms_norm_fp8(x, gamma, residual=res)[1]
    assert codes.view(torch.float8_e4m3fn)[1].float().isnan().all()


def test_repeats_graph_and_stream(msa):
    x, res, gamma = _inputs(300, 2048, 5)
    outs = torch.empty_like(x), torch.empty_like(x)
    call = lambda: msa.msa_add_rms_norm(x, gamma, residual=res, sum_out=outs[0], y=outs[1])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        x.normal_()
        g.replay()
        got = [t.clone() for t in outs]
        want = msa.msa_add_rms_norm(x, gamma, residual=res)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = msa.msa_add_rms_norm(x, gamma, residual=res)
    side.synchronize()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
