"""K_idx rows alone into bf16 index pages, beside K and V in E4M3 pages (what msa_forward_decode_paged_fp8 reads): refusals on the
host, rows on the GPU (exact)."""
import pytest
import torch

from test_many_tokens_abi_cpu import FAKE, accepted, msa  # noqa: F401

FINE = dict(k=None, sk=0, v=None, sv=0, i=FAKE, si=128, slots=FAKE, tokens=9, hkv=0, d=128, kc=None, vc=None, ic=FAKE, pages=100, ws=None, n=0)


def test_refusals(msa):
    def call(**kw):
        return msa._lib.msa_append_paged(*{**FINE, **kw}.values(), None)

    if not torch.cuda.is_available():
        assert accepted(call()) and accepted(call(d=64, si=64)) and accepted(call(hkv=4)) and accepted(call(ws=FAKE, n=256))
        assert accepted(call(tokens=0, i=None, slots=None))
    assert call(i=None) == -1 and call(ic=None) == -1 and call(slots=None) == -1
    for arg in ("k", "v", "kc", "vc"):   # none of the four, or all
        assert call(**{arg: FAKE}) == -1, arg
        assert call(**{arg: FAKE, "hkv": 1, "sk": 128, "sv": 128}) == -1, arg
    assert call(d=32) == -2 and call(si=120) == -1 and call(si=132) == -3 and call(i=FAKE + 8) == -3 and call(ic=FAKE + 8) == -3
    assert call(pages=0) == -1 and call(tokens=-1) == -1 and call(ws=FAKE, n=255) == -4


@pytest.mark.gpu
@pytest.mark.parametrize("d_idx", [64, 128])
@pytest.mark.parametrize("n", [1, 7, 5000])
def test_rows(msa, d_idx, n):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    pages = 50
    gen = torch.Generator().manual_seed(n)
    slots = torch.randperm(pages * 128, generator=gen)[:n].cuda()
    if n > 3:
        slots[2] = -1
    x = torch.randn(n, d_idx + 72, generator=gen).to(torch.bfloat16).cuda()[:, 72:]
    cache = torch.randn(pages * 128, d_idx, generator=gen).to(torch.bfloat16).cuda()
    want = cache.clone()
    want[slots[slots >= 0]] = x[slots >= 0]
    ws = msa.append_workspace(pages)
    msa.msa_append_paged(None, None, slots, None, None, k_idx=x, k_idx_cache=cache, ws=ws)
    assert msa.msa_read_device_status(ws) == 0 and torch.equal(cache, want)
    k = torch.zeros(n, 2, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k=k), dict(k_cache=cache)):
        with pytest.raises(ValueError, match="needed"):
            msa.msa_append_paged(bad.get("k"), None, slots, bad.get("k_cache"), None, k_idx=x, k_idx_cache=cache)
    with pytest.raises(ValueError, match="needed"):
        msa.msa_append_paged_fp8(None, None, slots, None, None, k, k, k_idx=x, k_idx8_cache=cache, k_idx_scale=k)


@pytest.mark.gpu
@pytest.mark.parametrize("topk", [3])
def test_a_sparse_step_over_e4m3_pages_and_bf16_index_pages(msa, topk):
    """The pages that the two calls fill give the sparse decode what packed rows give it."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    hq, hkv, lens, pages = 32, 2, [700, 129, 1500], 40
    gen = torch.Generator().manual_seed(5)
    x = [torch.randn(sum(lens), w, 128, generator=gen).to(torch.bfloat16).cuda() for w in (hkv, hkv, 1)]
    k8, v8 = (torch.zeros(pages * 128, hkv, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(pages, hkv, device="cuda") for _ in range(2))
    ki = torch.zeros(pages * 128, 128, dtype=torch.bfloat16, device="cuda")
    free = torch.randperm(pages, generator=gen).to(torch.int32).cuda()
    table = torch.zeros(3, 12, dtype=torch.int32, device="cuda")
    none, new = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([0] * 3, lens))
    _, cu_k, slots, _, _ = msa.msa_extend_block_table(none, new, free, table, sum(lens), num_pages=pages)
    msa.msa_append_paged_fp8(x[0], x[1], slots, k8, v8, ks, vs)
    msa.msa_append_paged(None, None, slots, None, None, k_idx=x[2][:, 0], k_idx_cache=ki)
    prob = msa.problem_from_seqlens([1] * 3, lens, hq, hkv, 128, topk)
    assert torch.equal(cu_k, prob.cu_k)
    q = torch.randn(3, hq, 128, generator=gen).to(torch.bfloat16).cuda()
    qi = torch.randn(3, hkv, 128, generator=gen).to(torch.bfloat16).cuda()
    idx, o, lse = msa.msa_forward_decode_paged_fp8(prob, q, k8, v8, ks, vs, qi, ki, table)
    # the index branch from the packed rows, and the same attention in 64 bits
    deq = [(c[slots].view(torch.float8_e4m3fn).double() * s.double()[slots // 128][:, :, None]) for c, s in ((k8, ks), (v8, vs))]
    assert torch.equal(idx, msa.msa_index_topk(prob, qi, x[2][:, 0].contiguous()))
    at = 0
    for s, n in enumerate(lens):
        for h in range(hq):
            g = h // (hq // hkv)
            keys = torch.cat([torch.arange(b * 128, min(n, b * 128 + 128)) for b in idx[s, g].tolist() if b >= 0]).cuda() + at
            z = deq[0][keys, g] @ q[s, h].double() * 128 ** -0.5
            p = torch.softmax(z, 0)
            assert (p @ deq[1][keys, g] - o[s, h].double()).abs().max() < 2 ** -6 * (p @ deq[1][keys, g].abs()).max()
        at += n
