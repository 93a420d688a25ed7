"""A whole step in one graph: tables, rows and attention of new tokens, replayed while the cache grows.

The attention's total_k and max_seqlen_k are what the table has room for; every replay is judged against 64 bits (bounds as in
test_gpu_prompt_attn).
"""
import pytest
import torch

from paged_reference import PAGE
from test_gpu_many_tokens_step import Loop, msa, same_bits  # noqa: F401
from test_gpu_prompt_attn import DIM, check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("width,first,new", [(5, [100, 300, 7], [1, 1, 1]), (5, [0, 120, 256], [3, 0, 9]), (40, [100, 4500, 7], [2, 2, 40])])
def test_a_step_follows_the_cache(msa, fp8, tree, width, first, new):
    S, hq, hkv, n, pages = 3, 16, 2, sum(new), 130
    lp = Loop(msa, S, hq, hkv, fp8, pages=pages, width=width, seed=3)
    lp.grow(first)
    dev_new = torch.tensor(new, dtype=torch.int32, device="cuda")
    x = torch.empty(n, (hq + 2 * hkv) * DIM, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([hq * DIM, hkv * DIM, hkv * DIM], dim=1)
    k, v, qs = k.view(n, hkv, DIM), v.view(n, hkv, DIM), torch.empty(n, hq, DIM, dtype=torch.bfloat16, device="cuda")
    outs = dict(cu_q=torch.zeros(S + 1, dtype=torch.int32, device="cuda"), cu_k=torch.zeros(S + 1, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(n, dtype=torch.int64, device="cuda"), positions=torch.zeros(n, dtype=torch.int32, device="cuda"))
    prob = msa.Problem(outs["cu_q"], outs["cu_k"], n, S * width * PAGE, max(new), width * PAGE, hq, hkv, 128, 16)
    op = msa.Op.TREE_ATTN if tree else msa.Op.DENSE_ATTN_PREFILL
    ws, ws_t, ws_a = msa.workspace(prob, op), msa.extend_workspace(S), msa.append_workspace(pages)
    see = [torch.tril(torch.rand(m, m) < 0.6) for m in new]
    words = -(-max(new) // 32)
    full = torch.cat([torch.nn.functional.pad(m, (0, words * 32 - m.shape[1])) for m in see])
    bits = (full.view(n, words, 32).long() << torch.arange(32)).sum(-1)
    bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).cuda()
    o, lse = torch.empty_like(qs), torch.empty(n, hq, device="cuda")

    def attend(**kw):
        caches = (lp.k, lp.v, *lp.scales(), lp.table)
        if tree:
            return (msa.msa_tree_attn_paged_fp8 if fp8 else msa.msa_tree_attn_paged)(prob, qs, *caches, bits, **kw)
        return (msa.msa_dense_attn_prefill_paged_fp8 if fp8 else msa.msa_dense_attn_prefill_paged)(prob, qs, *caches, **kw)

    def step():
        msa.msa_extend_block_table(lp.device_lens, dev_new, lp.free, lp.table, n, taken=lp.taken, taken_out=lp.taken,
                                   new_lengths=lp.device_lens, num_pages=pages, ws=ws_t, **outs)
        if fp8:
            msa.msa_append_paged_fp8(k, v, outs["slots"], lp.k, lp.v, lp.ks, lp.vs, ws=ws_a)
        else:
            msa.msa_append_paged(k, v, outs["slots"], lp.k, lp.v)
        qs.copy_(q.reshape(n, hq, DIM))
        attend(o=o, lse=lse, ws=ws)

    x.normal_(generator=lp.gen)
    step()   # before the capture
    lp.lens = [a + b for a, b in zip(lp.lens, new)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(30):
        x.normal_(generator=lp.gen)
        o.fill_(7)
        g.replay()
        lp.lens = [a + b for a, b in zip(lp.lens, new)]
        assert lp.device_lens.tolist() == lp.lens and msa.msa_read_device_status(ws) == 0
        if i % 7 == 0 or i == 29:
            check((o, lse), reference(new, lp.lens, lp.key_rows(), qs, lp.k, lp.v, lp.ks, lp.vs, 0.0, see if tree else None), f"replay {i}")
        assert same_bits((o, lse), attend())


def test_more_keys_than_total_k(msa):
    """The bound is one: more keys than total_k make the kernels skip the call."""
    lp = Loop(msa, 2, 16, 2, False)
    lp.grow([300, 40])
    prob, q = lp.grow([9, 1])
    prob.total_k -= 1
    ws = msa.workspace(prob, msa.Op.DENSE_ATTN_PREFILL)
    o = torch.full_like(q, 3)
    msa.msa_dense_attn_prefill_paged(prob, q.contiguous(), lp.k, lp.v, lp.table, o=o, ws=ws)
    assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_SEQLENS and (o == 3).all()
