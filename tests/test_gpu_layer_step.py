"""GPU: decode steps of a full-attention layer with the operators together -- residual sum and norm, the index prologue on
the normed states, dense attention over a paged cache that gains a token a step and accumulates weights, eviction, and
attention over what was kept -- each result against 64 bits on the inputs that the step had."""
import pytest
import torch

from paged_reference import DIM, PAGE, blocks, dense_reference, evict_reference, make_tables, quantize_pages, rows_of

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


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_steps_with_eviction(msa, fp8):
    S, hq, hkv, width, budget, recent, steps = 3, 32, 4, 512, 300, 40, 4
    lens = [290, 701, 128]
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16)
    tables, pages = make_tables([n + steps for n in lens] + [budget + 1] * S, torch.Generator().manual_seed(1))
    table, new_table = tables[:S].contiguous(), tables[S:].contiguous()
    k, v = rnd(pages * PAGE, hkv, DIM), rnd(pages * PAGE, hkv, DIM)
    ks = vs = None
    if fp8:
        k, ks = quantize_pages(k)
        v, vs = quantize_pages(v)
    gamma, w_q = 1 + rnd(width) / 8, rnd(hq * DIM, width) / width ** 0.5
    w_iq, w_ik, g_q, g_k = rnd(hkv * 128, width) / width ** 0.5, rnd(128, width) / width ** 0.5, 1 + rnd(128) / 8, 1 + rnd(128) / 8
    stream_sum = rnd(S, width)
    acc = torch.zeros(S, hkv, max(lens) + steps, device="cuda")

    def attend(q, prob, tab, weight, host_lens):
        before = weight.clone()
        if fp8:
            o, lse = msa.msa_dense_attn_decode_paged_fp8(prob, q, k, v, ks, vs, tab.cuda(), weight=weight)
        else:
            o, lse = msa.msa_dense_attn_decode_paged(prob, q, k, v, tab.cuda(), weight=weight)
        ref = dense_reference(host_lens, tab, q, k, v, ks, vs)
        assert ((o.double() - ref[0]).abs() <= ref[3]).all() and ((lse.double() - ref[1]).abs() <= ref[4]).all()
        for s, n in enumerate(host_lens):
            got, want = weight[s, :, :n].double(), before[s, :, :n].double() + ref[2][s]
            assert ((got - want).abs() <= ref[5][s] + 2.0 ** -24 * want).all()
        return o

    for step in range(steps):
        now = [n + step for n in lens]
        prob = msa.problem_from_seqlens([1] * S, now, hq, hkv, 128, 16)
        x = rnd(S, width)
        old = stream_sum.clone()
        _, h = msa.msa_add_rms_norm(x, gamma, residual=stream_sum, sum_out=stream_sum)  # the stream in place
        want = x.double() + old.double()
        assert ((stream_sum.double() - want).abs() <= 2.0 ** -8 * want.abs()).all()
        # the normed states go into the index prologue and the layer's own projection
        k_idx = torch.zeros(sum(now), 128, dtype=torch.bfloat16, device="cuda")
        q_idx = msa.msa_index_prologue(prob, h, w_iq, w_ik, g_q, g_k, k_idx)
        assert torch.isfinite(q_idx).all() and (k_idx[[sum(now[:s + 1]) - 1 for s in range(S)]] != 0).any(dim=1).all()
        q = (h @ w_q.T).view(S, hq, DIM)
        acc[torch.arange(S), :, [n - 1 for n in now]] = 0  # the step's own token enters with weight 0
        attend(q, prob, table, acc, now)

    # evict, and attend over what is left
    now = [n + steps - 1 for n in lens]
    slots = evict_reference(now, acc, budget, recent)
    src = [[values_of(k, ks, table, s, now[s], g)[slots[s][g]] for g in range(hkv)] for s in range(S)]
    if fp8:
        kept, new_acc, cu = msa.msa_evict_paged_fp8(prob, k, v, ks, vs, table.cuda(), acc, new_table.cuda(), budget, recent)
    else:
        kept, new_acc, cu = msa.msa_evict_paged(prob, k, v, table.cuda(), acc, new_table.cuda(), budget, recent)
    left = [min(n, budget) for n in now]
    assert cu.tolist() == [sum(left[:s]) for s in range(S + 1)]
    for s in range(S):
        for g in range(hkv):
            assert kept[s, g, :left[s]].tolist() == slots[s][g]
            got = values_of(k, ks, new_table, s, left[s], g)
            # bf16 rows move as they are; a code's value moves by half a step of E4M3 at the new page's scale at most
            tol = (2.0 ** -4 * src[s][g].abs() + src[s][g].abs().max() / 448 * 2.0 ** -10 * 1.01) if fp8 else 0.0
            assert ((got - src[s][g]).abs() <= tol).all()
    # one more token, in the new pages
    now = [n + 1 for n in left]
    rows = torch.stack([rows_of(new_table, s, now[s])[-1] for s in range(S)]).cuda()
    if not fp8:
        k[rows], v[rows] = rnd(S, hkv, DIM), rnd(S, hkv, DIM)
    else:
        k[rows], v[rows] = 0x30, 0x28  # codes, at whatever scale the page has
        for p in (rows // PAGE).tolist():
            ks[p], vs[p] = ks[p].clamp(max=1.0), vs[p].clamp(max=1.0)
    weight = torch.zeros(S, hkv, max(now), device="cuda")
    weight[:, :, :budget] = new_acc
    prob = msa.Problem(prob.cu_q, torch.tensor([sum(now[:s]) for s in range(S + 1)], dtype=torch.int32, device="cuda"), S,
                       sum(now), 1, max(now), hq, hkv, 128, 16)
    attend(rnd(S, hq, DIM), prob, new_table, weight, now)


def values_of(cache, scale, table, s, n, g):
    rows = rows_of(table, s, n).cuda()
    x = cache[rows, g]
    return x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale.double()[rows // PAGE, g][:, None]
