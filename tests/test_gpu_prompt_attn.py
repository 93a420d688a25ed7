"""Causal attention of prompts (packed, paged, E4M3 pages) and attention of drafted trees against 64-bit references.

Error bounds (u = 2^-24; a bf16 rounding is off by at most 2^-8 of the value): a logit is an fp32 sum of 128 exact
products, off by at most 130 * 2u * scale * sum_d |q_d k_d| (tensor cores may truncate); a weight exp(s - lse) by that of
its own logit and of lse, 2^x and the fp32 steps, and by 2^-8 of itself where it meets V (E4M3 pages: 2^-11); the sum over n keys adds
(n + 16) * 2u, a rescale 2u each, of which a row has at most one per block; the output's own rounding 2^-8.  Over E4M3
pages a query's value is two codes: off by at most 2^-18 of the row's largest, 2^-17 with the sum's own.
"""
import math

import pytest
import torch

from paged_reference import DIM, PAGE, U2, make_tables, quantize_pages, rows_of, values

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


def reference(q_lens, kv_lens, key_rows, q, k, v, k_scale, v_scale, scale, visible):
    """(o, lse, o_tol, lse_tol) in 64 bits; `key_rows`: the rows of k and v of each sequence's keys; `visible`: None for
    causal, or a list of [q_len, q_len] truth values."""
    T, hq, _ = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    scale = scale if scale else DIM ** -0.5
    o = torch.zeros(T, hq, DIM, dtype=torch.float64, device=q.device)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=q.device)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    at = 0
    for s, (ql, kl) in enumerate(zip(q_lens, kv_lens)):
        if ql == 0:
            continue
        rows = key_rows[s].to(q.device)
        seen = torch.zeros(ql, kl, dtype=torch.bool, device=q.device)
        if visible is None:
            seen[:] = torch.arange(kl, device=q.device)[None, :] <= kl - ql + torch.arange(ql, device=q.device)[:, None]
        else:
            seen[:, :kl - ql] = True
            seen[:, kl - ql:] = visible[s].to(q.device)
        some = seen.any(dim=1)
        for g in range(hkv):
            kd, vd = values(k, k_scale, rows, g), values(v, v_scale, rows, g)
            for h in range(g * G, (g + 1) * G):
                qd = q[at:at + ql, h].double()
                logits = (qd @ kd.T * scale).masked_fill(~seen, -math.inf)
                err = 130 * U2 * scale * (qd.abs() @ kd.abs().T)
                if k_scale is not None:
                    err = err + 2.0 ** -17 * scale * qd.abs().amax(dim=1)[:, None] * kd.abs().sum(dim=1)[None, :]
                top = torch.logsumexp(logits, dim=1)
                p = torch.exp(logits - top.masked_fill(~some, 0.0)[:, None])
                most = logits.masked_fill(~seen, 0.0).abs().amax(dim=1)
                lt = (p * err).sum(dim=1) + U2 + (kl + 16) * U2 + 4 * U2 * (top.masked_fill(~some, 0.0).abs() + most)
                rel = err + lt[:, None] + 4 * U2 * most[:, None] + (2.0 ** -8 if k_scale is None else 2.0 ** -11)
                lse[at:at + ql, h], lse_tol[at:at + ql, h] = top, lt
                o[at:at + ql, h] = p @ vd
                o_tol[at:at + ql, h] = (2.0 ** -8 * (p @ vd).abs() + (p * rel) @ vd.abs()
                                        + (kl + 16 + kl // 128) * U2 * (p @ vd.abs()) + 2.0 ** -120)
                if v_scale is not None:  # fp16 weights below 2^-21 of the largest weight times page scale: 2^-32 of it
                    sv = v_scale.double()[rows // PAGE, g]
                    o_tol[at:at + ql, h] += 2.0 ** -32 * (p * sv).amax(dim=1)[:, None] * (vd.abs() / sv[:, None]).sum(dim=0)
        at += ql
    return o, lse, o_tol, lse_tol


def check(got, want, what=""):
    o, lse = got
    ro, rl, to, tl = want
    none = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse), none), what
    assert (o[none] == 0).all(), what
    gap = ((o.double() - ro).abs() - to).amax().item() if o.numel() else 0.0
    assert gap <= 0, f"{what}: o off by {gap} more than its bound"
    d = (lse.double() - rl).masked_fill(none, 0.0).abs()
    assert (d <= tl).all(), f"{what}: lse off by {(d - tl).amax().item()} more than its bound"


class Batch:
    """Random queries and keys of a batch in one of the three layouts, what lies behind a sequence's keys being NaN."""

    def __init__(self, msa, q_lens, kv_lens, hq, hkv, layout, seed=0, scale=0.0, q_gain=2.0, tree=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        host = torch.Generator().manual_seed(seed)
        self.msa, self.q_lens, self.kv_lens, self.layout, self.scale = msa, q_lens, kv_lens, layout, scale
        self.prob = msa.problem_from_seqlens(q_lens, kv_lens, hq=hq, hkv=hkv, d_idx=128, topk=16, scale=scale)
        self.q = (torch.randn(sum(q_lens), hq, DIM, device="cuda", generator=gen) * q_gain).to(torch.bfloat16)
        self.table, self.ks, self.vs = None, None, None
        if layout == "packed":
            n = sum(kv_lens)
            starts = [sum(kv_lens[:s]) for s in range(len(kv_lens))]
            self.rows = [torch.arange(a, a + b) for a, b in zip(starts, kv_lens)]
        else:
            table, pages = make_tables(kv_lens, host)
            self.table, n = table.cuda(), pages * PAGE
            self.rows = [rows_of(table, s, b) for s, b in enumerate(kv_lens)]
        self.k = torch.randn(n, hkv, DIM, device="cuda", generator=gen).to(torch.bfloat16)
        self.v = torch.randn(n, hkv, DIM, device="cuda", generator=gen).to(torch.bfloat16)
        if layout == "fp8":
            self.k, self.ks = quantize_pages(self.k)
            self.v, self.vs = quantize_pages(self.v)
        if layout != "packed":
            used = torch.zeros(n, dtype=torch.bool)
            for r in self.rows:
                used[r] = True
            for x in (self.k, self.v):
                x[~used.cuda()] = 0x7F if layout == "fp8" else math.nan
        self.visible = self.bits = None
        if tree:
            self.visible, words = [], max(1, -(-max(q_lens) // 32))
            rows = []
            for ql in q_lens:
                see = torch.rand(ql, ql, generator=host) < 0.4
                if ql > 2:
                    see[2] = False   # a draft that sees no draft
                self.visible.append(see)
                full = torch.rand(ql, words * 32, generator=host) < 0.5   # bits past q_len do not count
                full[:, :ql] = see
                w = (full.view(ql, words, 32).long() << torch.arange(32)).sum(-1)
                rows.append(torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32))
            self.bits = torch.cat(rows).cuda()

    def run(self, **kw):
        m = self.msa
        if self.bits is not None:
            if self.layout == "fp8":
                return m.msa_tree_attn_paged_fp8(self.prob, self.q, self.k, self.v, self.ks, self.vs, self.table,
                                                 self.bits, **kw)
            return m.msa_tree_attn_paged(self.prob, self.q, self.k, self.v, self.table, self.bits, **kw)
        if self.layout == "packed":
            return m.msa_dense_attn_prefill(self.prob, self.q, self.k, self.v, **kw)
        if self.layout == "paged":
            return m.msa_dense_attn_prefill_paged(self.prob, self.q, self.k, self.v, self.table, **kw)
        return m.msa_dense_attn_prefill_paged_fp8(self.prob, self.q, self.k, self.v, self.ks, self.vs, self.table, **kw)

    def op(self):
        return self.msa.Op.DENSE_ATTN_PREFILL if self.bits is None else self.msa.Op.TREE_ATTN

    def want(self):
        return reference(self.q_lens, self.kv_lens, self.rows, self.q, self.k, self.v, self.ks, self.vs, self.scale,
                         self.visible)

    def check(self):
        ws = self.msa.workspace(self.prob, self.op())
        got = self.run(ws=ws)
        assert self.msa.msa_read_device_status(ws) == 0
        check(got, self.want(), f"{self.layout} {self.q_lens} {self.kv_lens}")
        return got


LAYOUTS = ("packed", "paged", "fp8")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n", [1, 2, 16, 17, 127, 128, 129, 257, 640])
def test_one_prompt(msa, layout, n):
    Batch(msa, [n], [n], 16, 1, layout, seed=n).check()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("hq,hkv", [(4, 4), (3, 1), (10, 2), (14, 2), (16, 2), (33, 1), (64, 1), (96, 2), (128, 1), (127, 1)])
def test_groups(msa, layout, hq, hkv):
    Batch(msa, [150, 0, 33, 1], [150, 0, 300, 129], hq, hkv, layout, seed=hq).check()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_ragged_batch(msa, layout):
    q = [5, 0, 130, 1, 64, 0, 255, 17]
    kv = [5, 300, 130, 1000, 65, 0, 700, 2000]
    Batch(msa, q, kv, 16, 2, layout, seed=5).check()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("q,kv,hq,hkv", [([3], [20000], 16, 1), ([1, 2], [9000, 2], 16, 4), ([40, 7], [5000, 12345], 32, 2),
                                         ([300], [6000], 8, 1), ([9, 9, 9], [4097, 128, 30000], 5, 1)])
def test_few_tokens_over_long_caches(msa, layout, q, kv, hq, hkv):
    """Calls that are cut into runs."""
    Batch(msa, q, kv, hq, hkv, layout, seed=7).check()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_many_sequences(msa, layout):
    gen = torch.Generator().manual_seed(3)
    q = torch.randint(0, 4, (1500,), generator=gen).tolist()
    kv = [a + int(b) for a, b in zip(q, torch.randint(0, 40, (1500,), generator=gen))]
    Batch(msa, q, kv, 8, 1, layout, seed=3).check()


@pytest.mark.parametrize("layout", ("paged", "fp8"))
@pytest.mark.parametrize("q,kv,hq,hkv", [([1], [1], 16, 1), ([8], [8], 16, 1), ([8], [700], 64, 4), ([64], [200], 16, 2),
                                         ([70], [300], 8, 1), ([5, 0, 33, 3], [2000, 40, 160, 3], 12, 4),
                                         ([31, 16], [20000, 129], 16, 2), ([200], [1000], 3, 1)])
def test_trees(msa, layout, q, kv, hq, hkv):
    Batch(msa, q, kv, hq, hkv, layout, seed=11, tree=True).check()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("gain", [40.0, 3000.0, 1e6])
def test_rising_and_large_logits(msa, layout, gain):
    """Keys that grow along the sequence: the reference rises block after block; large logits."""
    b = Batch(msa, [200, 3], [900, 5000], 16, 2, layout, seed=13, q_gain=gain)
    if layout == "packed":
        b.k *= torch.linspace(0.1, 4.0, b.k.shape[0], device="cuda").to(torch.bfloat16)[:, None, None]
    b.check()


def test_pages_of_very_different_scales(msa):
    """Pages of zeros (scale 1), of tiny and of large values side by side."""
    for tree in (False, True):
        b = Batch(msa, [40, 3], [900, 5000], 16, 2, "fp8", seed=31, tree=tree)
        gen = torch.Generator(device="cuda").manual_seed(1)
        f = 2.0 ** torch.randint(-30, 12, b.vs.shape, generator=gen, device="cuda").float()
        b.vs *= f
        b.ks *= 2.0 ** torch.randint(-6, 2, b.ks.shape, generator=gen, device="cuda").float()
        zero = b.rows[0][128:256].cuda()
        b.v[zero] = 0
        b.vs[zero[0] // PAGE] = 1.0
        b.check()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rows_apart(msa, layout):
    """What one query row holds (large values, inf, NaN) does not change another's bits; nor does a sequence's V."""
    b = Batch(msa, [70, 9], [400, 3000], 16, 2, layout, seed=37)
    o, lse = b.run()
    b.q[5, 3] = 1e4
    b.q[60, 0, 7] = math.inf
    b.q[72, 9, 1] = math.nan
    o2, lse2 = b.run()
    same = torch.ones(79, 16, dtype=torch.bool, device="cuda")
    same[5, 3] = same[60, 0] = same[72, 9] = False
    assert torch.equal(o[same], o2[same]) and torch.equal(lse[same], lse2[same])
    assert torch.isnan(o2[72, 9]).all() and torch.isnan(lse2[72, 9])
    last = b.rows[1][-1].item()   # the last key of the second sequence: no query of the first meets it
    b.v[last] = 0x7F if layout == "fp8" else math.nan
    o3, _ = b.run()
    same[70:] = False
    assert torch.equal(o[same], o3[same])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_hidden_keys(msa, layout):
    """K of keys that a query does not see: NaN and inf there change nothing."""
    n = 300
    b = Batch(msa, [n], [n], 16, 1, layout, seed=41)
    o, lse = b.run()
    late = b.rows[0][200:].cuda()
    b.k[late] = 0x7F if layout == "fp8" else math.inf
    o2, lse2 = b.run()
    assert torch.equal(o[:200], o2[:200]) and torch.equal(lse[:200], lse2[:200])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_softmax_scale(msa, layout):
    Batch(msa, [60], [400], 16, 1, layout, seed=17, scale=0.5).check()


def test_no_queries(msa):
    b = Batch(msa, [0, 0], [100, 0], 16, 2, "packed")
    ws = msa.workspace(b.prob, b.op())
    o, lse = b.run(ws=ws)
    assert o.shape == (0, 16, DIM) and lse.shape == (0, 16)
    assert msa.msa_read_device_status(ws) == 0


@pytest.mark.parametrize("q,kv", [([300, 40], [300, 1040]), ([4], [30000])])
def test_same_bits(msa, q, kv):
    b = Batch(msa, q, kv, 16, 2, "paged", seed=19)
    a = b.run()
    for _ in range(3):
        c = b.run()
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("seqs", [5, 1024, 2050])
def test_a_workspace_may_hold_anything(msa, layout, seqs):
    """What a workspace holds before a call does not matter: many sequences' lists are built in it."""
    q = [1 + s % 3 for s in range(seqs)]
    b = Batch(msa, q, [n + 7 * (s % 41) for s, n in enumerate(q)], 4, 2, layout, seed=47)
    want = b.run()
    ws = torch.empty_like(msa.workspace(b.prob, b.op()))
    for fill in (0xFF, 0x7F, 0x01):
        ws.fill_(fill)
        o, lse = b.run(ws=ws)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert msa.msa_read_device_status(ws) == 0


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("many", [40, 1100])
def test_long_caches_among_short_prompts(msa, layout, many):
    """Runs over items of very different cost: ends of two tiles and of one, items of a block, two long ones."""
    q = [1 + 7 * (s % 23) for s in range(many)] + [3, 40]
    kv = [n + (s % 5) * 90 for s, n in enumerate(q[:-2])] + [9000, 20000]
    Batch(msa, q, kv, 16, 2, layout, seed=53).check()


def test_packed_and_paged_agree(msa):
    """The same keys by either way: the same bits."""
    p = Batch(msa, [100, 3], [500, 9000], 16, 2, "paged", seed=23)
    rows = torch.cat(p.rows).cuda()
    o, lse = msa.msa_dense_attn_prefill(p.prob, p.q, p.k[rows].contiguous(), p.v[rows].contiguous())
    o2, lse2 = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_lengths_that_contradict_the_sizes(msa):
    b = Batch(msa, [10, 20], [100, 200], 16, 2, "packed")
    ws = msa.workspace(b.prob, b.op())
    o, lse = torch.full_like(b.q, 3), torch.full((30, 16), 3.0, device="cuda")
    for cu_q, cu_k in (([0, 10, 31], None), ([0, 12, 11], None), (None, [0, 5, 300]), ([1, 10, 30], None),
                       (None, [0, 100, 299])):
        if cu_q:
            b.prob.cu_q = torch.tensor(cu_q, dtype=torch.int32, device="cuda")
        if cu_k:
            b.prob.cu_k = torch.tensor(cu_k, dtype=torch.int32, device="cuda")
        b.run(o=o, lse=lse, ws=ws)
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_SEQLENS
        assert (o == 3).all() and (lse == 3).all()
        b.prob.cu_q = torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda")
        b.prob.cu_k = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    check(b.run(o=o, lse=lse, ws=ws), b.want())
    assert msa.msa_read_device_status(ws) == 0


@pytest.mark.parametrize("layout", ("paged", "fp8"))
def test_pages_outside_the_cache(msa, layout):
    """Such a page reads as zeros and raises the flag."""
    b = Batch(msa, [20], [600], 16, 1, layout, seed=29)
    ws = msa.workspace(b.prob, b.op())
    for bad in (-1, b.k.shape[0] // PAGE, 2 ** 31 - 1, -2 ** 31):
        table = b.table.clone()
        table[0, 2] = bad
        o, lse = b.run(ws=ws) if bad is None else (
            msa.msa_dense_attn_prefill_paged(b.prob, b.q, b.k, b.v, table, ws=ws) if layout == "paged" else
            msa.msa_dense_attn_prefill_paged_fp8(b.prob, b.q, b.k, b.v, b.ks, b.vs, table, ws=ws))
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX
        k, v = b.k.clone(), b.v.clone()
        k[b.rows[0][256:384].cuda()] = 0
        v[b.rows[0][256:384].cuda()] = 0
        want = reference(b.q_lens, b.kv_lens, b.rows, b.q, k, v, b.ks, b.vs, 0.0, None)
        check((o, lse), want)
