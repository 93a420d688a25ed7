"""GPU: msa_evict_paged(_fp8) against its rule written out on the host: kept slots, rows, weights and lengths are exact."""
import math

import pytest
import torch

from paged_reference import DIM, PAGE, blocks, evict_reference, make_tables, quantize_pages, rows_of

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


def _codes(x):
    """E4M3 codes of 64-bit values within +-448, rounded to nearest even once (a conversion by way of fp32 rounds
    twice and can miss a midpoint): 4 significant bits, the smallest step 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).float().to(torch.float8_e4m3fn).view(torch.uint8)


class Cache:
    def __init__(self, msa, lens, hkv, budget, recent, fp8=False, seed=0, stride=None):
        host = torch.Generator().manual_seed(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hkv, self.budget, self.recent, self.fp8 = lens, hkv, budget, recent, fp8
        both, pages = make_tables(list(lens) + [min(n, budget) for n in lens], host)
        S = len(lens)
        self.host_table, self.host_new = both[:S].contiguous(), both[S:].contiguous()
        self.table, self.new = self.host_table.cuda(), self.host_new.cuda()
        rnd = lambda: torch.randn(pages * PAGE, hkv, DIM, device="cuda", generator=gen).to(torch.bfloat16)
        self.k, self.v, self.ks, self.vs = rnd(), rnd(), None, None
        if fp8:
            self.k, self.ks = quantize_pages(self.k)
            self.v, self.vs = quantize_pages(self.v)
        self.weight = torch.randn(S, hkv, stride or max(1, max(lens)), device="cuda", generator=gen).exp()
        self.prob = msa.problem_from_seqlens([1] * S, lens, hkv * 4, hkv, 128, 16)

    def call(self, msa, **kw):
        if self.fp8:
            return msa.msa_evict_paged_fp8(self.prob, self.k, self.v, self.ks, self.vs, self.table, self.weight,
                                           self.new, self.budget, self.recent, **kw)
        return msa.msa_evict_paged(self.prob, self.k, self.v, self.table, self.weight, self.new, self.budget,
                                   self.recent, **kw)

    def ws(self, msa):
        return msa.evict_workspace(self.prob, self.budget, self.k.shape[0] // PAGE)

    def expected(self):
        """Caches (and scales), kept, new weights and lengths after the call, from the rule."""
        k, v = self.k.clone(), self.v.clone()
        ks, vs = (self.ks.clone(), self.vs.clone()) if self.fp8 else (None, None)
        slots = evict_reference(self.lens, self.weight, self.budget, self.recent)
        S = len(self.lens)
        kept = torch.full((S, self.hkv, self.budget), -1, dtype=torch.int32)
        cu = [0]
        weights = []
        for s, n in enumerate(self.lens):
            m = min(n, self.budget)
            cu.append(cu[-1] + m)
            weights.append([])
            if m == 0:
                continue
            src, dst = rows_of(self.host_table, s, n), rows_of(self.host_new, s, m)
            for g in range(self.hkv):
                at = torch.tensor(slots[s][g])
                assert len(at) == m
                kept[s, g, :m] = at.to(torch.int32)
                weights[-1].append(self.weight[s, g, at.cuda()])
                fr, to = src[at].cuda(), dst.cuda()
                if not self.fp8:
                    k[to, g], v[to, g] = self.k[fr, g], self.v[fr, g]
                    continue
                for new, old, sc, osc in ((k, self.k, ks, self.ks), (v, self.v, vs, self.vs)):
                    val = old[fr, g].view(torch.float8_e4m3fn).double() * osc[fr // PAGE, g].double()[:, None]
                    for b in range(blocks(m)):
                        part = val[b * PAGE:(b + 1) * PAGE]
                        top = part.abs().amax()
                        rows = to[b * PAGE:(b + 1) * PAGE]
                        new[rows, g] = _codes(part * 448 / top if top > 0 else part)
                        # a division of two tensors: by a number torch multiplies by its rounded inverse
                        sc[rows[0] // PAGE, g] = (top / torch.full_like(top, 448)).float() if top > 0 else 1.0
        return k, v, ks, vs, kept.cuda(), weights, torch.tensor(cu, dtype=torch.int32, device="cuda")

    def check(self, msa):
        k, v, ks, vs, kept, weights, cu = self.expected()
        ws = self.ws(msa)
        ws.fill_(0xFF)
        S = len(self.lens)
        nw = torch.full((S, self.hkv, self.budget + 3), -5.0, device="cuda")
        got_kept, got_w, got_cu = self.call(msa, new_weight=nw, ws=ws)
        assert msa.msa_read_device_status(ws) == 0
        assert torch.equal(got_cu, cu) and torch.equal(got_kept, kept)
        same = lambda a, b: torch.equal(a.view(torch.int32 if a.element_size() == 4 else torch.int16 if
                                               a.element_size() == 2 else torch.uint8),
                                        b.view(torch.int32 if b.element_size() == 4 else torch.int16 if
                                               b.element_size() == 2 else torch.uint8))
        for s, n in enumerate(self.lens):
            m = min(n, self.budget)
            for g in range(self.hkv):
                if m:
                    assert same(got_w[s, g, :m].contiguous(), weights[s][g])
                assert (got_w[s, g, m:] == -5).all()
        assert same(self.k, k) and same(self.v, v)  # the pool as a whole: what is not a new slot is as it was
        if self.fp8:
            assert same(self.ks, ks) and same(self.vs, vs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,budget,recent", [
    ([1], 1, 0), ([1], 1, 1), ([2], 1, 0), ([2], 1, 1), ([5], 3, 1), ([129], 128, 5), ([129], 128, 128), ([300], 129, 0),
    ([128], 128, 7), ([1000], 999, 0), ([700, 0, 3, 512, 513], 512, 64), ([0, 0], 4, 2), ([4095, 4096, 4097, 9000], 2000, 100),
    ([5000], 4999, 1), ([5000], 1, 0), ([300] * 90, 100, 10), ([20, 30], 1000, 1000), ([20000, 40], 130, 2)])
def test_lengths_and_budgets(msa, lens, budget, recent, fp8):
    Cache(msa, lens, 2, budget, recent, fp8, seed=len(lens) + budget).check(msa)


@pytest.mark.parametrize("hkv", [1, 3, 4, 8, 9, 20])
@pytest.mark.parametrize("fp8", [False, True])
def test_heads(msa, hkv, fp8):
    Cache(msa, [900, 100, 400], hkv, 300, 20, fp8, seed=hkv, stride=903).check(msa)


def test_long(msa):
    Cache(msa, [70000, 10], 2, 30001, 1000, seed=2).check(msa)


@pytest.mark.parametrize("kind", ["equal", "two_values", "zeros", "signs", "nan_inf", "close", "ascending", "descending"])
def test_weights_that_tie_or_are_no_numbers(msa, kind):
    c = Cache(msa, [3000, 130, 0, 5001], 2, 1000, 30, seed=3)
    w = c.weight
    i = torch.arange(w.shape[2], device="cuda")
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "two_values":
        w.copy_(((i * 7) % 3 == 0).float())
    elif kind == "zeros":
        w.copy_(torch.where(i % 2 == 0, 0.0, -0.0))
    elif kind == "signs":
        w.normal_()
    elif kind == "nan_inf":
        w.masked_fill_(i % 3 == 0, math.nan)
        w.masked_fill_(i % 5 == 0, -math.inf)
        w.masked_fill_(i % 11 == 0, math.inf)
    elif kind == "close":
        w.copy_((0x3F800000 + (i * 2654435761) % 4).to(torch.int32).view(torch.float32))
    elif kind == "ascending":
        w.copy_(i.float())
    else:
        w.copy_(-i.float())
    c.check(msa)


@pytest.mark.parametrize("kind", ["equal", "two_values", "few_values", "tail", "window_only", "uncached"])
@pytest.mark.parametrize("lens,hkv", [([70001], 1), ([40000, 36001, 0, 8192, 32768], 2), ([17000] * 13, 2), ([33000] * 77, 1)])
def test_ties_across_the_parts_of_a_long_row(msa, lens, hkv, kind):
    """Rows that are shared out over eight, four, two and one parts: equal weights begin and end in any of them."""
    if kind == "uncached" and len(lens) > 5:
        pytest.skip("the same as for shorter rows")
    if kind == "uncached":
        lens = [n * 6 for n in lens]  # shares past what a part keeps in shared memory
    budget, recent = max(lens) // 2 + 3, 0 if kind == "window_only" else 1001
    if kind == "window_only":
        budget = recent = 9000
    c = Cache(msa, lens, hkv, budget, recent, seed=5)
    w, i = c.weight, torch.arange(c.weight.shape[2], device="cuda")
    if kind in ("equal", "uncached"):
        w.fill_(0.25)
        if kind == "uncached":
            w[..., 5::7] = 0.5
    elif kind == "two_values":
        w.copy_(((i * 7) % 3 == 0).float())
    elif kind == "few_values":
        w.copy_((0x3F800000 + (i * 2654435761) % 4).to(torch.int32).view(torch.float32))
    elif kind == "tail":  # the threshold's ties all in the last parts
        w.copy_((i >= max(lens) * 3 // 4).float() - (i < 100).float())
    c.check(msa)


def test_shared_source_pages(msa):
    """A prefix that two sequences share stays as it is; each gets its own copy of what it keeps."""
    c = Cache(msa, [600, 700], 2, 200, 10, seed=4)
    c.host_table[1, :3] = c.host_table[0, :3]
    c.table = c.host_table.cuda()
    c.check(msa)


@pytest.mark.parametrize("fp8", [False, True])
def test_new_pages_that_may_not_be_written(msa, fp8):
    """A new page that is a page of the batch, is named twice or lies outside the cache is left alone and reported;
    the others are written."""
    for kind in ("own", "other", "twice", "outside", "negative"):
        c = Cache(msa, [600, 700], 2, 300, 10, fp8, seed=5)
        k, v, ks, vs, kept, _, cu = c.expected()
        bad = [(0, 1)]
        if kind == "own":
            c.host_new[0, 1] = c.host_table[0, 4]
        elif kind == "other":
            c.host_new[0, 1] = c.host_table[1, 0]
        elif kind == "twice":
            c.host_new[0, 1] = c.host_new[1, 2]
            bad.append((1, 2))
        else:
            c.host_new[0, 1] = c.k.shape[0] // PAGE if kind == "outside" else -1
        good = Cache(msa, [600, 700], 2, 300, 10, fp8, seed=5)
        for s, b in bad:  # those pages keep what they held
            p = int(good.host_new[s, b])
            k[p * PAGE:(p + 1) * PAGE], v[p * PAGE:(p + 1) * PAGE] = c.k[p * PAGE:(p + 1) * PAGE], c.v[p * PAGE:(p + 1) * PAGE]
            if fp8:
                ks[p], vs[p] = c.ks[p], c.vs[p]
        c.new = c.host_new.cuda()
        ws = c.ws(msa)
        got, _, got_cu = c.call(msa, ws=ws)
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX, kind
        assert torch.equal(got, kept) and torch.equal(got_cu, cu)
        view = torch.uint8 if fp8 else torch.int16
        assert torch.equal(c.k.view(view), k.view(view)) and torch.equal(c.v.view(view), v.view(view)), kind
        if fp8:
            assert torch.equal(c.ks, ks) and torch.equal(c.vs, vs)


def test_a_source_page_outside_the_cache_reads_as_zeros(msa):
    c = Cache(msa, [600], 2, 300, 10, seed=6)
    c.host_table[0, 4] = 10 ** 6  # holds the window
    c.table = c.host_table.cuda()
    ws = c.ws(msa)
    kept, _, _ = c.call(msa, ws=ws)
    assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX
    rows = rows_of(c.host_new, 0, 300).cuda()
    gone = (kept[0] >= 512).T  # [300, heads]
    assert (c.k[rows][gone] == 0).all() and (c.v[rows][gone] == 0).all() and (c.k[rows][~gone] != 0).any(-1).all()


def test_lengths_that_contradict_the_sizes_skip_the_call(msa):
    c = Cache(msa, [600, 700], 2, 300, 10, seed=7)
    k = c.k.clone()
    for cu in ([0, 600, 1299], [0, 700, 1301], [0, 800, 1300], [0, -5, 1300]):
        c.prob.cu_k.copy_(torch.tensor(cu, dtype=torch.int32))
        ws = c.ws(msa)
        kept = torch.full((2, 2, 300), 9, dtype=torch.int32, device="cuda")
        new_cu = torch.full((3,), 9, dtype=torch.int32, device="cuda")
        nw = torch.full((2, 2, 300), 9.0, device="cuda")
        c.call(msa, kept=kept, new_cu_k=new_cu, new_weight=nw, ws=ws)
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_SEQLENS
        assert (kept == 9).all() and (new_cu == 9).all() and (nw == 9).all() and torch.equal(c.k, k)


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_and_stream(msa, fp8):
    c = Cache(msa, [3000, 600, 10], 4, 500, 50, fp8, seed=8)
    ws = c.ws(msa)
    outs = dict(kept=torch.empty(3, 4, 500, dtype=torch.int32, device="cuda"),
                new_weight=torch.zeros(3, 4, 500, device="cuda"),
                new_cu_k=torch.empty(4, dtype=torch.int32, device="cuda"))
    c.call(msa, ws=ws, **outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(msa, ws=ws, **outs)
    for rep in range(2):
        c.weight.normal_().exp_()
        k, v, _, _, kept, _, cu = c.expected()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs["kept"], kept) and torch.equal(outs["new_cu_k"], cu)
        view = torch.uint8 if fp8 else torch.int16
        assert torch.equal(c.k.view(view), k.view(view)) and torch.equal(c.v.view(view), v.view(view))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.check(msa)


def test_far_pages(msa):
    """Rows whose byte offsets pass 2^32 on both sides."""
    pages, hkv, lens, budget = 40000, 4, [300], 140
    k = torch.empty(pages * PAGE, hkv, DIM, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    src, dst = [39999, 33001, 7], [39998, 34000]
    for p in src:
        k[p * PAGE:(p + 1) * PAGE].normal_()
        v[p * PAGE:(p + 1) * PAGE].normal_()
    weight = torch.rand(1, hkv, 300, device="cuda")
    prob = msa.problem_from_seqlens([1], lens, 16, hkv, 128, 16)
    t = lambda x: torch.tensor([x], dtype=torch.int32)
    kept, _, _ = msa.msa_evict_paged(prob, k, v, t(src).cuda(), weight, t(dst).cuda(), budget, 9)
    slots = evict_reference(lens, weight, budget, 9)
    s, d = rows_of(t(src), 0, 300), rows_of(t(dst), 0, budget).cuda()
    for g in range(hkv):
        assert kept[0, g].tolist() == slots[0][g]
        fr = s[torch.tensor(slots[0][g])].cuda()
        assert torch.equal(k[d, g], k[fr, g]) and torch.equal(v[d, g], v[fr, g])
