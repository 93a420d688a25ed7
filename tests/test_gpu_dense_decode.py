"""GPU: msa_dense_attn_decode_paged(_fp8) against a 64-bit reference, with its bounds (paged_reference)."""
import math

import pytest
import torch

from paged_reference import DIM, PAGE, blocks, dense_reference, make_tables, quantize_pages, rows_of

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


class Batch:
    """A decode batch over paged caches whose unused rows hold NaN (bf16) or random codes (fp8)."""

    def __init__(self, msa, lens, hq, hkv, fp8=False, weight=False, seed=0, scale=0.0, q_gain=2.0, spare=3):
        host = torch.Generator().manual_seed(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.fp8, self.scale = lens, fp8, scale
        self.host_table, pages = make_tables(lens, host, spare)
        self.table = self.host_table.cuda()
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16)
        self.q = rnd(len(lens), hq, DIM) * q_gain
        self.k, self.v = rnd(pages * PAGE, hkv, DIM), rnd(pages * PAGE, hkv, DIM)
        self.ks = self.vs = None
        if fp8:
            self.k, self.ks = quantize_pages(self.k)
            self.v, self.vs = quantize_pages(self.v)
        used = torch.zeros(pages * PAGE, dtype=torch.bool)
        for s, n in enumerate(lens):
            if n:
                used[rows_of(self.host_table, s, n)] = True
        unused = (~used).cuda()
        # rows behind a sequence and pages of nobody hold NaN (0x7F is E4M3's NaN)
        self.k[unused] = 0x7F if fp8 else math.nan
        self.v[unused] = 0x7F if fp8 else math.nan
        self.prob = msa.problem_from_seqlens([1] * len(lens), lens, hq, hkv, 128, 16, scale=scale)
        self.weight = None
        if weight:
            self.weight = torch.rand(len(lens), hkv, max(lens) + 7, device="cuda", generator=gen)

    def call(self, msa, **kw):
        kw.setdefault("weight", self.weight)
        if self.fp8:
            return msa.msa_dense_attn_decode_paged_fp8(self.prob, self.q, self.k, self.v, self.ks, self.vs, self.table,
                                                       **kw)
        return msa.msa_dense_attn_decode_paged(self.prob, self.q, self.k, self.v, self.table, **kw)

    def ws(self, msa):
        return msa.workspace(self.prob, msa.Op.DENSE_ATTN_DECODE_WEIGHT if self.weight is not None
                             else msa.Op.DENSE_ATTN_DECODE)

    def check(self, msa):
        before = None if self.weight is None else self.weight.clone()
        ws = self.ws(msa)
        ws.fill_(0xFF)  # a workspace may hold anything
        o, lse = self.call(msa, ws=ws)
        assert msa.msa_read_device_status(ws) == 0
        ref_o, ref_lse, ref_w, o_tol, lse_tol, w_tol = dense_reference(self.lens, self.table, self.q, self.k, self.v,
                                                                       self.ks, self.vs, self.scale)
        bad = (o.double() - ref_o).abs() > o_tol
        assert torch.isfinite(o).all() and not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
        empty = torch.tensor([n == 0 for n in self.lens], device="cuda")
        assert (lse[empty] == -math.inf).all() and (o[empty] == 0).all()
        off = (lse.double() - ref_lse).abs()[~empty]
        assert (off <= lse_tol[~empty]).all(), float(off.max())
        if before is None:
            return
        for s, n in enumerate(self.lens):
            got, want = self.weight[s, :, :n].double(), before[s, :, :n].double() + ref_w[s]
            tol = w_tol[s] + 2.0 ** -24 * want.abs()
            assert ((got - want).abs() <= tol).all(), (s, float((got - want).abs().max()))
            assert torch.equal(self.weight[s, :, n:], before[s, :, n:]), "entries past the length changed"


LENS = {
    "one": [1], "two": [2], "15": [15], "16": [16], "17": [17], "63": [63], "64": [64], "65": [65], "127": [127],
    "128": [128], "129": [129], "1000": [1000],
    "ragged": [0, 1, 300, 0, 64, 129, 2000, 0],
    "trailing_empty": [500, 0, 0, 0],
    "all_empty": [0, 0, 0],
    "long_and_short": [30000] + [1] * 40 + [0] * 5 + [77] * 3,
    "many_short": [(i * 37) % 200 for i in range(700)],
}


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", list(LENS))
def test_lengths(msa, lens, fp8, weight):
    Batch(msa, LENS[lens], 32, 2, fp8, weight, seed=len(lens)).check(msa)


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (5, 1), (8, 1), (16, 1), (17, 1), (32, 1), (33, 1), (64, 1), (65, 1),
                                    (127, 1), (128, 1), (12, 12), (40, 8), (64, 4), (96, 2), (48, 3), (160, 160),
                                    (400, 400), (35, 7)])
def test_head_layouts(msa, hq, hkv, fp8, weight):
    lens = [700, 1, 0, 333] if hkv < 100 else [130, 1]
    Batch(msa, lens, hq, hkv, fp8, weight, seed=hq).check(msa)


@pytest.mark.parametrize("hq,hkv", [(64, 4), (128, 1), (24, 1), (56, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_long(msa, hq, hkv, fp8):
    Batch(msa, [60001, 17, 9000], hq, hkv, fp8, True, seed=3).check(msa)


@pytest.mark.parametrize("lens,hq,hkv", [
    ([(i * 97) % 800 for i in range(700)], 10, 2),      # many sequences, several to a run
    ([1, 200000, 0, 70000, 3], 16, 1),                  # long ones, cut into many runs
    ([(i * 13) % 61 for i in range(5000)], 3, 1),       # more sequences than a warp looks through
    ([90000] + [(i * 31) % 50 for i in range(4500)], 6, 3),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_large_batches(msa, lens, hq, hkv, fp8):
    Batch(msa, lens, hq, hkv, fp8, True, seed=len(lens)).check(msa)


@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_and_flat_logits(msa, fp8):
    Batch(msa, [3000, 129], 16, 1, fp8, True, seed=4, q_gain=60.0).check(msa)     # one key takes nearly all
    Batch(msa, [3000, 129], 16, 1, fp8, True, seed=5, scale=1e-4).check(msa)      # uniform weights
    Batch(msa, [3000, 129], 16, 1, fp8, True, seed=6, scale=0.5, q_gain=0.01).check(msa)


def test_rising_and_falling_logits(msa):
    """The running maximum moves at every tile, or never after the first."""
    for sign in (1.0, -1.0):
        b = Batch(msa, [2000], 16, 2, False, True, seed=7)
        rows = rows_of(b.host_table, 0, 2000).cuda()
        ramp = torch.linspace(-3, 3, 2000, device="cuda") * sign
        b.k[rows] = (b.q[0, ::8][None].float() / 8 * ramp[:, None, None]).to(torch.bfloat16)
        b.check(msa)


@pytest.mark.parametrize("hq", [16, 32, 64, 128])
def test_first_keys_without_weight(msa, hq):
    """The first 300 keys' logits are -inf, the others' far below 0; in the second sequence no key counts."""
    b = Batch(msa, [700, 200, 290], hq, 1, seed=11)
    b.q[:, :, 0] = 16.0
    for s, n in ((0, 300), (1, 200), (2, 10)):
        rows = rows_of(b.host_table, s, b.lens[s]).cuda()
        b.k[rows, :, 0] = -200.0
        b.k[rows[:n], :, 0] = -math.inf
    o, lse = b.call(msa)
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    k = b.k.clone()
    k[k == -math.inf] = -1e5  # weight exp(-140000): 0 in 64 bits too, and bounds without infinities
    ref_o, ref_lse, _, o_tol, lse_tol, _ = dense_reference(b.lens, b.table, b.q, k, b.v)
    for s in (0, 2):
        assert ((o[s].double() - ref_o[s]).abs() <= o_tol[s]).all()
        # the bound on the largest logit is that of the keys that count
        assert ((lse[s].double() - ref_lse[s]).abs() <= 2.0 ** -23 * (130 * 0.09 * (16 * 200 + 3000) + 720 + 8 * 300)).all()


def test_fp8_scales_of_any_size(msa):
    """Pages whose K and V scales differ by many orders of magnitude."""
    b = Batch(msa, [1500, 400], 32, 2, True, True, seed=8)
    n = b.vs.shape[0]
    b.vs *= (2.0 ** torch.linspace(-60, 40, n, device="cuda"))[torch.randperm(n, device="cuda")][:, None]
    b.ks *= (2.0 ** torch.linspace(-12, 0, n, device="cuda"))[:, None]
    b.q *= torch.tensor([2.0 ** -30, 2.0 ** 8], device="cuda").to(torch.bfloat16).view(2, 1, 1)
    b.check(msa)


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("hq", [40, 64, 128])
def test_fp8_scales_of_any_size_large_groups(msa, hq, order):
    """The same where O's exponent moves at every page, never after the first, or now and then."""
    b = Batch(msa, [2900, 130, 1], hq, 1, True, True, seed=10)
    n = b.vs.shape[0]
    grow = 2.0 ** torch.linspace(-60, 40, n, device="cuda")
    at = torch.randperm(n, device="cuda")
    if order != "mixed":
        pages = b.host_table[0, :23].cuda().long()
        rest = torch.tensor([p for p in range(n) if p not in set(pages.tolist())], device="cuda")
        at[torch.cat([pages, rest])] = torch.arange(n, device="cuda")
        if order == "down":
            at = n - 1 - at
    b.vs *= grow[at][:, None]
    b.ks *= (2.0 ** torch.linspace(-12, 0, n, device="cuda"))[:, None]
    b.q *= torch.tensor([2.0 ** -30, 2.0 ** 8, 1.0], device="cuda").to(torch.bfloat16).view(3, 1, 1)
    b.check(msa)


def test_zero_pages_and_queries_fp8(msa):
    b = Batch(msa, [300], 16, 1, True, False, seed=9)
    b.k[rows_of(b.host_table, 0, 128).cuda()] = 0
    b.v[rows_of(b.host_table, 0, 300).cuda()] = 0
    b.q[0, 3] = 0
    b.check(msa)


def test_shared_pages(msa):
    """Two sequences with a common prefix."""
    b = Batch(msa, [400, 500], 16, 2, False, True, seed=10)
    b.host_table[1, :2] = b.host_table[0, :2]
    b.table = b.host_table.cuda()
    b.check(msa)


def test_far_pages(msa):
    """Rows whose byte offsets pass 2^32 (and element offsets 2^31)."""
    pages, hkv = 40000, 4
    k = torch.empty(pages * PAGE, hkv, DIM, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    lens = [200, 129]
    table = torch.tensor([[39999, 1], [33000, 25001]], dtype=torch.int32)
    for p in (39999, 1, 33000, 25001):
        k[p * PAGE:(p + 1) * PAGE].normal_()
        v[p * PAGE:(p + 1) * PAGE].normal_()
    q = torch.randn(2, 64, DIM, device="cuda").to(torch.bfloat16)
    prob = msa.problem_from_seqlens([1, 1], lens, 64, hkv, 128, 16)
    weight = torch.zeros(2, hkv, 200, device="cuda")
    o, lse = msa.msa_dense_attn_decode_paged(prob, q, k, v, table.cuda(), weight=weight)
    ref = dense_reference(lens, table, q, k, v)
    assert ((o.double() - ref[0]).abs() <= ref[3]).all() and ((lse.double() - ref[1]).abs() <= ref[4]).all()
    assert ((weight[0, :, :200].double() - ref[2][0]).abs() <= ref[5][0] + U_W).all()


U_W = 2.0 ** -23


@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_are_bit_equal(msa, fp8):
    b = Batch(msa, [5000, 0, 131, 9], 64, 4, fp8, True, seed=11)
    start = b.weight.clone()
    o, lse = b.call(msa)
    first = b.weight.clone()
    for _ in range(3):
        b.weight.copy_(start)
        o2, lse2 = b.call(msa)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(first, b.weight)


@pytest.mark.parametrize("hq,hkv", [(64, 4), (32, 1), (64, 1), (128, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_many_calls_in_a_row(msa, hq, hkv, fp8):
    """Calls that follow one another without a pause, over caches larger than L2: every one gives the first one's bits."""
    b = Batch(msa, [1 + (i * 5021) % 16384 for i in range(32)], hq, hkv, fp8, True, seed=16)
    start, ws = b.weight.clone(), b.ws(msa)
    o, lse = b.call(msa, ws=ws)
    first = b.weight.clone()
    for _ in range(5):
        b.weight.copy_(start)
        outs = [b.call(msa, ws=ws)]
        once = b.weight.clone()
        outs += [b.call(msa, ws=ws) for _ in range(6)]
        assert torch.equal(once, first) and msa.msa_read_device_status(ws) == 0
        for o2, lse2 in outs:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_outputs_given_by_the_caller_and_another_stream(msa):
    b = Batch(msa, [777, 12], 64, 4, False, False, seed=12)
    o, lse = b.call(msa)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        mine = torch.empty_like(b.q), torch.empty(2, 64, dtype=torch.float32, device="cuda")
        got = b.call(msa, o=mine[0], lse=mine[1], ws=b.ws(msa))
    side.synchronize()
    assert got[0] is mine[0] and torch.equal(o, mine[0]) and torch.equal(lse, mine[1])


def test_two_streams_at_once(msa):
    """Calls in flight on two streams, each with its own workspace, give what they give alone."""
    batches = [Batch(msa, [9000, 700, 0, 4100], 128, 1, False, True, seed=21), Batch(msa, [12000, 77], 96, 2, True, seed=22),
               Batch(msa, [5000] * 6, 64, 4, False, True, seed=23), Batch(msa, [300] * 50, 40, 8, True, seed=24)]
    alone, spaces = [], []
    for b in batches:
        b.start = None if b.weight is None else b.weight.clone()
        o, lse = b.call(msa)
        alone.append((o, lse, None if b.weight is None else b.weight.clone()))
        spaces.append((b.ws(msa), torch.empty_like(o), torch.empty_like(lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(10):
        for i, (b, (ws, o, lse)) in enumerate(zip(batches, spaces)):
            with torch.cuda.stream(streams[i % 2]):
                if b.weight is not None:
                    b.weight.copy_(b.start)
                b.call(msa, ws=ws, o=o, lse=lse)
    torch.cuda.synchronize()
    for b, (ws, o, lse), (want_o, want_lse, want_w) in zip(batches, spaces, alone):
        assert msa.msa_read_device_status(ws) == 0
        assert torch.equal(o, want_o) and torch.equal(lse, want_lse)
        assert want_w is None or torch.equal(b.weight, want_w)


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_replays_follow_the_inputs(msa, fp8):
    b = Batch(msa, [3000, 500, 0], 64, 4, fp8, True, seed=13)
    ws = b.ws(msa)
    o, lse = torch.empty_like(b.q), torch.empty(3, 64, dtype=torch.float32, device="cuda")
    b.call(msa, o=o, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(msa, o=o, lse=lse, ws=ws)
    start = b.weight.clone()
    for rep in range(3):
        b.q.normal_()
        if rep == 2:  # a step later: the lengths grow within the captured bounds
            b.prob.cu_k.copy_(torch.tensor([0, 2900, 3400, 3500], dtype=torch.int32))
            b.host_table[2, 0] = b.host_table[1, 0]
            b.table.copy_(b.host_table)
        b.weight.copy_(start)
        g.replay()
        got = o.clone(), lse.clone(), b.weight.clone()
        b.weight.copy_(start)
        ref = b.call(msa)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and torch.equal(got[2], b.weight)


def test_graph_behind_copies_and_memsets(msa):
    """The call captured behind a memset and a copy of its own inputs, and behind itself."""
    b = Batch(msa, [2000, 129], 64, 4, False, True, seed=17)
    q, total = b.q.clone(), torch.empty_like(b.q)
    ws = b.ws(msa)
    o, lse = torch.empty_like(b.q), torch.empty(2, 64, dtype=torch.float32, device="cuda")
    gamma = torch.ones(DIM, dtype=torch.bfloat16, device="cuda")

    def step():
        b.weight.zero_()
        b.q.copy_(q)
        b.call(msa, o=o, lse=lse, ws=ws)
        b.call(msa, o=o, lse=lse, ws=ws)
        msa.msa_add_rms_norm(o, gamma, residual=b.q, sum_out=total, y=o)

    step()
    torch.cuda.synchronize()
    want = o.clone(), lse.clone(), b.weight.clone(), total.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (o, lse, b.weight, total):
            t.fill_(7)
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(want, (o, lse, b.weight, total)))


def test_lengths_that_contradict_the_sizes_skip_the_call(msa):
    b = Batch(msa, [300, 200], 16, 1, False, True, seed=14)
    good = b.prob.cu_k.clone()
    for cu in ([0, 300, 499], [1, 300, 500], [0, 400, 500], [0, -1, 500]):  # total, start, longest, negative
        b.prob.cu_k.copy_(torch.tensor(cu, dtype=torch.int32))
        ws = b.ws(msa)
        o, lse = torch.full_like(b.q, 7), torch.full((2, 16), 7.0, device="cuda")
        before = b.weight.clone()
        b.call(msa, o=o, lse=lse, ws=ws)
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_SEQLENS
        assert (o == 7).all() and (lse == 7).all() and torch.equal(b.weight, before)
    b.prob.cu_k.copy_(good)
    b.check(msa)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_page_outside_the_cache_reads_as_zeros(msa, fp8):
    b = Batch(msa, [300, 200], 16, 2, fp8, True, seed=15)
    pages = b.k.shape[0] // PAGE
    for entry in (pages, -1, 2 ** 31 - 1, -2 ** 31):
        table = b.host_table.clone()
        table[0, 1] = entry
        b.table = table.cuda()
        ws = b.ws(msa)
        o, lse = b.call(msa, ws=ws)
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX
        zero = b.k.shape[0] // PAGE  # the same batch with a page of zeros in that place
        pad = lambda x: torch.cat([x, torch.zeros_like(x[:PAGE])])
        table[0, 1] = zero
        ones = lambda x: None if x is None else torch.cat([x, torch.ones_like(x[:1])])
        ref = dense_reference(b.lens, table, b.q, pad(b.k), pad(b.v), ones(b.ks), ones(b.vs))
        assert ((o.double() - ref[0]).abs() <= ref[3]).all() and ((lse.double() - ref[1]).abs() <= ref[4]).all()
