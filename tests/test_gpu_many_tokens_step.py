"""The cache's life as a serving loop runs it: tables for the new tokens, their rows into the pages, the prompt in chunks,
a tree of drafts, the accepted tokens, decode steps; captured steps; calls on several streams at once.

Bounds as in test_gpu_prompt_attn (prompts and trees) and paged_reference (decode); E4M3 pages are judged against the values
that the pages hold.
"""
import pytest
import torch

from paged_reference import DIM, PAGE, blocks, dense_reference, rows_of
from test_gpu_prompt_attn import Batch, check, reference

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


def same_bits(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


class Loop:
    """A batch of sequences over one pool of pages, filled through the calls under test."""

    def __init__(self, msa, seqs, hq, hkv, fp8, pages=200, width=24, seed=0):
        self.msa, self.S, self.hq, self.hkv, self.fp8 = msa, seqs, hq, hkv, fp8
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        dtype = torch.uint8 if fp8 else torch.bfloat16
        self.k = torch.zeros(pages * PAGE, hkv, DIM, dtype=dtype, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.ks = torch.ones(pages, hkv, device="cuda") if fp8 else None
        self.vs = torch.ones(pages, hkv, device="cuda") if fp8 else None
        host = torch.Generator().manual_seed(seed)
        self.free = torch.randperm(pages, generator=host).to(torch.int32).cuda()
        self.taken = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        self.lens = [0] * seqs
        self.device_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    def rows(self, n):
        """New q, k, v of n tokens, slices of one projection's output."""
        x = torch.randn(n, (self.hq + 2 * self.hkv) * DIM, device="cuda", generator=self.gen).to(torch.bfloat16)
        q, k, v = x.split([self.hq * DIM, self.hkv * DIM, self.hkv * DIM], dim=1)
        return q.reshape(n, self.hq, DIM) * 2, k.view(n, self.hkv, DIM), v.view(n, self.hkv, DIM)

    def grow(self, new):
        """Tables and rows for `new` tokens a sequence; returns (problem, q)."""
        m, n = self.msa, sum(new)
        cu_q, cu_k, slots, positions, _ = m.msa_extend_block_table(
            self.device_lens, torch.tensor(new, dtype=torch.int32, device="cuda"), self.free, self.table, n,
            taken=self.taken, taken_out=self.taken, new_lengths=self.device_lens, num_pages=self.k.shape[0] // PAGE)
        before = self.lens
        self.lens = [a + b for a, b in zip(before, new)]
        assert positions.tolist() == [p for a, b in zip(before, new) for p in range(a, a + b)]
        q, k, v = self.rows(n)
        if self.fp8:
            m.msa_append_paged_fp8(k, v, slots, self.k, self.v, self.ks, self.vs)
        else:
            m.msa_append_paged(k, v, slots, self.k, self.v)
        return m.Problem(cu_q, cu_k, n, sum(self.lens), max(new), max(self.lens), self.hq, self.hkv, 128, 16), q

    def scales(self):
        return (self.ks, self.vs) if self.fp8 else ()

    def key_rows(self):
        table = self.table.cpu()
        return [rows_of(table, s, n) for s, n in enumerate(self.lens)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(16, 2), (10, 2)])
def test_serving_loop(msa, fp8, hq, hkv):
    lp = Loop(msa, 4, hq, hkv, fp8)
    prefill = msa.msa_dense_attn_prefill_paged_fp8 if fp8 else msa.msa_dense_attn_prefill_paged
    tree = msa.msa_tree_attn_paged_fp8 if fp8 else msa.msa_tree_attn_paged
    decode = msa.msa_dense_attn_decode_paged_fp8 if fp8 else msa.msa_dense_attn_decode_paged
    for new in ([300, 0, 17, 129], [100, 260, 1, 128], [0, 5, 700, 3]):
        prob, q = lp.grow(new)
        got = prefill(prob, q, lp.k, lp.v, *lp.scales(), lp.table)
        check(got, reference(new, lp.lens, lp.key_rows(), q, lp.k, lp.v, lp.ks, lp.vs, 0.0, None), f"prompt {new}")
    # drafts: a chain of two and its sibling; each sees itself and its ancestors
    new = [3, 3, 0, 3]
    prob, q = lp.grow(new)
    see = torch.tensor([[1, 0, 0], [1, 1, 0], [1, 0, 1]], dtype=torch.bool)
    bits = torch.tensor([1, 3, 5] * 3, dtype=torch.int32, device="cuda").view(9, 1)
    got = tree(prob, q, lp.k, lp.v, *lp.scales(), lp.table, bits)
    check(got, reference(new, lp.lens, lp.key_rows(), q, lp.k, lp.v, lp.ks, lp.vs, 0.0,
                         [see, see, see[:0, :0], see]), "tree")
    # the first two are accepted: the third's slot is taken back and written by the next step
    lp.lens = [n - (1 if x else 0) for n, x in zip(lp.lens, new)]
    lp.device_lens.copy_(torch.tensor(lp.lens, dtype=torch.int32))
    if all(n % PAGE for n in lp.lens):
        for _ in range(3):
            prob, q = lp.grow([1] * 4)
            o, lse = decode(prob, q, lp.k, lp.v, *lp.scales(), lp.table)
            ro, rl, _, to, tl, _ = dense_reference(lp.lens, lp.table, q, lp.k, lp.v, lp.ks, lp.vs)
            assert ((o.double() - ro).abs() <= to).all() and ((lse.double() - rl).abs() <= tl).all()
            # one new token a sequence is a prompt chunk too
            got = prefill(prob, q, lp.k, lp.v, *lp.scales(), lp.table)
            check(got, reference([1] * 4, lp.lens, lp.key_rows(), q, lp.k, lp.v, lp.ks, lp.vs, 0.0, None), "step")


@pytest.mark.parametrize("layout,tree", [("packed", False), ("paged", False), ("fp8", False), ("paged", True), ("fp8", True)])
@pytest.mark.parametrize("q,kv", [([200, 3], [300, 700]), ([7], [20000])])
def test_captured(msa, layout, tree, q, kv):
    """A replay gives the direct call's bits, follows queries and lengths rewritten in place, and two graphs may take turns
    on one workspace."""
    b = Batch(msa, q, kv, 16, 2, layout, seed=43, tree=tree)
    ws = msa.workspace(b.prob, b.op())
    outs = [(torch.empty_like(b.q), torch.empty(sum(q), 16, device="cuda")) for _ in range(2)]
    b.run(ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for o, lse in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(o=o, lse=lse, ws=ws)
        graphs.append(g)
    for rep in range(3):
        b.q.copy_(torch.randn(b.q.shape, device="cuda").to(torch.bfloat16) * (1 + rep))
        if rep == 2 and len(kv) == 2:   # another cut between the sequences: the batch's sizes stay
            b.prob.cu_k[1] += 1
        for o, _ in outs:
            o.fill_(7)
        for g in graphs:
            g.replay()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = b.run()
        for got in outs:
            assert same_bits(got, want)


def test_streams_at_once(msa):
    """Calls on several streams, each with a workspace of its own."""
    batches = [Batch(msa, [50 * i + 1, 9], [900, 4000 + i], 16, 2, ("packed", "paged", "fp8")[i % 3], seed=i) for i in range(6)]
    want = [b.run() for b in batches]
    spaces = [msa.workspace(b.prob, b.op()) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(5):
        got = []
        for b, ws, s in zip(batches, spaces, streams):
            with torch.cuda.stream(s):
                got.append(b.run(ws=ws))
        torch.cuda.synchronize()
        for g, w, ws in zip(got, want, spaces):
            assert same_bits(g, w)
            assert msa.msa_read_device_status(ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_beyond_32_bits(msa, fp8):
    """The last pages of caches of more than 2^32 bytes, and of more than 2^31 values."""
    pages = 66000 if fp8 else 33000
    lp = Loop(msa, 3, 16, 4, fp8, pages=pages)
    lp.free = torch.arange(pages - 1, pages - 60, -1, dtype=torch.int32, device="cuda")
    prefill = msa.msa_dense_attn_prefill_paged_fp8 if fp8 else msa.msa_dense_attn_prefill_paged
    for new in ([300, 17, 0], [5, 900, 129]):
        prob, q = lp.grow(new)
        rows = lp.key_rows()
        assert min(int(r.min()) for r in rows if len(r)) * lp.k.shape[1] * DIM > 2 ** (32 if fp8 else 31)
        got = prefill(prob, q, lp.k, lp.v, *lp.scales(), lp.table)
        check(got, reference(new, lp.lens, rows, q, lp.k, lp.v, lp.ks, lp.vs, 0.0, None), f"{new}")


def test_captured_loop(msa):
    """Tables, rows and attention of a step in one graph, replayed: the cache grows by itself."""
    S, hq, hkv, steps = 3, 16, 2, 40
    lp = Loop(msa, S, hq, hkv, False, pages=40, width=8, seed=3)
    lp.grow([100, 255, 7])
    new, ws_t = torch.ones(S, dtype=torch.int32, device="cuda"), msa.extend_workspace(S)
    x = torch.empty(S, (hq + 2 * hkv) * DIM, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([hq * DIM, hkv * DIM, hkv * DIM], dim=1)
    outs = dict(cu_q=torch.zeros(S + 1, dtype=torch.int32, device="cuda"), cu_k=torch.zeros(S + 1, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(S, dtype=torch.int64, device="cuda"), positions=torch.zeros(S, dtype=torch.int32, device="cuda"))
    qs, o, lse = torch.empty(S, hq, DIM, dtype=torch.bfloat16, device="cuda"), None, None

    def step(prob, **kw):
        msa.msa_extend_block_table(lp.device_lens, new, lp.free, lp.table, S, taken=lp.taken, taken_out=lp.taken,
                                   new_lengths=lp.device_lens, num_pages=40, ws=ws_t, **outs)
        msa.msa_append_paged(k.view(S, hkv, DIM), v.view(S, hkv, DIM), outs["slots"], lp.k, lp.v)
        qs.copy_(q.reshape(S, hq, DIM))
        return msa.msa_dense_attn_prefill_paged(prob, qs, lp.k, lp.v, lp.table, **kw)

    for i in range(steps):
        lp.lens = [n + 1 for n in lp.lens]
        x.normal_(generator=lp.gen)
        prob = msa.Problem(outs["cu_q"], outs["cu_k"], S, sum(lp.lens), 1, max(lp.lens), hq, hkv, 128, 16)
        o, lse = step(prob)
        if i % 13 == 0:
            check((o, lse), reference([1] * S, lp.lens, lp.key_rows(), qs, lp.k, lp.v, None, None, 0.0, None), f"step {i}")
    # the same step captured: its tables and rows move on with every replay
    g = torch.cuda.CUDAGraph()
    slots = []
    with torch.cuda.graph(g):
        msa.msa_extend_block_table(lp.device_lens, new, lp.free, lp.table, S, taken=lp.taken, taken_out=lp.taken,
                                   new_lengths=lp.device_lens, num_pages=40, ws=ws_t, **outs)
        msa.msa_append_paged(k.view(S, hkv, DIM), v.view(S, hkv, DIM), outs["slots"], lp.k, lp.v)
    for _ in range(30):
        x.normal_(generator=lp.gen)
        g.replay()
        slots.append(outs["slots"].tolist())
        assert torch.equal(lp.k[outs["slots"]], k.view(S, hkv, DIM))
    assert lp.device_lens.tolist() == [n + 30 for n in lp.lens]
    assert len({s for row in slots for s in row}) == 30 * S   # no slot twice
    assert blocks(lp.lens[0] + 30) <= 8
