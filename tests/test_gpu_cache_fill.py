"""Block tables and slot maps from lengths, and new tokens' rows written into pages, against plain implementations.

Numbers: tables, slots and bf16 rows are exact.  An E4M3 scale is one fp32 division, a code is that of an exact quotient
or of the same fp32 operations as in the reference: both are equal.
"""
import pytest
import torch

from paged_reference import PAGE, blocks, quantize_pages

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def extend_reference(lengths, new, free, table, capacity, taken, n_pages):
    """Plain loops on the host; returns (table, cu_q, cu_k, slots, positions, taken)."""
    table = [row[:] for row in table]
    cu_q, cu_k, slots, positions = [0], [0], [], []
    want = taken
    for s, (a, b) in enumerate(zip(lengths, new)):
        for j in range(blocks(a), blocks(a + b)):
            page = free[want] if want < len(free) else -1
            table[s][j] = page if 0 <= page < n_pages else -1
            want += 1
        for p in range(a, a + b):
            page = table[s][p // PAGE]
            slots.append(page * PAGE + p % PAGE if 0 <= page < n_pages else -1)
            positions.append(p)
        cu_q.append(cu_q[-1] + b)
        cu_k.append(cu_k[-1] + a + b)
    pad = capacity - len(slots)
    return table, cu_q, cu_k, slots + [-1] * pad, positions + [0] * pad, min(want, len(free))


def extend_case(lengths, new, spare, seed, extra_width=1):
    gen = torch.Generator().manual_seed(seed)
    used = sum(map(blocks, lengths))
    need = sum(blocks(a + b) - blocks(a) for a, b in zip(lengths, new))
    pages = torch.randperm(used + need + spare, generator=gen).tolist()
    width = max(1, max(blocks(a + b) for a, b in zip(lengths, new))) + extra_width
    table, at = [], 0
    for n in lengths:
        table.append(pages[at:at + blocks(n)] + [-7] * (width - blocks(n)))
        at += blocks(n)
    return pages, pages[at:], table


def check_extend(msa, lengths, new, free, table, capacity, n_pages, taken=0, status=0, **kw):
    t = i32(table)
    ws = msa.extend_workspace(len(lengths))
    got = msa.msa_extend_block_table(i32(lengths), i32(new), i32(free) if free else torch.empty(0, dtype=torch.int32, device="cuda"),
                                     t, capacity, taken=i32([taken]) if taken else None, num_pages=n_pages, ws=ws, **kw)
    assert msa.msa_read_device_status(ws) == status
    want = extend_reference(lengths, new, free, table, capacity, taken, n_pages)
    assert t.tolist() == want[0]
    for g, w, name in zip(got, (*want[1:5], [want[5]]), ("cu_q", "cu_k", "slots", "positions", "taken")):
        assert g.tolist() == w, name
    return t, got


@pytest.mark.parametrize("lengths,new", [
    ([0], [0]), ([0], [1]), ([127], [1]), ([128], [1]), ([128], [0]), ([1], [127]), ([1], [128]), ([5], [700]),
    ([0, 128, 300, 1], [1, 1, 1, 1]), ([0, 0, 0], [0, 0, 0]), ([10, 20, 0, 127], [0, 300, 0, 2]),
    ([255, 256, 257], [129, 128, 127])])
def test_tables(msa, lengths, new):
    pages, free, table = extend_case(lengths, new, 3, 1)
    for pad in (0, 5):
        check_extend(msa, lengths, new, free, table, sum(new) + pad, len(pages))


@pytest.mark.parametrize("seqs,most", [(33, 300), (1025, 40), (3000, 3), (2, 70000), (5000, 0)])
def test_large_tables(msa, seqs, most):
    gen = torch.Generator().manual_seed(seqs)
    lengths = torch.randint(0, 1000, (seqs,), generator=gen).tolist()
    new = torch.randint(0, most + 1, (seqs,), generator=gen).tolist()
    pages, free, table = extend_case(lengths, new, 3, 2)
    check_extend(msa, lengths, new, free, table, sum(new) + 17, len(pages))


def test_pages_run_out(msa):
    lengths, new = [100, 0, 200], [200, 300, 400]
    pages, free, table = extend_case(lengths, new, 0, 3)
    for left in (0, 1, 4, len(free) - 1):
        check_extend(msa, lengths, new, free[:left], table, 900, len(pages), status=msa.DEVICE_BAD_INDEX)
    check_extend(msa, lengths, new, free, table, 900, len(pages))
    check_extend(msa, lengths, new, [0, 0] + free, table, 900, len(pages), taken=2)


def test_pages_outside_the_cache(msa):
    lengths, new = [100, 0], [200, 300]
    pages, free, table = extend_case(lengths, new, 0, 4)
    for bad in (-1, len(pages), 2 ** 31 - 1, -2 ** 31):
        f = free[:]
        f[1] = bad
        check_extend(msa, lengths, new, f, table, 500, len(pages), status=msa.DEVICE_BAD_INDEX)
    table[0][0] = -1   # the block that the first sequence's new tokens begin in
    t = i32(table)
    ws = msa.extend_workspace(2)
    slots = msa.msa_extend_block_table(i32(lengths), i32(new), i32(free), t, 500, ws=ws)[2].tolist()
    assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX
    assert slots[:28] == [-1] * 28 and min(slots[28:]) >= 0


@pytest.mark.parametrize("lengths,new,capacity,taken", [
    ([-1, 5], [1, 1], 10, 0), ([1, 5], [1, -1], 10, 0), ([1, 5], [3, 4], 6, 0), ([1, 300], [1, 400], 1000, 0),
    ([1, 5], [1, 1], 10, 9), ([1, 5], [1, 1], 10, -1), ([2 ** 31 - 1, 1], [2 ** 31 - 1, 1], 10, 0)])
def test_lengths_that_cannot_be(msa, lengths, new, capacity, taken):
    """Nothing is taken; tokens have no slots."""
    table = i32([[3, 4], [5, 6]])
    before = table.clone()
    ws = msa.extend_workspace(2)
    grown = i32([-5, -5])
    cu_q, cu_k, slots, positions, out = msa.msa_extend_block_table(
        i32(lengths), i32(new), i32([9, 8, 7]), table, capacity, taken=i32([taken]), new_lengths=grown, ws=ws)
    assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_SEQLENS
    assert torch.equal(table, before) and out.tolist() == [taken] and grown.tolist() == [-5, -5]
    assert cu_q.tolist() == [0, 0, 0] and cu_k.tolist() == [0, 0, 0]
    assert slots.tolist() == [-1] * capacity and positions.tolist() == [0] * capacity


def test_steps_advance_by_themselves(msa):
    """A captured step, replayed: lengths and the place in the free list move on in place."""
    lengths, free = i32([120, 0, 300]), i32(list(range(10, 40)))
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[2, :3] = 1, i32([2, 3, 4])
    new, taken = i32([1, 1, 0]), i32([0])
    outs = dict(cu_q=i32([0] * 4), cu_k=i32([0] * 4), slots=torch.zeros(4, dtype=torch.int64, device="cuda"),
                positions=i32([0] * 4), ws=msa.extend_workspace(3))

    def step():
        msa.msa_extend_block_table(lengths, new, free, table, 4, taken=taken, new_lengths=lengths, taken_out=taken, **outs)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert lengths.tolist() == [141, 21, 300] and taken.tolist() == [2]
    assert table[0, :2].tolist() == [1, 11] and table[1, 0].item() == 10 and table[2, 3].item() == -1
    assert outs["cu_k"].tolist() == [0, 141, 162, 462] and outs["positions"].tolist() == [140, 20, 0, 0]
    assert outs["slots"].tolist() == [11 * 128 + 12, 10 * 128 + 20, -1, -1]


# ------------------------------------------------------------------------------------------------ rows
def slots_of(lengths, new, gen):
    """Slots of the new tokens of sequences in pages of random order; returns (slots, pages)."""
    n = sum(blocks(a + b) for a, b in zip(lengths, new)) + 2
    pages = torch.randperm(n, generator=gen).tolist()
    slots, at = [], 0
    for a, b in zip(lengths, new):
        mine = pages[at:at + blocks(a + b)]
        at += blocks(a + b)
        slots += [mine[p // PAGE] * PAGE + p % PAGE for p in range(a, a + b)]
    return slots, n


BATCHES = [([0], [1]), ([0], [128]), ([127], [2]), ([5], [300]), ([0, 130, 64, 1], [1, 1, 1, 1]), ([0] * 9, [100] * 9),
           ([17 * i % 400 for i in range(700)], [1] * 700), ([3, 0, 250], [1000, 0, 1500]), ([40] * 1100, [1 + i % 3 for i in range(1100)])]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("hkv,d_idx", [(1, 0), (4, 128), (3, 64), (12, 128)])
def test_rows(msa, batch, hkv, d_idx):
    lengths, new = BATCHES[batch]
    gen = torch.Generator().manual_seed(batch)
    slots, pages = slots_of(lengths, new, gen)
    N = len(slots)
    wide = torch.randn(N, (2 * hkv + 3) * 128 + 8, generator=gen).to(torch.bfloat16).cuda()
    k, v = wide[:, 8:8 + hkv * 128].view(N, hkv, 128), wide[:, 8 + hkv * 128:8 + 2 * hkv * 128].view(N, hkv, 128)
    caches = [torch.randn(pages * PAGE, hkv, 128, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    rows, more = [k, v], {}
    if d_idx:
        rows.append(wide[:, -d_idx:])
        caches.append(torch.randn(pages * PAGE, d_idx, generator=gen).to(torch.bfloat16).cuda())
        more = dict(k_idx=rows[2], k_idx_cache=caches[2])
    if N > 3:
        slots[2] = -1
    want = [c.clone() for c in caches]
    at = torch.tensor(slots, dtype=torch.int64, device="cuda")
    for w, x in zip(want, rows):
        w[at[at >= 0]] = x[at >= 0]
    ws = msa.append_workspace(pages)
    msa.msa_append_paged(k, v, at, caches[0], caches[1], ws=ws, **more)
    assert msa.msa_read_device_status(ws) == 0
    for w, c in zip(want, caches):
        assert torch.equal(w, c)


def append_fp8_reference(x, slots, codes, scale):
    """Page by page on the host, in fp32: (codes, scale) [pages * 128, heads, 128] and [pages, heads]."""
    codes, scale = codes.cpu().clone(), scale.cpu().clone()
    x = x.float().cpu()
    runs, last = [], None
    for i, s in enumerate(slots):
        page = s // PAGE if s >= 0 else None
        if page is not None and page == last:
            runs[-1].append(i)
        elif page is not None:
            runs.append([i])
        last = page
    for run in runs:
        page, offs = slots[run[0]] // PAGE, torch.tensor([slots[i] % PAGE for i in run])
        low, mine = int(offs.min()), x[run]
        finite = torch.where(torch.isfinite(mine), mine.abs(), torch.zeros_like(mine))
        amax = finite.amax(dim=(0, 2))
        fresh = torch.where(amax >= 2.0 ** -118, amax / 448.0, torch.zeros_like(amax))
        was = scale[page].clone()
        now = torch.maximum(was, fresh) if low > 0 else fresh
        now = torch.where(now > 0, now, torch.ones_like(now))
        p = codes[page * PAGE:(page + 1) * PAGE]
        old = (p[:low].view(torch.float8_e4m3fn).float() * 448.0 * was[None, :, None]) / amax[None, :, None]
        grew = (now != was)[None, :, None].expand(old.shape)
        p[:low] = torch.where(grew, e4m3(old), p[:low])
        # exact where the new rows set the scale: 11 significant bits over 8 are at least 2^-14 away from the middle of two
        # codes or in it, and the quotient's roundings to 53 and 24 bits keep that
        exact = (mine.double() * 448.0 / amax.double()[None, :, None]).float()
        p[offs] = e4m3(torch.where(((now == fresh) & (fresh > 0))[None, :, None], exact, mine / now[None, :, None]))
        scale[page] = now
    return codes, scale


def e4m3(x):
    """Round to nearest even, saturated; NaN stays NaN."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("gain", [0.2, 5.0])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("hkv,index", [(1, False), (4, True), (12, False)])
def test_rows_fp8(msa, batch, hkv, index, gain):
    lengths, new = BATCHES[batch]
    gen = torch.Generator().manual_seed(batch)
    slots, pages = slots_of(lengths, new, gen)
    N = len(slots)
    wide = (torch.randn(N, (2 * hkv + 1) * 128, generator=gen) * gain).to(torch.bfloat16).cuda()
    k, v = wide[:, :hkv * 128].view(N, hkv, 128), wide[:, hkv * 128:2 * hkv * 128].view(N, hkv, 128)
    rows, caches, scales, more = [k, v], [], [], {}
    heads = [hkv, hkv] + ([1] if index else [])
    for h in heads:
        c, s = quantize_pages(torch.randn(pages * PAGE, h, 128, generator=gen).to(torch.bfloat16))
        caches.append(c.cuda())
        scales.append(s.cuda())
    if index:
        rows.append(wide[:, -128:].unsqueeze(1))
        more = dict(k_idx=rows[2][:, 0], k_idx8_cache=caches[2][:, 0], k_idx_scale=scales[2][:, 0])
    if N > 3:
        slots[N // 2] = -1
    if N == 2500:   # a slot left out inside a page: its tokens then come twice
        slots[N // 2] = slots[N // 2 - 1] + 1
    at = torch.tensor(slots, dtype=torch.int64, device="cuda")
    want = [append_fp8_reference(x, slots, c, s) for x, c, s in zip(rows, caches, scales)]
    ws = msa.append_workspace(pages)
    msa.msa_append_paged_fp8(k, v, at, caches[0], caches[1], scales[0], scales[1], ws=ws, **more)
    twice = len({s // PAGE for s in slots if s >= 0}) != sum(
        1 for i, s in enumerate(slots) if s >= 0 and (i == 0 or slots[i - 1] < 0 or slots[i - 1] // PAGE != s // PAGE))
    assert msa.msa_read_device_status(ws) == (msa.DEVICE_BAD_INDEX if twice else 0)
    if twice:
        return
    for (wc, wsc), c, s in zip(want, caches, scales):
        assert torch.equal(wsc, s.cpu())
        assert torch.equal(wc, c.cpu())


def test_fp8_values_out_of_the_ordinary(msa):
    """Zeros, tiny values, inf and NaN: they do not decide a page's scale; inf saturates, NaN stays."""
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(6, 2, 128, generator=gen).to(torch.bfloat16)
    x[0] = 0
    x[1] = 1e-37
    x[2, 0, 3], x[2, 1, 5] = float("inf"), float("nan")
    x[3] = torch.finfo(torch.bfloat16).max
    x[4, 0, 0] = -float("inf")
    slots = [0, PAGE, 2 * PAGE, 3 * PAGE + 4, 4 * PAGE + 100, 4 * PAGE + 127]
    codes, scale = quantize_pages(torch.randn(6 * PAGE, 2, 128, generator=gen).to(torch.bfloat16))
    wc, wsc = append_fp8_reference(x, slots, codes, scale)
    c, s, c2, s2 = codes.cuda(), scale.cuda(), codes.cuda(), scale.cuda()
    ws = msa.append_workspace(6)
    msa.msa_append_paged_fp8(x.cuda(), x.cuda(), torch.tensor(slots, device="cuda"), c, c2, s, s2, ws=ws)
    assert msa.msa_read_device_status(ws) == 0
    assert torch.equal(s.cpu(), wsc) and torch.equal(s2.cpu(), wsc)
    nan = torch.isnan(wc.view(torch.float8_e4m3fn).float())
    for got in (c, c2):
        assert torch.equal(torch.isnan(got.cpu().view(torch.float8_e4m3fn).float()), nan)
        assert torch.equal(got.cpu()[~nan], wc[~nan])


def test_slots_outside_the_cache(msa):
    for fp8 in (False, True):
        x = torch.randn(5, 2, 128, device="cuda").to(torch.bfloat16)
        slots = torch.tensor([0, 3 * PAGE, -2, 2 ** 62, -2 ** 63], device="cuda")
        ws = msa.append_workspace(3)
        if fp8:
            c = [torch.zeros(3 * PAGE, 2, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
            s = [torch.ones(3, 2, device="cuda") for _ in range(2)]
            msa.msa_append_paged_fp8(x, x, slots, *c, *s, ws=ws)
            assert (s[0][1:] == 1).all()
        else:
            c = [torch.zeros(3 * PAGE, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            msa.msa_append_paged(x, x, slots, *c, ws=ws)
            assert torch.equal(c[0][0], x[0]) and torch.equal(c[1][0], x[0])
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX
        assert (c[0][1:] == 0).all() and (c[1][1:] == 0).all()
