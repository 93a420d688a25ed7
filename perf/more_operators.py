"""Measured cases of the operators that fill a paged cache and read it with many new tokens at once: block tables and
slot maps from the requests' lengths, the new tokens' K and V rows written into the pages (bf16 or E4M3), causal
attention of prompts and prompt chunks, and attention of a tree of drafted tokens over the cache.

``own`` selects the framework's kernels; otherwise ``run`` computes the same results with elementary torch operations
in 32 bits, rounded once at the end.  ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

PAGE = 128        # tokens of a cache page
DIM = 128         # head dimension
E4M3_MAX = 448.0
TINY = 2.0 ** -118  # values below this are zeros in E4M3


def listed():
    return [
        # one user's short prompt: latency
        {"name": "prompt_1x333", "op": "prompt", "seqs": 1, "new": 333, "past": 0, "ragged": False, "hq": 64,
         "hkv": 4, "cache": "packed"},
        # chunks of long prompts behind what is cached already
        {"name": "prompt_6_chunks", "op": "prompt", "seqs": 6, "new": 2048, "past": 30000, "ragged": True, "hq": 64,
         "hkv": 4, "cache": "paged"},
        # a batch of ordinary prompts over an 8-bit cache, a group of five heads
        {"name": "prompt_20_ragged_fp8", "op": "prompt", "seqs": 20, "new": 3001, "past": 0, "ragged": True, "hq": 40,
         "hkv": 8, "cache": "fp8"},
        # one long prompt
        {"name": "prompt_1x20000", "op": "prompt", "seqs": 1, "new": 20000, "past": 0, "ragged": False, "hq": 64,
         "hkv": 4, "cache": "packed"},
        # one user's drafted tokens: latency
        {"name": "tree_1x8", "op": "tree", "seqs": 1, "new": 8, "past": 2000, "ragged": False, "hq": 64, "hkv": 4,
         "cache": "paged"},
        # a serving batch of mixed lengths and mixed trees
        {"name": "tree_16_ragged", "op": "tree", "seqs": 16, "new": 31, "past": 32768, "ragged": True, "hq": 64,
         "hkv": 4, "cache": "paged"},
        # large trees over long 8-bit caches
        {"name": "tree_8x61_fp8", "op": "tree", "seqs": 8, "new": 61, "past": 65521, "ragged": False, "hq": 32,
         "hkv": 8, "cache": "fp8"},
        # the tables of a decode step
        {"name": "tables_24_step", "op": "tables", "seqs": 24, "new": 1, "past": 16384, "ragged": False},
        # the tables of a large batch, prompts and decode steps mixed
        {"name": "tables_2000_mixed", "op": "tables", "seqs": 2000, "new": 701, "past": 8192, "ragged": True},
        # a decode step's rows
        {"name": "append_16_step", "op": "append", "seqs": 16, "new": 1, "past": 5000, "ragged": True, "hq": 64,
         "hkv": 4, "cache": "paged", "index": True},
        # a large decode step's rows into 8-bit pages that have rows already
        {"name": "append_256_step_fp8", "op": "append", "seqs": 256, "new": 1, "past": 1500, "ragged": True, "hq": 40,
         "hkv": 8, "cache": "fp8", "index": False},
        # prompts into 8-bit pages
        {"name": "append_6_prompts_fp8", "op": "append", "seqs": 6, "new": 12001, "past": 300, "ragged": True,
         "hq": 64, "hkv": 4, "cache": "fp8", "index": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "tree", "tree", "tables", "append"))
    if op == "tables":
        seqs = _spread(rng, 1, 4000)
        return {"op": op, "seqs": seqs, "new": _spread(rng, 1, max(1, 1_400_000 // seqs)),
                "past": _spread(rng, 1, 16384), "ragged": rng.random() < 0.7}
    hq, hkv = rng.choice(((64, 4), (64, 4), (32, 8), (40, 8), (128, 1), (12, 12), (28, 4), (96, 2)))
    ragged = rng.random() < 0.7
    if op == "append":
        seqs = _spread(rng, 1, 256)
        new = _spread(rng, 1, max(1, min(12000, 500_000 // (seqs * hkv))))
        past = _spread(rng, 1, max(1, min(8192, 1_500_000 // (seqs * hkv))))
        return {"op": op, "seqs": seqs, "new": new, "past": past, "ragged": ragged, "hq": hq, "hkv": hkv,
                "cache": rng.choice(("paged", "fp8")), "index": rng.random() < 0.5}
    seqs = _spread(rng, 1, 32)
    if op == "tree":
        new = _spread(rng, 1, 64)
        past = _spread(rng, 1, max(1, min(300_000, 3_000_000 // (seqs * hkv), 1_000_000_000 // (seqs * new * hq))))
        return {"op": op, "seqs": seqs, "new": new, "past": past, "ragged": ragged, "hq": hq, "hkv": hkv,
                "cache": rng.choice(("paged", "fp8"))}
    new = _spread(rng, 1, 16384)
    past = 0 if rng.random() < 0.5 else _spread(rng, 1, 50000)
    # a batch's pairs of query and key, over all heads, stay under those of the largest prompt, its keys in memory
    while seqs * new * (past + new) * hq > 9_000_000_000 or seqs * (past + new) * hkv > 3_000_000:
        seqs, new, past = -(-seqs // 2), -(-new * 2 // 3), past * 2 // 3
    return {"op": op, "seqs": seqs, "new": new, "past": past, "ragged": ragged, "hq": hq, "hkv": hkv,
            "cache": rng.choice(("packed", "paged", "fp8"))}


def _lengths(case):
    """(new tokens, cached tokens before them) of each sequence, by the case alone; in a ragged batch of eight or more
    some have no new tokens and some are new."""
    n, new, past = case["seqs"], case["new"], case["past"]
    if not case["ragged"]:
        return [new] * n, [past] * n
    q = [1 + int((new - 1) * (((i + 1) * 0.6180339887) % 1.0)) for i in range(n)]
    p = [int(past * (((i + 1) * 0.7548776662) % 1.0)) for i in range(n)]
    q[0], p[0] = new, past
    return [0 if i % 8 == 5 else v for i, v in enumerate(q)], [0 if i % 8 == 6 else v for i, v in enumerate(p)]


def _blocks(n):
    return -(-n // PAGE)


def _ends(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _table(pages, blocks, width):
    """A block table of the given numbers of pages, which are taken from `pages` in order; -1 past the last."""
    table = torch.full((len(blocks), width), -1, dtype=torch.int32)
    at = 0
    for s, b in enumerate(blocks):
        table[s, :b] = pages[at:at + b]
        at += b
    return table.cuda()


def _quantized(x):
    """bf16 pages [pages * 128, heads, 128] as E4M3 codes and one scale per (page, head)."""
    f = x.view(-1, PAGE, x.shape[1], DIM)
    amax = f.abs().amax(dim=(1, 3)).float()
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    codes = (f.float() / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(x.shape), scale


def _tree(q_lens, words, host):
    """Visibility of drafts to drafts, a bit each: every draft sees itself and its ancestors; a parent is any earlier
    draft or the last cached token."""
    rows = []
    for n in q_lens:
        pick = torch.rand(max(1, n), generator=host).tolist()
        own_rows = []
        for i in range(n):
            parent = int(pick[i] * (i + 1)) - 1
            own_rows.append((own_rows[parent] if parent >= 0 else 0) | (1 << i))
        rows += own_rows
    signed = [[((r >> (32 * w)) & 0xFFFFFFFF) - (1 << 32 if (r >> (32 * w + 31)) & 1 else 0) for w in range(words)]
              for r in rows]
    return torch.tensor(signed, dtype=torch.int32).reshape(len(rows), words).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen)

    st = dict(case)
    new, past = _lengths(case)
    total = [a + b for a, b in zip(new, past)]
    S, N = case["seqs"], sum(new)
    st["tokens"] = N
    st["q_lens"], st["kv_lens"] = new, total
    if case["op"] == "tables":
        # a pool of pages, some of them in use in random order, the others free in random order
        order = torch.randperm(sum(map(_blocks, total)) + 5, generator=host).to(torch.int32)
        used = sum(map(_blocks, past))
        st["table"] = _table(order, list(map(_blocks, past)), max(map(_blocks, total)) + 2)
        st["free"] = order[used:].cuda()
        st["past_lens"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        if own:
            import block_sparse_attention_05_gb300 as msa
            st["ws"] = msa.extend_workspace(S)
        return st
    hq, hkv = case["hq"], case["hkv"]
    st["cu_q"], st["cu_k"] = _ends(new), _ends(total)
    paged = case["cache"] != "packed"
    if paged:
        pages = torch.randperm(sum(map(_blocks, total)) + 3, generator=host).to(torch.int32)
        n_pages = len(pages)
        st["table"] = _table(pages, list(map(_blocks, total)), max(1, max(map(_blocks, total))))
        rows = n_pages * PAGE
    else:
        n_pages, rows = 0, max(1, sum(total))
    st["k"], st["v"] = normal(rows, hkv, DIM), normal(rows, hkv, DIM)
    if case["op"] == "append":
        # the new rows are slices of one projection's output
        width = (hq + 2 * hkv) * DIM
        qkv = normal(N, width) * 2
        st["k_new"] = qkv[:, hq * DIM:(hq + hkv) * DIM].view(N, hkv, DIM)
        st["v_new"] = qkv[:, (hq + hkv) * DIM:].view(N, hkv, DIM)
        if case["index"]:
            st["i_new"], st["i"] = normal(N, DIM), normal(rows, DIM)
        at = []
        table = st["table"].tolist()
        for s in range(S):
            at += [table[s][p // PAGE] * PAGE + p % PAGE for p in range(past[s], total[s])]
        st["slots"] = torch.tensor(at, dtype=torch.int64, device="cuda")
    if case["cache"] == "fp8":
        st["k"], st["k_scale"] = _quantized(st["k"])
        st["v"], st["v_scale"] = _quantized(st["v"])
        if case.get("index"):
            codes, scale = _quantized(st["i"][:, None, :])
            st["i"], st["i_scale"] = codes[:, 0], scale[:, 0].contiguous()
    if case["op"] == "tree":
        st["visible"] = _tree(new, -(-max(new) // 32), host)
    if case["op"] in ("prompt", "tree"):
        st["q"] = normal(N, hq, DIM) * 2
    if own:
        # what a serving loop keeps from step to step: the batch's sizes and a workspace; no work on the data
        import block_sparse_attention_05_gb300 as msa
        if case["op"] == "append":
            st["ws"] = msa.append_workspace(n_pages) if case["cache"] == "fp8" else None
        else:
            st["problem"] = msa.Problem(st["cu_q"], st["cu_k"], N, sum(total), max(new), max(total), hq, hkv, 128, 16)
            st["ws"] = msa.workspace(st["problem"], msa.Op.TREE_ATTN if case["op"] == "tree"
                                     else msa.Op.DENSE_ATTN_PREFILL)
    return st


def _plain_tables(st):
    past, new, free = st["past_lens"], st["new_lens"], st["free"]
    total = past + new
    old, now = (past + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    need = now - old
    last = torch.cumsum(need, 0)
    col = torch.arange(st["table"].shape[1], device="cuda")
    fresh = (col[None, :] >= old[:, None]) & (col[None, :] < now[:, None])
    take = ((last - need)[:, None] + col[None, :] - old[:, None]).clamp_(0, len(free) - 1)
    st["table"].copy_(torch.where(fresh, free[take], st["table"]))
    cu_q, cu_k = (torch.nn.functional.pad(torch.cumsum(x, 0, dtype=torch.int32), (1, 0)) for x in (new, total))
    N = st["tokens"]
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=N)
    pos = past[seq] + (torch.arange(N, dtype=torch.int32, device="cuda") - cu_q[:-1][seq])
    slots = st["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE
    return {"table": st["table"], "cu_q": cu_q, "cu_k": cu_k, "slots": slots, "positions": pos,
            "taken": last[-1:].to(torch.int32)}


def _caches(st):
    out = {}
    for name in ("k", "v", "i"):
        if name in st:
            out[name] = st[name].view(torch.float8_e4m3fn) if st["cache"] == "fp8" else st[name]
            if st["cache"] == "fp8":
                out[name + "_scale"] = st[name + "_scale"]
    return out


def _plain_append(st):
    slots = st["slots"]
    if st["cache"] != "fp8":
        st["k"][slots], st["v"][slots] = st["k_new"], st["v_new"]
        if st["index"]:
            st["i"][slots] = st["i_new"]
        return _caches(st)
    page, off = slots // PAGE, slots % PAGE
    pages = st["k"].shape[0] // PAGE
    # the rows of a page before its first new one are live and keep their values
    first = torch.full((pages,), PAGE, dtype=torch.int64, device="cuda").scatter_reduce_(0, page, off, "amin")
    # the pages to look at: the tokens' where those are few (a page of two tokens is then written twice alike), or all
    sel = page if len(page) < pages else torch.arange(pages, device="cuda")
    names = (("k", st["k_new"]), ("v", st["v_new"])) + ((("i", st["i_new"][:, None, :]),) if st["index"] else ())
    for name, x in names:
        heads = x.shape[1]
        codes, scale = st[name].view(pages, PAGE, heads, DIM), st[name + "_scale"].view(pages, heads)
        amax = torch.zeros(pages, heads, device="cuda")
        amax.scatter_reduce_(0, page[:, None].expand(-1, heads), x.float().abs().amax(-1), "amax")
        was, top, live = scale[sel], amax[sel] / E4M3_MAX, first[sel]
        now = torch.where(amax[sel] >= TINY, top, torch.zeros_like(top))
        now = torch.maximum(now, torch.where(live[:, None] > 0, was, torch.zeros_like(was)))
        now = torch.where(live[:, None] < PAGE, torch.where(now > 0, now, torch.ones_like(now)), was)
        old = codes[sel]
        again = old.view(torch.float8_e4m3fn).float() * was[:, None, :, None] / now[:, None, :, None]
        mine = (torch.arange(PAGE, device="cuda")[None, :] < live[:, None]) & (live < PAGE)[:, None]
        grew = mine[:, :, None, None] & (now != was)[:, None, :, None]
        codes[sel] = torch.where(grew, again.to(torch.float8_e4m3fn).view(torch.uint8), old)
        scale[sel] = now
        rows = (x.float() / scale[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        st[name].view(-1, heads, DIM)[slots] = rows
    return _caches(st)


def _plain_attention(st):
    S, hq, hkv = st["seqs"], st["hq"], st["hkv"]
    G, N = hq // hkv, st["tokens"]
    max_q, n = max(st["q_lens"]), max(st["kv_lens"])
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    q_len, kv_len = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    past = kv_len - q_len
    key = torch.arange(n, device="cuda")
    if st["cache"] == "packed":
        rows = (cu_k[:-1, None] + key).clamp_(max=st["k"].shape[0] - 1)
    else:
        rows = (st["table"][:, key // PAGE].long() * PAGE + key % PAGE).clamp_(min=0)
    k, v = st["k"][rows], st["v"][rows]
    if st["cache"] == "fp8":
        k = k.view(torch.float8_e4m3fn).float() * st["k_scale"][rows // PAGE][..., None]
        v = v.view(torch.float8_e4m3fn).float() * st["v_scale"][rows // PAGE][..., None]
    k, v = k.float().permute(0, 2, 3, 1), v.float().permute(0, 2, 1, 3)
    t = torch.arange(max_q, device="cuda")
    q = st["q"][(cu_q[:-1, None] + t).clamp_(max=N - 1)].float().view(S, max_q, hkv, G, DIM)
    o = torch.empty(S, max_q, hq, DIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(S, max_q, hq, device="cuda")
    step = max(1, 2_000_000_000 // (S * hq * n))       # logits of 8 GB at a time
    for a in range(0, max_q, step):
        b = min(max_q, a + step)
        # keys that these queries can see in any sequence
        top = n if st["op"] == "tree" else max(kv - ql + min(b, ql) for ql, kv in zip(st["q_lens"], st["kv_lens"]))
        s = q[:, a:b].permute(0, 2, 3, 1, 4).reshape(S, hkv, G * (b - a), DIM) @ k[..., :top]
        s = s.view(S, hkv, G, b - a, top) * DIM ** -0.5
        d = key[:top] - past[:, None]                  # a key's place among the new tokens
        if st["op"] == "tree":
            mask = st["visible"][(cu_q[:-1, None] + t[a:b]).clamp_(max=N - 1)]
            at = d.clamp(0, 32 * mask.shape[-1] - 1)
            word = torch.gather(mask, 2, (at // 32)[:, None, :].expand(S, b - a, top))
            seen = ((word >> (at % 32)[:, None, :].to(torch.int32)) & 1).bool() & (d < q_len[:, None])[:, None, :]
            seen |= (d < 0)[:, None, :]
        else:
            seen = d[:, None, :] <= t[None, a:b, None]
        s.masked_fill_(~seen[:, None, None], -math.inf)
        m = s.amax(dim=-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = s.sub_(m).exp_()
        total = p.sum(dim=-1, keepdim=True)
        part = p.view(S, hkv, G * (b - a), top) @ v[:, :, :top]
        part = part.view(S, hkv, G, b - a, DIM) / torch.where(total > 0, total, torch.ones_like(total))
        o[:, a:b] = part.permute(0, 3, 1, 2, 4).reshape(S, b - a, hq, DIM).to(torch.bfloat16)
        lse[:, a:b] = (m + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(S, b - a, hq)
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), q_len, output_size=N)
    row = torch.arange(N, device="cuda") - cu_q[:-1][seq]
    return {"o": o[seq, row], "lse": lse[seq, row]}


def run(state):
    st = state
    if not own:
        if st["op"] == "tables":
            return _plain_tables(st)
        if st["op"] == "append":
            return _plain_append(st)
        return _plain_attention(st)
    import block_sparse_attention_05_gb300 as msa
    if st["op"] == "tables":
        cu_q, cu_k, slots, positions, taken = msa.msa_extend_block_table(
            st["past_lens"], st["new_lens"], st["free"], st["table"], st["tokens"], ws=st["ws"])
        return {"table": st["table"], "cu_q": cu_q, "cu_k": cu_k, "slots": slots, "positions": positions,
                "taken": taken}
    if st["op"] == "append":
        if st["cache"] == "fp8":
            msa.msa_append_paged_fp8(st["k_new"], st["v_new"], st["slots"], st["k"], st["v"], st["k_scale"],
                                     st["v_scale"], k_idx=st.get("i_new"), k_idx8_cache=st.get("i"),
                                     k_idx_scale=st.get("i_scale"), ws=st["ws"])
        else:
            msa.msa_append_paged(st["k_new"], st["v_new"], st["slots"], st["k"], st["v"], k_idx=st.get("i_new"),
                                 k_idx_cache=st.get("i"))
        return _caches(st)
    if st["op"] == "tree":
        if st["cache"] == "fp8":
            o, lse = msa.msa_tree_attn_paged_fp8(st["problem"], st["q"], st["k"], st["v"], st["k_scale"],
                                                 st["v_scale"], st["table"], st["visible"], ws=st["ws"])
        else:
            o, lse = msa.msa_tree_attn_paged(st["problem"], st["q"], st["k"], st["v"], st["table"], st["visible"],
                                             ws=st["ws"])
    elif st["cache"] == "fp8":
        o, lse = msa.msa_dense_attn_prefill_paged_fp8(st["problem"], st["q"], st["k"], st["v"], st["k_scale"],
                                                      st["v_scale"], st["table"], ws=st["ws"])
    elif st["cache"] == "paged":
        o, lse = msa.msa_dense_attn_prefill_paged(st["problem"], st["q"], st["k"], st["v"], st["table"], ws=st["ws"])
    else:
        o, lse = msa.msa_dense_attn_prefill(st["problem"], st["q"], st["k"], st["v"], ws=st["ws"])
    return {"o": o, "lse": lse}


def _pairs(case):
    """Visible pairs of a query and a key, over the batch (a tree's drafts as if all saw one another)."""
    if case["op"] == "tree":
        return sum(a * (a + b) for a, b in zip(*_lengths(case)))
    return sum(a * b + a * (a + 1) // 2 for a, b in zip(*_lengths(case)))


def work(case):
    new, past = _lengths(case)
    N = sum(new)
    if case["op"] == "tables":
        fresh = sum(_blocks(a + b) - _blocks(b) for a, b in zip(new, past))
        # lengths in, prefix sums out; a free page read and written into the table; a slot and a position per token
        return {"bytes": 16 * len(new) + 8 + 8 * fresh + 12 * N, "flops": 4 * N}
    hkv = case["hkv"]
    size = 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        width = 2 * hkv * DIM + (DIM if case["index"] else 0)
        total = N * (width * (2 + size) + 8)
        if case["cache"] == "fp8":
            pages = sum(_blocks(b + a) - b // PAGE for a, b in zip(new, past) if a)
            total += pages * 8 * (2 * hkv + case["index"])
        return {"bytes": total, "flops": N * width}
    hq = case["hq"]
    keys = sum(a + b for a, b in zip(new, past) if a)
    total = keys * 2 * hkv * DIM * size + N * hq * (4 * DIM + 4)
    if case["cache"] != "packed":
        total += sum(_blocks(a + b) for a, b in zip(new, past) if a) * (4 + (8 * hkv if size == 1 else 0))
    if case["op"] == "tree":
        total += N * 4 * -(-case["new"] // 32)
    return {"bytes": total, "flops": 4 * DIM * hq * _pairs(case)}


def _exact_tables(case, st):
    new, past = _lengths(case)
    table, free = st["table"].tolist(), st["free"].tolist()
    taken, slots, positions = 0, [], []
    for s, (a, b) in enumerate(zip(new, past)):
        for j in range(_blocks(b), _blocks(a + b)):
            table[s][j] = free[taken]
            taken += 1
        slots += [table[s][p // PAGE] * PAGE + p % PAGE for p in range(b, a + b)]
        positions += range(b, a + b)

    def whole(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device="cuda")

    return {"table": whole(table), "cu_q": _ends(new), "cu_k": _ends([a + b for a, b in zip(new, past)]),
            "slots": whole(slots, torch.int64), "positions": whole(positions), "taken": whole([taken])}


def _exact_append(case, st):
    new, past = _lengths(case)
    table = st["table"].tolist()
    fp8 = case["cache"] == "fp8"
    out = {}
    for name in ("k", "v", "i"):
        if name not in st:
            continue
        x = st[name + "_new"].double()
        if not fp8:
            pool = st[name].double()
            pool[st["slots"]] = x
            out[name] = pool
            continue
        pool, scales = st[name].view(torch.float8_e4m3fn).double(), st[name + "_scale"].double()
        at = 0
        for s, (a, b) in enumerate(zip(new, past)):
            p = b
            while p < a + b:
                off, n = p % PAGE, min(PAGE - p % PAGE, a + b - p)
                page = table[s][p // PAGE]
                rows, mine = pool[page * PAGE:(page + 1) * PAGE], x[at:at + n]
                top = mine.abs().amax(dim=(0, -1)) / E4M3_MAX
                now = torch.maximum(top, scales[page]) if off else top
                ratio = (scales[page] / now)[..., None] if now.dim() else scales[page] / now
                if off:
                    rows[:off] = (rows[:off] * ratio).float().to(torch.float8_e4m3fn).double()
                unit = now[..., None] if now.dim() else now
                rows[off:off + n] = (mine / unit).float().to(torch.float8_e4m3fn).double()
                scales[page] = now
                at, p = at + n, p + n
        out[name], out[name + "_scale"] = pool, scales
    return out


def exact(case, seed):
    # logits in 64 bits, a head at a time: too long beyond the largest listed prompt
    if case["op"] in ("prompt", "tree") and _pairs(case) * case["hq"] > 14_000_000_000:
        return None
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    hq, hkv = case["hq"], case["hkv"]
    G = hq // hkv
    o = torch.zeros(st["tokens"], hq, DIM, dtype=torch.float64, device="cuda")
    lse = torch.full((st["tokens"], hq), -math.inf, dtype=torch.float64, device="cuda")
    starts_q, starts_k = st["cu_q"].tolist(), st["cu_k"].tolist()
    for s, (ql, kl) in enumerate(zip(st["q_lens"], st["kv_lens"])):
        if ql == 0:
            continue
        if case["cache"] == "packed":
            rows = torch.arange(starts_k[s], starts_k[s] + kl, device="cuda")
        else:
            rows = (st["table"][s, :_blocks(kl)].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda"))
            rows = rows.reshape(-1)[:kl]
        step = max(1, 300_000_000 // (G * kl))
        for g in range(hkv):
            heads = slice(g * G, (g + 1) * G)
            if case["cache"] == "fp8":
                keys, vals = (st[n][rows, g].view(torch.float8_e4m3fn).double()
                              * st[n + "_scale"].double()[rows // PAGE, g][:, None] for n in ("k", "v"))
            else:
                keys, vals = st["k"][rows, g].double(), st["v"][rows, g].double()
            for a in range(0, ql, step):
                b = min(ql, a + step)
                top = kl if case["op"] == "tree" else kl - ql + b
                mine = slice(starts_q[s] + a, starts_q[s] + b)
                logits = torch.einsum("thd,jd->thj", st["q"][mine, heads].double(), keys[:top]) / math.sqrt(DIM)
                if case["op"] == "tree":
                    bits = st["visible"][mine]
                    hidden = torch.zeros(b - a, top, dtype=torch.bool, device="cuda")
                    for d in range(ql):
                        hidden[:, kl - ql + d] = ((bits[:, d // 32] >> (d % 32)) & 1) == 0
                else:
                    last = kl - ql + torch.arange(a, b, device="cuda")
                    hidden = torch.arange(top, device="cuda")[None, :] > last[:, None]
                logits.masked_fill_(hidden[:, None, :], -math.inf)
                lse[mine, heads] = torch.logsumexp(logits, dim=-1)
                o[mine, heads] = torch.einsum("thj,jd->thd", torch.softmax(logits, dim=-1), vals[:top])
    return {"o": o, "lse": lse}
