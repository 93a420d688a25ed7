"""Measured cases of the decode-step operators beside the sparse attention: dense attention of one new token over a
paged cache (bf16 or E4M3 pages, optionally accumulating each key's attention weight), eviction from that cache by the
accumulated weight, and the residual sum with its root-mean-square norm (bf16 or E4M3 output).

``own`` selects the framework's kernels; otherwise ``run`` computes the same results with elementary torch operations
in 32 bits, rounded once at the end.  ``exact`` gives the results in 64 bits.
"""
import math

import torch

own = False

PAGE = 128        # tokens of a cache page
DIM = 128         # head dimension
E4M3_MAX = 448.0


def listed():
    return [
        # one user's first tokens: the latency of a decode step's attention
        {"name": "dense_1x333", "op": "dense", "seqs": 1, "max_len": 333, "ragged": False, "hq": 64, "hkv": 4,
         "fp8": False, "weight": False},
        # a serving batch of mixed lengths (an empty slot among them) whose cache is going to be evicted from
        {"name": "dense_32_ragged_weight", "op": "dense", "seqs": 32, "max_len": 16384, "ragged": True, "hq": 64,
         "hkv": 4, "fp8": False, "weight": True},
        # one long context
        {"name": "dense_1x1m", "op": "dense", "seqs": 1, "max_len": 1048576, "ragged": False, "hq": 64, "hkv": 4,
         "fp8": False, "weight": False},
        # a serving batch over an 8-bit cache
        {"name": "dense_24_fp8", "op": "dense", "seqs": 24, "max_len": 65521, "ragged": True, "hq": 64, "hkv": 4,
         "fp8": True, "weight": False},
        # one KV head for all query heads
        {"name": "dense_8_mqa", "op": "dense", "seqs": 8, "max_len": 50000, "ragged": True, "hq": 128, "hkv": 1,
         "fp8": False, "weight": False},
        # many short sequences, a group of five heads
        {"name": "dense_200_short", "op": "dense", "seqs": 200, "max_len": 700, "ragged": True, "hq": 40, "hkv": 8,
         "fp8": False, "weight": False},
        # one user's cache trimmed at a small budget: latency
        {"name": "evict_1x700", "op": "evict", "seqs": 1, "max_len": 700, "ragged": False, "hq": 64, "hkv": 4,
         "fp8": False, "budget": 512, "recent": 64},
        # a batch in 8 bits, some of whose sequences are under the budget
        {"name": "evict_16_fp8", "op": "evict", "seqs": 16, "max_len": 9001, "ragged": True, "hq": 64, "hkv": 4,
         "fp8": True, "budget": 4096, "recent": 333},
        # long caches halved
        {"name": "evict_12x64k", "op": "evict", "seqs": 12, "max_len": 65536, "ragged": False, "hq": 64, "hkv": 4,
         "fp8": False, "budget": 32768, "recent": 1024},
        # a decode batch between two layers
        {"name": "norm_7x4096", "op": "norm", "rows": 7, "width": 4096, "fp8": False},
        # a short prefill into an 8-bit projection
        {"name": "norm_1001x5120_fp8", "op": "norm", "rows": 1001, "width": 5120, "fp8": True},
        # a long prefill
        {"name": "norm_16384x8192", "op": "norm", "rows": 16384, "width": 8192, "fp8": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("dense", "dense", "evict", "norm"))
    if op == "norm":
        width = _spread(rng, 64, 16384)
        if rng.random() < 0.7:
            width = -(-width // 8) * 8
        rows = _spread(rng, 1, max(1, min(32768, 100_000_000 // width)))
        return {"op": op, "rows": rows, "width": width, "fp8": rng.random() < 0.5}
    hq, hkv = rng.choice(((64, 4), (64, 4), (32, 8), (40, 8), (128, 1), (12, 12), (28, 4), (96, 2)))
    seqs = _spread(rng, 1, 128)
    max_len = _spread(rng, 1, max(1, min(400_000, 3_000_000 // (seqs * hkv))))
    case = {"op": op, "seqs": seqs, "max_len": max_len, "ragged": rng.random() < 0.7, "hq": hq, "hkv": hkv,
            "fp8": rng.random() < 0.4}
    if op == "dense":
        case["weight"] = rng.random() < 0.4
    else:
        case["budget"] = max(1, int(max_len * rng.uniform(0.2, 0.9)))
        case["recent"] = int(case["budget"] * rng.uniform(0.0, 0.5))
    return case


def _lengths(case):
    """Cached tokens of each sequence, by the case alone; a ragged batch of eight or more has empty slots."""
    n, top = case["seqs"], case["max_len"]
    if not case["ragged"]:
        return [top] * n
    out = [1 + int((top - 1) * (((i + 1) * 0.6180339887) % 1.0)) for i in range(n)]
    out[0] = top
    return [0 if i % 8 == 5 else v for i, v in enumerate(out)]


def _blocks(n):
    return -(-n // PAGE)


def _tables(pages, lens, width):
    """A block table whose pages are drawn from `pages` in random order, -1 past each sequence's last block."""
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        b = _blocks(n)
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, dtype=dtype, device="cuda", generator=gen)

    st = dict(case)
    if case["op"] == "norm":
        st["x"] = normal(case["rows"], case["width"])
        st["residual"] = normal(case["rows"], case["width"]) * 4   # a residual stream outgrows a layer's output
        st["gamma"] = 1 + normal(case["width"]) / 8
        return st
    lens = _lengths(case)
    S, hq, hkv = case["seqs"], case["hq"], case["hkv"]
    kept = [min(n, case["budget"]) for n in lens] if case["op"] == "evict" else []
    st["lens"] = lens
    st["max_len"] = max(lens)
    used, new = sum(map(_blocks, lens)), sum(map(_blocks, kept))
    n_pages = used + new + 3   # a few pages belong to nobody
    pages = torch.randperm(n_pages, generator=host).to(torch.int32)
    width = max(1, _blocks(max(lens)))
    st["table"] = _tables(pages, lens, width)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st["cu_k"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["cu_q"] = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    st["k"], st["v"] = normal(n_pages * PAGE, hkv, DIM), normal(n_pages * PAGE, hkv, DIM)
    if case["fp8"]:
        st["k"], st["k_scale"] = _quantized(st["k"])
        st["v"], st["v_scale"] = _quantized(st["v"])
    if case["op"] == "dense":
        st["q"] = normal(S, hq, DIM) * 2
        if case["weight"]:
            st["acc"] = normal(S, hkv, max(lens), dtype=torch.float32).exp() / 64
    else:
        # weights of a cache in use: spread over orders of magnitude, some keys never attended to
        st["acc"] = (normal(S, hkv, max(lens), dtype=torch.float32) * 2).exp()
        st["acc"] *= torch.rand(st["acc"].shape, device="cuda", generator=gen) > 0.1
        st["new_table"] = _tables(pages[used:], kept, max(1, _blocks(max(kept))))
    if own:
        # what a serving loop keeps from step to step: the batch's sizes and a workspace; no work on the data
        import block_sparse_attention_05_gb300 as msa
        st["problem"] = msa.Problem(st["cu_q"], st["cu_k"], S, cu[-1], 1, max(lens), hq, hkv, 128, 16)
        if case["op"] == "evict":
            st["ws"] = msa.evict_workspace(st["problem"], case["budget"], n_pages)
        else:
            st["ws"] = msa.workspace(st["problem"], msa.Op.DENSE_ATTN_DECODE_WEIGHT if case["weight"]
                                     else msa.Op.DENSE_ATTN_DECODE)
    return st


def _rows(st, table, n):
    """Cache rows of slots 0..n-1 of each sequence through a block table ([S, n], 0 where there is none)."""
    pos = torch.arange(n, device="cuda")
    return (table[:, pos // PAGE].long() * PAGE + pos % PAGE).clamp_(min=0)


def _valid(st, n):
    lens = st["cu_k"][1:] - st["cu_k"][:-1]
    return torch.arange(n, device="cuda")[None, :] < lens[:, None]


def _plain_dense(st):
    S, hq, hkv, n = st["seqs"], st["hq"], st["hkv"], st["max_len"]
    rows, ok = _rows(st, st["table"], n), _valid(st, n)
    k, v = st["k"][rows], st["v"][rows]
    if st["fp8"]:
        k = k.view(torch.float8_e4m3fn).float() * st["k_scale"][rows // PAGE][..., None]
        v = v.view(torch.float8_e4m3fn).float() * st["v_scale"][rows // PAGE][..., None]
    else:
        k, v = k.float(), v.float()
    q = st["q"].float().view(S, hkv, hq // hkv, DIM)
    s = (q @ k.permute(0, 2, 3, 1)) * (DIM ** -0.5)
    s = s.masked_fill(~ok[:, None, None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = {"o": (p @ v.permute(0, 2, 1, 3)).to(torch.bfloat16).view(S, hq, DIM),
           "lse": (m + torch.log(total)).view(S, hq)}
    if st["weight"]:
        st["acc"] += p.sum(dim=2)
        out["weight"] = st["acc"]
    return out


def _plain_evict(st):
    S, hkv, n = st["seqs"], st["hkv"], st["max_len"]
    budget = st["budget"]
    lens = (st["cu_k"][1:] - st["cu_k"][:-1])
    slot = torch.arange(n, device="cuda")
    ok = _valid(st, n)
    late = slot[None, :] >= (lens - st["recent"])[:, None]
    key = st["acc"].masked_fill(late[:, None, :], math.inf).masked_fill(~ok[:, None, :], -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    new_len = lens.clamp(max=budget)
    width = order.shape[-1]
    there = torch.arange(width, device="cuda")[None, :] < new_len[:, None]                  # [S, width]
    slots = torch.sort(order.masked_fill(~there[:, None, :], n), dim=-1).values             # ascending, none last
    kept = torch.full((S, hkv, budget), -1, dtype=torch.int32, device="cuda")
    kept[..., :width] = slots.masked_fill(~there[:, None, :], -1)
    slots = slots.clamp(max=n - 1)
    src = torch.gather(_rows(st, st["table"], n)[:, None, :].expand(S, hkv, n), 2, slots)   # [S, hkv, width]
    dst = _rows(st, st["new_table"], width)
    head = torch.arange(hkv, device="cuda")[None, :, None].expand(S, hkv, width)
    to = dst[:, None, :].expand(S, hkv, width)
    mask = there[:, None, :].expand(S, hkv, width)
    weight = torch.gather(st["acc"], 2, slots).masked_fill(~mask, 0.0)
    cu = torch.zeros_like(st["cu_k"])
    cu[1:] = torch.cumsum(new_len, 0)
    for name in ("k", "v"):
        if st["fp8"]:
            val = st[name][src, head].view(torch.float8_e4m3fn).float()
            val *= st[name + "_scale"][src // PAGE, head][..., None]
            pad = _blocks(width) * PAGE - width
            amax = torch.nn.functional.pad((val.abs().amax(-1)).masked_fill(~mask, 0.0), (0, pad))
            amax = amax.view(S, hkv, -1, PAGE).amax(-1)                                     # per new page
            scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
            each = scale.repeat_interleave(PAGE, dim=2)[..., :width]
            codes = (val / each[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            st[name + "_scale"][(to // PAGE)[mask], head[mask]] = each[mask]
            st[name][to[mask], head[mask]] = codes[mask]
        else:
            st[name][to[mask], head[mask]] = st[name][src[mask], head[mask]]
    return kept, weight, cu


def _evicted(st, kept, weight, cu):
    out = {"kept": kept, "weight": weight, "cu_k": cu}
    for name in ("k", "v"):
        if st["fp8"]:
            out[name], out[name + "_scale"] = st[name].view(torch.float8_e4m3fn), st[name + "_scale"]
        else:
            out[name] = st[name]
    return out


def _plain_norm(st):
    h = st["x"].float() + st["residual"].float()
    y = h / torch.sqrt((h * h).mean(dim=-1, keepdim=True) + 1e-6) * st["gamma"].float()
    if not st["fp8"]:
        return {"sum": h.to(torch.bfloat16), "y": y.to(torch.bfloat16)}
    amax = y.abs().amax(dim=-1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return {"sum": h.to(torch.bfloat16), "y": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}


def run(state):
    st = state
    if not own:
        if st["op"] == "dense":
            return _plain_dense(st)
        if st["op"] == "evict":
            return _evicted(st, *_plain_evict(st))
        return _plain_norm(st)
    import block_sparse_attention_05_gb300 as msa
    if st["op"] == "norm":
        if st["fp8"]:
            total, y, scale = msa.msa_add_rms_norm_fp8(st["x"], st["gamma"], residual=st["residual"])
            return {"sum": total, "y": y.view(torch.float8_e4m3fn), "scale": scale}
        total, y = msa.msa_add_rms_norm(st["x"], st["gamma"], residual=st["residual"])
        return {"sum": total, "y": y}
    if st["op"] == "dense":
        if st["fp8"]:
            o, lse = msa.msa_dense_attn_decode_paged_fp8(st["problem"], st["q"], st["k"], st["v"], st["k_scale"],
                                                         st["v_scale"], st["table"], weight=st.get("acc"), ws=st["ws"])
        else:
            o, lse = msa.msa_dense_attn_decode_paged(st["problem"], st["q"], st["k"], st["v"], st["table"],
                                                     weight=st.get("acc"), ws=st["ws"])
        return {"o": o, "lse": lse, "weight": st["acc"]} if st["weight"] else {"o": o, "lse": lse}
    width = min(st["budget"], st["max_len"])
    weight = torch.zeros((st["seqs"], st["hkv"], width), dtype=torch.float32, device="cuda")
    if st["fp8"]:
        kept, weight, cu = msa.msa_evict_paged_fp8(st["problem"], st["k"], st["v"], st["k_scale"], st["v_scale"],
                                                   st["table"], st["acc"], st["new_table"], budget=st["budget"],
                                                   recent=st["recent"], new_weight=weight, ws=st["ws"])
    else:
        kept, weight, cu = msa.msa_evict_paged(st["problem"], st["k"], st["v"], st["table"], st["acc"],
                                               st["new_table"], budget=st["budget"], recent=st["recent"],
                                               new_weight=weight, ws=st["ws"])
    return _evicted(st, kept, weight, cu)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        out = n + 4 * case["rows"] if case["fp8"] else 2 * n
        return {"bytes": 6 * n + out + 2 * case["width"], "flops": 6 * n}
    lens, hq, hkv = _lengths(case), case["hq"], case["hkv"]
    total = sum(lens)
    row = 2 * DIM * (1 if case["fp8"] else 2)           # K and V of a key and KV head
    scales = 8 * hkv * sum(map(_blocks, lens)) if case["fp8"] else 0
    table = 4 * sum(map(_blocks, lens))
    if case["op"] == "dense":
        size = total * hkv * row + scales + table + len(lens) * hq * (4 * DIM + 4)
        if case["weight"]:
            size += 8 * total * hkv
        return {"bytes": size, "flops": 4 * DIM * hq * total}
    kept = [min(n, case["budget"]) for n in lens]
    size = 4 * total * hkv + 2 * sum(kept) * hkv * row + 8 * sum(kept) * hkv + 2 * scales + table
    return {"bytes": size, "flops": total * hkv}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double() + st["residual"].double()
        y = torch.einsum("rw,w->rw", h, st["gamma"].double())
        y = y * (h.pow(2).sum(dim=1).div(case["width"]) + 1e-6).pow(-0.5)[:, None]
        if not case["fp8"]:
            return {"sum": h, "y": y}
        scale = y.abs().max(dim=1).values / E4M3_MAX
        return {"sum": h, "y": (y / scale[:, None]).float().to(torch.float8_e4m3fn).double(), "scale": scale}
    lens, hq, hkv = st["lens"], case["hq"], case["hkv"]

    def values(name, rows, g):
        x = st[name][rows, g]
        if not case["fp8"]:
            return x.double()
        return x.view(torch.float8_e4m3fn).double() * st[name + "_scale"].double()[rows // PAGE, g][:, None]

    def rows_of(table, s, n):
        at = table[s, :_blocks(n)].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")
        return at.reshape(-1)[:n]

    if case["op"] == "dense":
        G = hq // hkv
        o = torch.zeros(case["seqs"], hq, DIM, dtype=torch.float64, device="cuda")
        lse = torch.full((case["seqs"], hq), -math.inf, dtype=torch.float64, device="cuda")
        weight = st["acc"].double() if case["weight"] else None
        for s, n in enumerate(lens):
            if n == 0:
                continue
            rows = rows_of(st["table"], s, n)
            for g in range(hkv):
                heads = slice(g * G, (g + 1) * G)
                logits = st["q"][s, heads].double() @ values("k", rows, g).T / math.sqrt(DIM)
                lse[s, heads] = torch.logsumexp(logits, dim=1)
                p = torch.softmax(logits, dim=1)
                o[s, heads] = p @ values("v", rows, g)
                if weight is not None:
                    weight[s, g, :n] += p.sum(dim=0)
        return {"o": o, "lse": lse, "weight": weight} if case["weight"] else {"o": o, "lse": lse}
    budget, recent = case["budget"], case["recent"]
    kept = torch.full((case["seqs"], hkv, budget), -1, dtype=torch.int32, device="cuda")
    weight = torch.zeros(case["seqs"], hkv, min(budget, max(lens)), dtype=torch.float64, device="cuda")
    ends = [0]
    pools, scales = {}, {}
    for name in ("k", "v"):
        pools[name] = st[name].view(torch.float8_e4m3fn).double() if case["fp8"] else st[name].double()
        if case["fp8"]:
            scales[name] = st[name + "_scale"].double()
    for s, n in enumerate(lens):
        m = min(n, budget)
        ends.append(ends[-1] + m)
        if m == 0:
            continue
        src, dst = rows_of(st["table"], s, n), rows_of(st["new_table"], s, m)
        for g in range(hkv):
            w = st["acc"][s, g, :n].double()
            free = min(n, max(0, n - recent)) if n > budget else 0
            take = m - (n - free)
            # by weight downward, equal weights by slot upward
            first = w[:free].cpu().numpy()
            order = sorted(range(free), key=lambda j: (-first[j], j))[:take] if free < 4096 else None
            if order is None:
                edge = torch.topk(w[:free], take).values[-1] if take else None
                above = (w[:free] > edge) if take else torch.zeros(free, dtype=torch.bool, device="cuda")
                same = torch.nonzero(w[:free] == edge).flatten()[:take - int(above.sum())] if take else []
                keep = above.clone()
                keep[same] = True
                early = torch.nonzero(keep).flatten()
            else:
                early = torch.tensor(sorted(order), dtype=torch.int64, device="cuda")
            slots = torch.cat([early, torch.arange(free, n, device="cuda")])
            kept[s, g, :m] = slots.to(torch.int32)
            weight[s, g, :m] = w[slots]
            for name in ("k", "v"):
                val = values(name, src[slots], g)
                if not case["fp8"]:
                    pools[name][dst, g] = val
                    continue
                top = torch.zeros(_blocks(m), dtype=torch.float64, device="cuda")
                page = torch.arange(m, device="cuda") // PAGE
                top.scatter_reduce_(0, page, val.abs().amax(dim=1), "amax")
                scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
                scales[name][dst[::PAGE] // PAGE, g] = scale
                pools[name][dst, g] = (val / scale[page][:, None]).float().to(torch.float8_e4m3fn).double()
    out = {"kept": kept, "weight": weight, "cu_k": torch.tensor(ends, dtype=torch.int32, device="cuda")}
    for name in ("k", "v"):
        out[name] = pools[name]
        if case["fp8"]:
            out[name + "_scale"] = scales[name]
    return out
