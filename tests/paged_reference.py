"""64-bit references of the dense paged decode attention, the eviction and the norm, and paged caches to test them on.

Error bounds (u = 2^-24, half a step of fp32 at 1; a bf16 rounding is off by at most 2^-8 of the value, fp16 2^-11):
a logit is an fp32 sum of 128 exact products, off by at most g = 130 * 2u * scale * sum_d |q_d k_d| (the factor 2
because tensor cores may truncate); a weight exp(s - lse) is then off by at most its 2 g + (n + 16) * 2u + 2u (|s| + |lse|)
(the sum over n keys, exp2, and the logits' and lse's own roundings); the weights' rounding for the product with V adds
2^-16 (bf16 value plus bf16 rest) or 2^-11 (fp16, fp8 caches); the sum over keys (n + 16) * 2u of sum_j p_j |v_j|.
"""
import math

import torch

PAGE, DIM = 128, 128
U2 = 2.0 ** -23


def blocks(n):
    return -(-n // PAGE)


def make_tables(lens, gen, spare=3, width=None):
    """Random page numbers for each sequence's blocks, -1 behind them; returns (table, number of pages)."""
    need = sum(blocks(n) for n in lens)
    pages = torch.randperm(need + spare, generator=gen).to(torch.int32)
    table = torch.full((len(lens), width or max(1, max(blocks(n) for n in lens))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        table[s, :blocks(n)] = pages[at:at + blocks(n)]
        at += blocks(n)
    return table, need + spare


def rows_of(table, s, n):
    """Cache rows of slots 0..n-1 of sequence s (host table)."""
    at = table[s, :blocks(n)].long()[:, None] * PAGE + torch.arange(PAGE)
    return at.reshape(-1)[:n]


def quantize_pages(x):
    """bf16 [pages * 128, heads, 128] -> (uint8 codes, scales [pages, heads])."""
    f = x.view(-1, PAGE, x.shape[1], DIM).float()
    amax = f.abs().amax(dim=(1, 3))
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (f / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape), scale


def values(cache, scale, rows, g):
    """The 64-bit values of some rows of one head."""
    x = cache[rows, g]
    if scale is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * scale.double()[rows // PAGE, g][:, None]


def dense_reference(lens, table, q, k, v, k_scale=None, v_scale=None, scale=None):
    """Per sequence and head in 64 bits: o, lse, the keys' weights per KV head (list of [hkv, n]) and the bounds
    (o_tol, lse_tol, list of weight tolerances), on q's device."""
    S, hq, _ = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    scale = scale if scale else DIM ** -0.5
    dev = q.device
    o = torch.zeros(S, hq, DIM, dtype=torch.float64, device=dev)
    o_tol = torch.zeros_like(o)
    lse = torch.full((S, hq), -math.inf, dtype=torch.float64, device=dev)
    lse_tol = torch.zeros_like(lse)
    w, w_tol = [], []
    table = table.cpu()
    for s, n in enumerate(lens):
        ws = torch.zeros(hkv, n, dtype=torch.float64, device=dev)
        wt = torch.zeros_like(ws)
        if n:
            rows = rows_of(table, s, n).to(dev)
            for g in range(hkv):
                hs = slice(g * G, (g + 1) * G)
                kd, vd, qd = values(k, k_scale, rows, g), values(v, v_scale, rows, g), q[s, hs].double()
                logits = qd @ kd.T * scale
                err = 130 * U2 * scale * (qd.abs() @ kd.abs().T)            # per logit
                top = torch.logsumexp(logits, dim=1)
                p = torch.exp(logits - top[:, None])
                gmax = (p * err).sum(dim=1) + U2                            # lse moves by the weighted mean error
                lse[s, hs] = top
                lse_tol[s, hs] = gmax + (n + 16) * U2 + 4 * U2 * (top.abs() + logits.abs().amax(dim=1))
                rel = err + lse_tol[s, hs][:, None] + 4 * U2 * logits.abs()
                ws[g] = p.sum(dim=0)
                wt[g] = (p * rel).sum(dim=0) + G * U2 * ws[g]
                o[s, hs] = p @ vd
                spread = (p * (rel + (2.0 ** -11 if k_scale is not None else 2.0 ** -16))) @ vd.abs()
                o_tol[s, hs] = 2.0 ** -8 * o[s, hs].abs() + spread + (n + 16) * U2 * (p @ vd.abs()) + 2.0 ** -120
                if k_scale is not None:  # fp16 weights below 2^-38 of the largest vanish, queries below 2^-24 of theirs
                    o_tol[s, hs] += 2.0 ** -24 * n * (p.amax(dim=1)[:, None] * vd.abs().amax(dim=0)[None, :])
        w.append(ws)
        w_tol.append(wt)
    return o, lse, w, o_tol, lse_tol, w_tol


def evict_reference(lens, weight, budget, recent):
    """Kept slots (list of [hkv] lists of ascending slot lists), on the host."""
    out = []
    wt = weight.cpu()
    for s, n in enumerate(lens):
        heads = []
        for g in range(weight.shape[1]):
            if n <= budget:
                heads.append(list(range(n)))
                continue
            free, take = n - recent, budget - recent
            key = [(-math.inf if math.isnan(x) else x, not math.isnan(x)) for x in wt[s, g, :free].tolist()]
            # by weight downward, NaN last (below -inf), equal weights by slot upward
            order = sorted(range(free), key=lambda j: (-key[j][0], not key[j][1], j))[:take]
            heads.append(sorted(order) + list(range(free, n)))
        out.append(heads)
    return out
