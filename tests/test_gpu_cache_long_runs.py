"""New rows of whole pages and of many thousand tokens at once, bf16 and E4M3: the codes and scales of long runs, over every size
of a CTA's share of the tokens and behind rows that are there already.  All exact (see test_gpu_cache_fill).
"""
import pytest
import torch

from paged_reference import PAGE, quantize_pages
from test_gpu_cache_fill import append_fp8_reference, msa, slots_of  # noqa: F401

pytestmark = pytest.mark.gpu

# up to 1,024, 2,048, 4,096, 8,192 and more tokens a call; runs of 17 to 128 tokens, alone in a page or behind others
BATCHES = [([0], [128]), ([5], [300]), ([60], [60]), ([0] * 9, [100] * 9), ([17, 111, 40], [111, 17, 88]), ([100], [1500]), ([0, 77], [1000, 900]),
           ([3, 0, 250], [1000, 0, 2500]), ([64] * 3, [1700] * 3), ([0, 1, 2], [7000, 12001, 999]), ([31 + i % 90 for i in range(300)], [30 + i % 41 for i in range(300)])]


def without_ends(slots, gen):
    """Some tokens without a row: the first or last ones of a page's run, so that no page comes twice."""
    out = slots[:]
    for i in torch.randint(0, len(slots), (6,), generator=gen).tolist():
        j = i
        while j + 1 < len(slots) and slots[j + 1] // PAGE == slots[i] // PAGE:
            j += 1
        k = i
        while k > 0 and slots[k - 1] // PAGE == slots[i] // PAGE:
            k -= 1
        out[j] = -1
        if j - k > 20:
            out[k] = -1
    return out


@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("hkv,index,gain,holes", [(1, False, 0.2, False), (4, True, 5.0, True), (3, True, 0.2, True)])
def test_long_runs_fp8(msa, batch, hkv, index, gain, holes):
    lengths, new = BATCHES[batch]
    gen = torch.Generator().manual_seed(batch)
    slots, pages = slots_of(lengths, new, gen)
    if holes:
        slots = without_ends(slots, gen)
    N = len(slots)
    wide = (torch.randn(N, (2 * hkv + 1) * 128, generator=gen) * gain).to(torch.bfloat16).cuda()
    heads = [hkv, hkv] + ([1] if index else [])
    rows = [wide[:, :hkv * 128].view(N, hkv, 128), wide[:, hkv * 128:2 * hkv * 128].view(N, hkv, 128), wide[:, -128:].unsqueeze(1)]
    caches, scales = [], []
    for h in heads:
        c, s = quantize_pages(torch.randn(pages * PAGE, h, 128, generator=gen).to(torch.bfloat16))
        caches.append(c.cuda())
        scales.append(s.cuda())
    more = dict(k_idx=rows[2][:, 0], k_idx8_cache=caches[2][:, 0], k_idx_scale=scales[2][:, 0]) if index else {}
    want = [append_fp8_reference(x, slots, c, s) for x, c, s in zip(rows, caches, scales)]
    ws = msa.append_workspace(pages)
    msa.msa_append_paged_fp8(rows[0], rows[1], torch.tensor(slots, dtype=torch.int64, device="cuda"), caches[0], caches[1], scales[0],
                             scales[1], ws=ws, **more)
    assert msa.msa_read_device_status(ws) == 0
    for (wc, wsc), c, s in zip(want, caches, scales):
        assert torch.equal(wsc, s.cpu())
        assert torch.equal(wc, c.cpu())


def test_a_page_that_comes_twice(msa):
    """A token without a row in the middle of a page's run, and a page's tokens apart: both raise the flag."""
    for slots in ([0, 1, -1, 3], [0, PAGE, 1], list(range(40)) + [-1] + list(range(41, 128))):
        x = torch.randn(len(slots), 2, 128, device="cuda").to(torch.bfloat16)
        c = [torch.zeros(2 * PAGE, 2, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.ones(2, 2, device="cuda") for _ in range(2)]
        ws = msa.append_workspace(2)
        msa.msa_append_paged_fp8(x, x, torch.tensor(slots, device="cuda"), *c, *s, ws=ws)
        assert msa.msa_read_device_status(ws) == msa.DEVICE_BAD_INDEX


@pytest.mark.parametrize("hkv,d_idx", [(4, 128), (7, 64)])
def test_many_bf16_rows(msa, hkv, d_idx):
    lengths, new = [0, 100, 5], [20000, 9000, 2777]
    gen = torch.Generator().manual_seed(hkv)
    slots, pages = slots_of(lengths, new, gen)
    N = len(slots)
    at = torch.tensor(slots, dtype=torch.int64, device="cuda")
    at[torch.randint(0, N, (50,), generator=gen).cuda()] = -1
    wide = torch.randn(N, 2 * hkv * 128 + d_idx, generator=gen).to(torch.bfloat16).cuda()
    rows = [wide[:, :hkv * 128].view(N, hkv, 128), wide[:, hkv * 128:2 * hkv * 128].view(N, hkv, 128), wide[:, -d_idx:]]
    caches = [torch.randn(pages * PAGE, *x.shape[1:], generator=gen).to(torch.bfloat16).cuda() for x in rows]
    want = [c.clone() for c in caches]
    for w, x in zip(want, rows):
        w[at[at >= 0]] = x[at >= 0]
    msa.msa_append_paged(rows[0], rows[1], at, caches[0], caches[1], k_idx=rows[2], k_idx_cache=caches[2])
    for w, c in zip(want, caches):
        assert torch.equal(w, c)
