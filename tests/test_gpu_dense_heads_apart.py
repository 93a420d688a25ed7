"""GPU: the heads of a group do not touch one another's results, whatever one head's query holds.

A batch over enough KV heads leaves each CTA a whole sequence, so that every CTA has several units of keys: the two
warpgroups of a large group's CTA (units in turn), the teams of a small one's."""
import math

import pytest
import torch

from paged_reference import DIM, PAGE, blocks, dense_reference, quantize_pages, rows_of
from test_gpu_dense_decode import Batch

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


def one_run_heads(group):
    """KV heads that leave the batch one run (two CTAs an SM run groups of up to 16 heads, one CTA the others)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sms * (2 if group <= 16 else 1) // 2 + 1


def batch(msa, lens, group, hkv, fp8, damp):
    """A batch whose dimension 0 is free: queries 0 there, keys 2 in the slots that `damp` names."""
    b = Batch(msa, lens, group * hkv, hkv, False, False, seed=group)
    b.q[:, :, 0] = 0
    for s, n in enumerate(lens):
        slot = torch.arange(n)
        b.k[rows_of(b.host_table, s, n).cuda(), :, 0] = (2.0 * damp(slot)).to(torch.bfloat16).cuda()[:, None]
    if fp8:
        b.k, b.v, b.fp8 = b.k.nan_to_num(0.0), b.v.nan_to_num(0.0), True
        b.k, b.ks = quantize_pages(b.k)
        b.v, b.vs = quantize_pages(b.v)
    return b


@pytest.mark.parametrize("what", ["nan", "no key", "no even unit", "no odd unit"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [16, 24, 40, 64, 128])
def test_one_heads_query(msa, group, fp8, what):
    """One head's query is NaN, or its logits overflow to -inf at every key, or at every other unit of 128 keys."""
    hkv = one_run_heads(group)
    lens = [700, 130, 129]
    damp = {"nan": lambda j: j * 0, "no key": lambda j: j * 0 + 1, "no even unit": lambda j: 1 - (j // 128) % 2,
            "no odd unit": lambda j: (j // 128) % 2}[what]
    b = batch(msa, lens, group, hkv, fp8, damp)
    clean_o, clean_lse = b.call(msa)
    hurt = [(0, 5), (1, 0), (2, group - 1)]  # (sequence, head of the group), of every KV head
    view = lambda t: t.view(len(lens), hkv, group, -1)
    others = torch.ones(len(lens), hkv, group, dtype=torch.bool)
    for s, h in hurt:
        others[s, :, h] = False
        if what == "nan":
            view(b.q)[s, :, h, 77] = math.nan
        else:  # times a key's 2 (or its code): past fp32
            view(b.q)[s, :, h, 0] = -3e38
    o, lse = b.call(msa)
    others = others.cuda()
    assert torch.equal(view(o)[others], view(clean_o)[others])
    assert torch.equal(view(lse)[others], view(clean_lse)[others])
    for s, h in hurt:
        got_o, got_lse = view(o)[s, :, h], view(lse)[s, :, h, 0]
        if what == "nan":
            assert got_o.isnan().all() and got_lse.isnan().all()
            continue
        if fp8 and group <= 32:
            # the query's other dimensions are 2^-24 of its largest and vanish beside it, and the product is scaled before
            # it passes fp32: a finite logit, of 10^37 and more
            continue
        assert torch.isfinite(got_o).all()
        left = [i for i in range(blocks(lens[s])) if damp(torch.tensor(128 * i)) == 0]  # its pages that count
        if not left:
            assert (got_o == 0).all() and (got_lse == -math.inf).all()
            continue
        n = sum(min(PAGE, lens[s] - PAGE * i) for i in left)
        q = view(b.q)[s, :, h].clone()[None]
        q[..., 0] = 0
        ref = dense_reference([n], b.host_table[s:s + 1, left], q, b.k, b.v, b.ks, b.vs)
        assert ((got_o.double() - ref[0][0]).abs() <= ref[3][0]).all()
        assert ((got_lse.double() - ref[1][0]).abs() <= ref[4][0]).all()
