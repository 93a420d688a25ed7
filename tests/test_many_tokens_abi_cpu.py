"""Refusals of the prompt and tree attention, the table extension and the cache writes, on the host (pointers are never
dereferenced: every call here returns before any CUDA call, or with "no usable device" where all arguments are fine)."""
import ctypes
import math

import pytest
import torch

FAKE = 0x10000
NONE = -6  # no usable device: everything was accepted


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_05_gb300 as m
    return m


def batch(msa, **kw):
    p = dict(num_seqs=4, cu_seqlens_q=FAKE, cu_seqlens_k=FAKE, total_q=400, total_k=1024, max_seqlen_q=100,
             max_seqlen_k=1024, num_q_heads=64, num_kv_heads=4, head_dim=128, index_dim=128, block_size=128, topk=16,
             softmax_scale=0.0)
    p.update(kw)
    return msa.MsaProblem(**p)


def accepted(status):
    """Accepted on the host: without a GPU the call stops at the device check."""
    return status == NONE


CALLS = {
    "packed": lambda lib, p, a: lib.msa_dense_attn_prefill(p, a["q"], a["k"], a["v"], a["o"], a["lse"], a["ws"], a["n"], None),
    "paged": lambda lib, p, a: lib.msa_dense_attn_prefill_paged(
        p, a["q"], a["k"], a["v"], a["bt"], a["mb"], a["pages"], a["o"], a["lse"], a["ws"], a["n"], None),
    "fp8": lambda lib, p, a: lib.msa_dense_attn_prefill_paged_fp8(
        p, a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["mb"], a["pages"], a["o"], a["lse"], a["ws"], a["n"], None),
    "tree": lambda lib, p, a: lib.msa_tree_attn_paged(
        p, a["q"], a["k"], a["v"], a["bt"], a["mb"], a["pages"], a["vis"], a["words"], a["o"], a["lse"], a["ws"], a["n"], None),
    "tree_fp8": lambda lib, p, a: lib.msa_tree_attn_paged_fp8(
        p, a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["mb"], a["pages"], a["vis"], a["words"], a["o"], a["lse"],
        a["ws"], a["n"], None),
}
FINE = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=8, pages=100, vis=FAKE, words=4, o=FAKE, lse=FAKE,
            ws=FAKE, n=1 << 40)


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=0), -1), (dict(cu_seqlens_q=None), -1), (dict(cu_seqlens_k=None), -1), (dict(total_q=-1), -1),
    (dict(total_k=-1), -1), (dict(max_seqlen_q=401), -1), (dict(max_seqlen_k=1025), -1), (dict(max_seqlen_q=-1), -1),
    (dict(num_q_heads=63), -1), (dict(num_kv_heads=0), -1), (dict(num_q_heads=0), -1), (dict(softmax_scale=math.nan), -1),
    (dict(softmax_scale=math.inf), -1), (dict(softmax_scale=3e38), -1), (dict(head_dim=0), -1), (dict(head_dim=64), -2),
    (dict(block_size=64), -2), (dict(num_q_heads=129, num_kv_heads=1), -2), (dict(num_q_heads=1025, num_kv_heads=1025), -2),
    (dict(num_seqs=(1 << 20) + 1), -2), (dict(total_q=1 << 25), -2),
    (dict(total_k=(1 << 30) + 1, max_seqlen_k=(1 << 30) + 1), -2)])
def test_problems_outside_the_range(msa, name, kw, status):
    p = batch(msa, **kw)
    n = ctypes.c_size_t(0)
    for op in (msa.Op.DENSE_ATTN_PREFILL, msa.Op.TREE_ATTN):
        assert msa._lib.msa_workspace_size(p, int(op), ctypes.byref(n)) == status
    assert CALLS[name](msa._lib, p, FINE) == status


@pytest.mark.parametrize("name", list(CALLS))
def test_attention_refusals(msa, name):
    lib, p = msa._lib, batch(msa)

    def call(problem=p, **kw):
        return CALLS[name](lib, problem, {**FINE, **kw})

    n = ctypes.c_size_t(0)
    assert lib.msa_workspace_size(p, int(msa.Op.TREE_ATTN), ctypes.byref(n)) == 0
    need = n.value
    if not torch.cuda.is_available():
        assert accepted(call()) and accepted(call(n=need))
    uses = {"packed": (), "paged": ("bt",), "fp8": ("bt", "ks", "vs"), "tree": ("bt", "vis"),
            "tree_fp8": ("bt", "ks", "vs", "vis")}[name]
    for arg in ("q", "k", "v", "o", "lse") + uses:
        assert call(**{arg: None}) == -1, arg
        assert call(**{arg: FAKE + 2}) == -3, arg
    for arg in ("q", "k", "v", "o", "lse"):
        assert call(**{arg: FAKE + 8}) == -3, arg
    assert call(ws=None) == -4 and call(n=need - 1) == -4 and call(ws=FAKE + 16) == -3
    if "bt" in uses:
        assert call(mb=7) == -1 and call(pages=0) == -1 and call(pages=1 << 24) == -1
    if "vis" in uses:
        assert call(words=3) == -1 and call(words=0) == -1
        if not torch.cuda.is_available():
            assert accepted(call(words=100))
    if not torch.cuda.is_available():   # a batch without query rows needs no rows
        none = batch(msa, total_q=0, max_seqlen_q=0)
        assert accepted(call(problem=none, q=None, o=None, lse=None, vis=None))


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("kw", [dict(total_q=500, total_k=400, max_seqlen_k=400), dict(total_q=1, total_k=0, max_seqlen_q=1,
                                max_seqlen_k=0), dict(max_seqlen_q=100, max_seqlen_k=99)])
def test_more_queries_than_keys(msa, name, kw):
    p = batch(msa, **kw)
    n = ctypes.c_size_t(0)
    assert msa._lib.msa_workspace_size(p, int(msa.Op.TREE_ATTN), ctypes.byref(n)) == -1
    assert CALLS[name](msa._lib, p, FINE) == -1


def test_any_group(msa):
    n = ctypes.c_size_t(0)
    for hq, hkv in ((1, 1), (5, 1), (128, 1), (35, 7), (1024, 1024), (96, 2)):
        p = batch(msa, num_q_heads=hq, num_kv_heads=hkv, topk=0, index_dim=0)
        assert msa._lib.msa_workspace_size(p, int(msa.Op.DENSE_ATTN_PREFILL), ctypes.byref(n)) == 0
        if not torch.cuda.is_available():
            assert accepted(CALLS["packed"](msa._lib, p, FINE))


def test_extend_refusals(msa):
    lib = msa._lib
    n = ctypes.c_size_t(0)
    assert lib.msa_extend_workspace_size(5, ctypes.byref(n)) == 0
    need = n.value
    assert lib.msa_extend_workspace_size(0, ctypes.byref(n)) == -1 and lib.msa_extend_workspace_size(5, None) == -1
    assert lib.msa_extend_workspace_size((1 << 20) + 1, ctypes.byref(n)) == -2
    fine = dict(S=5, len=FAKE, new=FAKE, cap=9, free=FAKE, nf=7, taken=FAKE, pages=100, bt=FAKE, mb=8, grown=FAKE, q=FAKE,
                k=FAKE, slots=FAKE, pos=FAKE, out=FAKE, ws=FAKE, n=need)

    def call(**kw):
        return lib.msa_extend_block_table(*{**fine, **kw}.values(), None)

    if not torch.cuda.is_available():
        assert accepted(call()) and accepted(call(taken=None, grown=None))
        assert accepted(call(free=None, nf=0)) and accepted(call(cap=0, slots=None, pos=None))
    for arg in ("len", "new", "free", "bt", "q", "k", "slots", "pos", "out"):
        assert call(**{arg: None}) == -1, arg
    for arg in ("len", "new", "free", "taken", "bt", "grown", "q", "k", "slots", "pos", "out"):
        assert call(**{arg: FAKE + 2}) == -3, arg
    assert call(slots=FAKE + 4) == -3
    assert call(S=0) == -1 and call(S=(1 << 20) + 1) == -2 and call(cap=-1) == -1 and call(cap=1 << 31) == -1
    assert call(nf=-1) == -1 and call(pages=0) == -1 and call(pages=1 << 24) == -1 and call(mb=0) == -1
    assert call(ws=None) == -4 and call(n=need - 1) == -4 and call(ws=FAKE + 16) == -3


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(msa, fp8):
    lib = msa._lib
    n = ctypes.c_size_t(0)
    assert lib.msa_append_workspace_size(100, ctypes.byref(n)) == 0
    need = n.value
    assert lib.msa_append_workspace_size(0, ctypes.byref(n)) == -1 and lib.msa_append_workspace_size(5, None) == -1
    assert lib.msa_append_workspace_size(1 << 24, ctypes.byref(n)) == -1
    fine = dict(k=FAKE, sk=512, v=FAKE, sv=512, i=FAKE, si=128, slots=FAKE, tokens=9, hkv=4)
    if fp8:
        fine |= dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, ic=FAKE, isc=FAKE, pages=100, ws=FAKE, n=need)
    else:
        fine |= dict(d=128, kc=FAKE, vc=FAKE, ic=FAKE, pages=100, ws=FAKE, n=need)
    fn = lib.msa_append_paged_fp8 if fp8 else lib.msa_append_paged

    def call(**kw):
        return fn(*{**fine, **kw}.values(), None)

    if not torch.cuda.is_available():
        assert accepted(call()) and accepted(call(sk=520, si=1024)) and accepted(call(tokens=0, k=None, v=None, i=None, slots=None))
        if fp8:
            assert accepted(call(i=None, ic=None, isc=None))
        else:
            assert accepted(call(i=None, ic=None)) and accepted(call(ws=None, n=0)) and accepted(call(d=64, n=256))
    for arg in ("k", "v", "i", "slots", "kc", "vc", "ic") + (("ks", "vs", "isc") if fp8 else ()):
        assert call(**{arg: None}) == -1, arg
        assert call(**{arg: FAKE + 2}) == -3, arg
    assert call(sk=511) == -1 and call(sk=504) == -1 and call(sk=516) == -3 and call(sv=516) == -3 and call(si=120) == -1
    assert call(hkv=0) == -1 and call(hkv=1025) == -2 and call(tokens=-1) == -1 and call(pages=0) == -1
    assert call(pages=1 << 24) == -1 and call(n=need - 1 if fp8 else 255) == -4 and call(ws=FAKE + 16) == -3
    if fp8:
        assert call(ws=None) == -4
        assert call(hkv=1024, sk=1 << 17, sv=1 << 17, tokens=1 << 31) == -2   # more CTAs than a launch has
    else:
        assert call(d=32) == -2


def test_binding_refuses_before_any_call(msa):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="slots"):
        msa.msa_append_paged(x, x, slots, x, x)
    with pytest.raises(TypeError, match="lengths"):
        msa.msa_extend_block_table(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1),
                                   torch.zeros(2, 2), 5)
    with pytest.raises(ValueError, match="capacity"):
        msa.msa_extend_block_table(torch.zeros(2), torch.zeros(2), torch.zeros(1), torch.zeros(2, 2), 1 << 40)
    prob = msa.Problem(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4, 4, 4, 4, 2, 1, 128, 16)
    with pytest.raises(TypeError, match="cu_q"):
        msa.msa_dense_attn_prefill(prob, x, x, x)
