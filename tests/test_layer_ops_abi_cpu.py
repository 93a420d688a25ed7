"""Refusals of the dense decode attention, the eviction and the norm, on the host (pointers are never dereferenced:
every call here returns before any CUDA call, or with "no usable device" where all arguments are fine)."""
import ctypes
import math

import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def msa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_05_gb300 as m
    return m


def decode(msa, **kw):
    p = dict(num_seqs=4, cu_seqlens_q=FAKE, cu_seqlens_k=FAKE, total_q=4, total_k=1024, max_seqlen_q=1,
             max_seqlen_k=1024, num_q_heads=64, num_kv_heads=4, head_dim=128, index_dim=128, block_size=128, topk=16,
             softmax_scale=0.0)
    p.update(kw)
    return msa.MsaProblem(**p)


BAD_PROBLEMS = [
    (dict(num_seqs=0, total_q=0), -1), (dict(cu_seqlens_k=None), -1), (dict(max_seqlen_q=2, total_q=8), -1),
    (dict(total_q=5), -1), (dict(total_k=-1), -1), (dict(max_seqlen_k=2000), -1), (dict(max_seqlen_k=-1), -1),
    (dict(num_q_heads=63), -1), (dict(num_kv_heads=0), -1), (dict(num_q_heads=0), -1),
    (dict(softmax_scale=math.nan), -1), (dict(softmax_scale=math.inf), -1), (dict(softmax_scale=3e38), -1),
    (dict(head_dim=64), -2), (dict(max_seqlen_k=(1 << 30) + 1, total_k=(1 << 30) + 1), -2),
    (dict(block_size=64), -2), (dict(num_q_heads=129, num_kv_heads=1), -2),
    (dict(num_q_heads=1025, num_kv_heads=1025), -2), (dict(num_seqs=(1 << 20) + 1, total_q=(1 << 20) + 1), -2),
]


def ws_size(msa, p, op):
    n = ctypes.c_size_t(0)
    return msa._lib.msa_workspace_size(ctypes.byref(p), int(op), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", BAD_PROBLEMS)
def test_problems_outside_the_range(msa, kw, status):
    p = decode(msa, **kw)
    lib = msa._lib
    n = ctypes.c_size_t(0)
    for op in (msa.Op.DENSE_ATTN_DECODE, msa.Op.DENSE_ATTN_DECODE_WEIGHT):
        assert ws_size(msa, p, op)[0] == status
    assert lib.msa_evict_workspace_size(p, 100, 100, ctypes.byref(n)) == status
    assert lib.msa_dense_attn_decode_paged(p, FAKE, FAKE, FAKE, FAKE, 8, 100, None, 0, FAKE, FAKE, FAKE, 1 << 40,
                                           None) == status
    assert lib.msa_evict_paged(p, FAKE, FAKE, FAKE, 8, 100, FAKE, 1024, 100, 0, FAKE, 8, FAKE, FAKE + 16, 100,
                               FAKE + 16, FAKE, 1 << 40, None) == status


def test_any_group_up_to_128_and_ignored_index_fields(msa):
    for hq, hkv in ((1, 1), (5, 1), (128, 1), (35, 7), (1024, 1024), (96, 2)):
        st, small = ws_size(msa, decode(msa, num_q_heads=hq, num_kv_heads=hkv, topk=0, index_dim=0),
                            msa.Op.DENSE_ATTN_DECODE)
        st2, large = ws_size(msa, decode(msa, num_q_heads=hq, num_kv_heads=hkv), msa.Op.DENSE_ATTN_DECODE_WEIGHT)
        assert st == st2 == 0 and 0 < small < large
    assert ws_size(msa, decode(msa, total_k=0, max_seqlen_k=0), msa.Op.DENSE_ATTN_DECODE)[0] == 0
    n = ctypes.c_size_t(0)
    assert msa._lib.msa_workspace_size(ctypes.byref(decode(msa)), 15, ctypes.byref(n)) == -1
    assert msa._lib.msa_workspace_size(ctypes.byref(decode(msa)), 14, None) == -1


def test_dense_decode_refusals(msa):
    lib = msa._lib
    p = decode(msa)
    need = ws_size(msa, p, msa.Op.DENSE_ATTN_DECODE)[1]

    def call(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=8, pages=100, w=None, stride=0, o=FAKE, lse=FAKE, ws=FAKE, n=1 << 40):
        return lib.msa_dense_attn_decode_paged(p, q, k, v, bt, mb, pages, w, stride, o, lse, ws, n, None)

    for name in ("q", "k", "v", "bt", "o", "lse"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: FAKE + 2}) == -3, name
    assert call(mb=7) == -1 and call(pages=0) == -1 and call(pages=1 << 24) == -1
    assert call(w=FAKE, stride=1023) == -1 and call(w=FAKE + 1, stride=1024) == -3
    assert call(ws=None) == -4 and call(n=need - 1) == -4 and call(ws=FAKE + 16) == -3
    assert call(w=FAKE, stride=1024, n=need) == -4  # the logits need room
    assert lib.msa_dense_attn_decode_paged(None, FAKE, FAKE, FAKE, FAKE, 8, 100, None, 0, FAKE, FAKE, FAKE, 1 << 40,
                                           None) == -1

    def call8(ks=FAKE, vs=FAKE):
        return lib.msa_dense_attn_decode_paged_fp8(p, FAKE, FAKE, FAKE, ks, vs, FAKE, 8, 100, None, 0, FAKE, FAKE, FAKE,
                                                   1 << 40, None)

    assert call8(ks=None) == -1 and call8(vs=None) == -1 and call8(ks=FAKE + 2) == -3 and call8(vs=FAKE + 1) == -3
    if not torch.cuda.is_available():
        assert call(n=need) == -6 and call8() == -6  # everything fits but the device


def test_evict_refusals(msa):
    lib = msa._lib
    p = decode(msa)
    n = ctypes.c_size_t(0)
    assert lib.msa_evict_workspace_size(p, 100, 1000, ctypes.byref(n)) == 0 and n.value >= 4000
    need = n.value
    assert lib.msa_evict_workspace_size(p, 0, 1000, ctypes.byref(n)) == -1
    assert lib.msa_evict_workspace_size(p, 10, 0, ctypes.byref(n)) == -1
    assert lib.msa_evict_workspace_size(p, 10, 1000, None) == -1

    def call(k=FAKE, v=FAKE, bt=FAKE, mb=8, pages=1000, w=FAKE, ws_=1024, budget=300, recent=10, nt=FAKE, nb=3,
             kept=FAKE, nw=FAKE + 64, nws=300, cu=FAKE + 64, ws=FAKE, size=1 << 40):
        return lib.msa_evict_paged(p, k, v, bt, mb, pages, w, ws_, budget, recent, nt, nb, kept, nw, nws, cu, ws, size,
                                   None)

    for name in ("k", "v", "bt", "w", "nt", "kept", "nw", "cu"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: FAKE + 2}) == -3, name
    assert call(mb=7) == -1 and call(pages=0) == -1 and call(pages=1 << 24) == -1
    assert call(budget=0) == -1 and call(recent=-1) == -1 and call(recent=301) == -1
    assert call(ws_=1023) == -1 and call(nws=299) == -1 and call(nb=2) == -1
    assert call(nw=FAKE) == -1 and call(cu=FAKE) == -1  # outputs on top of what is read
    assert call(ws=None) == -4 and call(size=need - 1) == -4 and call(ws=FAKE + 8) == -3

    def call8(ks=FAKE, vs=FAKE):
        return lib.msa_evict_paged_fp8(p, FAKE, FAKE, ks, vs, FAKE, 8, 1000, FAKE, 1024, 300, 10, FAKE, 3, FAKE,
                                       FAKE + 64, 300, FAKE + 64, FAKE, 1 << 40, None)

    assert call8(ks=None) == -1 and call8(vs=None) == -1 and call8(ks=FAKE + 2) == -3
    if not torch.cuda.is_available():
        assert call(size=need) == -6 and call8() == -6


def test_norm_refusals(msa):
    lib = msa._lib

    def call(x=FAKE, r=FAKE, g=FAKE, rows=3, d=64, eps=1e-6, s=FAKE, y=FAKE):
        return lib.msa_add_rms_norm(x, r, g, rows, d, eps, s, y, None)

    for name in ("x", "g", "y"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "r", "g", "s", "y"):
        assert call(**{name: FAKE + 8}) == -3, name
    assert call(rows=-1) == -1 and call(d=0) == -1 and call(eps=-1.0) == -1 and call(eps=math.nan) == -1
    assert call(eps=math.inf) == -1 and call(d=65537) == -2 and call(rows=1 << 31) == -2
    assert call(rows=0) == 0 and call(rows=0, x=None, y=None) == 0  # no work

    def call8(y8=FAKE, sc=FAKE):
        return lib.msa_add_rms_norm_fp8(FAKE, None, FAKE, 3, 64, 1e-6, None, y8, sc, None)

    assert call8(y8=None) == -1 and call8(sc=None) == -1 and call8(y8=FAKE + 4) == -3 and call8(sc=FAKE + 2) == -3
    if not torch.cuda.is_available():
        assert call() == -6 and call(r=None, s=None) == -6 and call8() == -6


def test_the_binding_checks_types_devices_and_shapes(msa):
    """CPU tensors are refused before anything is called."""
    prob = msa.problem_from_seqlens([1, 1], [100, 200], 8, 2, 128, 16, device="cpu")
    t = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    cache, table = t(3 * 128, 2, 128), t(2, 2, d=torch.int32)
    with pytest.raises(TypeError):
        msa.msa_dense_attn_decode_paged(prob, t(2, 8, 128), cache, cache, table)
    with pytest.raises(TypeError):
        msa.msa_evict_paged(prob, cache, cache, table, t(2, 2, 200, d=torch.float32), table, 100)
    with pytest.raises(TypeError):
        msa.msa_add_rms_norm(t(3, 64), t(64))
    with pytest.raises(TypeError):
        msa.msa_add_rms_norm_fp8(t(3, 64, d=torch.float32), t(64))
    for budget, recent in ((2 ** 32 + 5, 0), (100, 2 ** 32), (-2 ** 31 - 1, 0)):  # would be cut off to 5, 0, 2^31 - 1
        with pytest.raises(ValueError):
            msa.msa_evict_paged(prob, cache, cache, table, t(2, 2, 200, d=torch.float32), table, budget, recent)
    with pytest.raises(ValueError):
        msa.msa_evict_workspace_size(prob, 2 ** 32 + 5, 3)
