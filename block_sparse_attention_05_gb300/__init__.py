"""MiniMax Sparse Attention (MSA) forward pass on GB300 -- Python binding.

A thin ctypes layer over the C ABI in ``include/msa.h`` (library
``_lib/libmsa.so``, built for sm_103a by ``__graft_entry__.build()``).  This
module only marshals torch tensors into pointers and sizes and raises on a
non-OK status; every step of the method runs in the library's CUDA kernels.
There is no CPU fallback: importing without the built library raises.

Entry points (same names as the C functions):
  msa_index_pool, msa_topk_pooled, msa_index_topk,
  msa_sparse_attn_prefill, msa_sparse_attn_decode, msa_forward,
  msa_sparse_attn_decode_static, msa_forward_decode_paged,
  msa_quantize_kv_fp8, msa_sparse_attn_prefill_fp8, msa_sparse_attn_decode_fp8, msa_forward_fp8,
  msa_forward_decode_paged_fp8,
  msa_quantize_index_fp8, msa_index_pool_fp8, msa_index_topk_fp8, msa_forward_fp8_index,
  msa_forward_decode_paged_fp8_index,
  msa_index_prologue,
  msa_dense_attn_decode_paged, msa_dense_attn_decode_paged_fp8,
  msa_evict_paged, msa_evict_paged_fp8, msa_evict_workspace_size,
  msa_add_rms_norm, msa_add_rms_norm_fp8,
  msa_dense_attn_prefill, msa_dense_attn_prefill_paged, msa_dense_attn_prefill_paged_fp8,
  msa_tree_attn_paged, msa_tree_attn_paged_fp8,
  msa_extend_block_table, msa_extend_workspace_size, msa_append_paged, msa_append_paged_fp8, msa_append_workspace_size,
  msa_workspace_size, msa_read_device_status.
"""
from __future__ import annotations

import ctypes
import dataclasses
import enum
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmsa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first (python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)


class MsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = _lib.msa_last_error_detail().decode() if status == -5 else ""
        super().__init__(f"{where}: {_lib.msa_status_string(status).decode()} (status {status})"
                         + (f" [{detail}]" if detail else ""))


class Op(enum.IntEnum):
    INDEX_PROLOGUE = 11
    INDEX_POOL = 1
    INDEX_TOPK = 2
    SPARSE_ATTN_PREFILL = 3
    SPARSE_ATTN_DECODE = 4
    FORWARD = 5
    TOPK_POOLED = 6
    QUANTIZE_KV_FP8 = 7
    SPARSE_ATTN_PREFILL_FP8 = 8
    SPARSE_ATTN_DECODE_FP8 = 9
    FORWARD_FP8 = 10
    QUANTIZE_INDEX_FP8 = 12
    DENSE_ATTN_DECODE = 13
    DENSE_ATTN_DECODE_WEIGHT = 14
    DENSE_ATTN_PREFILL = 16
    TREE_ATTN = 17


DEVICE_TIMEOUT = 1
DEVICE_BAD_SEQLENS = 2
DEVICE_BAD_INDEX = 4


class MsaProblem(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("cu_seqlens_q", ctypes.c_void_p),
        ("cu_seqlens_k", ctypes.c_void_p),
        ("total_q", ctypes.c_int32),
        ("total_k", ctypes.c_int32),
        ("max_seqlen_q", ctypes.c_int32),
        ("max_seqlen_k", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("index_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
    ]


_P = ctypes.POINTER(MsaProblem)
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t

_lib.msa_status_string.restype = ctypes.c_char_p
_lib.msa_status_string.argtypes = [ctypes.c_int]
_lib.msa_abi_version.restype = ctypes.c_int32
_lib.msa_workspace_size.restype = ctypes.c_int
_lib.msa_workspace_size.argtypes = [_P, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
_lib.msa_index_pool.restype = ctypes.c_int
_lib.msa_index_pool.argtypes = [_P, _vp, _vp, _vp, _i64, _vp, _sz, _vp]
_lib.msa_topk_pooled.restype = ctypes.c_int
_lib.msa_topk_pooled.argtypes = [_P, _vp, _i64, _vp, _vp, _sz, _vp]
_lib.msa_index_topk.restype = ctypes.c_int
_lib.msa_index_topk.argtypes = [_P, _vp, _vp, _vp, _vp, _sz, _vp]
for _fn in (_lib.msa_sparse_attn_prefill, _lib.msa_sparse_attn_decode):
    _fn.restype = ctypes.c_int
    _fn.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.msa_sparse_attn_decode_static.restype = ctypes.c_int
_lib.msa_sparse_attn_decode_static.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.msa_forward.restype = ctypes.c_int
_lib.msa_forward.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.msa_forward_decode_paged.restype = ctypes.c_int
_lib.msa_forward_decode_paged.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int32, _i64, _vp, _vp, _vp, _vp,
                                          _sz, _vp]
_lib.msa_quantize_kv_fp8.restype = ctypes.c_int
_lib.msa_quantize_kv_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
for _fn in (_lib.msa_sparse_attn_prefill_fp8, _lib.msa_sparse_attn_decode_fp8):
    _fn.restype = ctypes.c_int
    _fn.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.msa_forward_fp8.restype = ctypes.c_int
_lib.msa_forward_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
# problem, q, k8, v8, k_scale, v_scale, q_idx, k_idx cache, block table, stride, pages, idx, o, lse, ws, bytes, stream
_lib.msa_forward_decode_paged_fp8.restype = ctypes.c_int
_lib.msa_forward_decode_paged_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int32, _i64, _vp,
                                              _vp, _vp, _vp, _sz, _vp]
# problem, q_idx, k_idx, q_idx8, q_idx_scale, k_idx8, k_idx_scale, ws, bytes, stream
_lib.msa_quantize_index_fp8.restype = ctypes.c_int
_lib.msa_quantize_index_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
# problem, q_idx8, q_idx_scale, k_idx8, k_idx_scale, pooled, stride, ws, bytes, stream
_lib.msa_index_pool_fp8.restype = ctypes.c_int
_lib.msa_index_pool_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]
_lib.msa_index_topk_fp8.restype = ctypes.c_int
_lib.msa_index_topk_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
# problem, q, k8, v8, k_scale, v_scale, q_idx8, q_idx_scale, k_idx8, k_idx_scale, idx, o, lse, ws, bytes, stream
_lib.msa_forward_fp8_index.restype = ctypes.c_int
_lib.msa_forward_fp8_index.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
# problem, q, k8, v8, k_scale, v_scale, q_idx8, q_idx_scale, k_idx8 cache, k_idx_scale, block table, stride, pages,
# idx, o, lse, ws, bytes, stream
_lib.msa_forward_decode_paged_fp8_index.restype = ctypes.c_int
_lib.msa_forward_decode_paged_fp8_index.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                    ctypes.c_int32, _i64, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.msa_index_prologue.restype = ctypes.c_int
_lib.msa_index_prologue.argtypes = [_P, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
# problem, q, k, v, block table, stride, pages, weight, weight stride, o, lse, ws, bytes, stream
_lib.msa_dense_attn_decode_paged.restype = ctypes.c_int
_lib.msa_dense_attn_decode_paged.argtypes = [_P, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp]
_lib.msa_dense_attn_decode_paged_fp8.restype = ctypes.c_int
_lib.msa_dense_attn_decode_paged_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _i64, _vp, _vp,
                                                 _vp, _sz, _vp]
_lib.msa_evict_workspace_size.restype = ctypes.c_int
_lib.msa_evict_workspace_size.argtypes = [_P, _i32, _i64, ctypes.POINTER(ctypes.c_size_t)]
# problem, k, v, block table, stride, pages, weight, weight stride, budget, recent, new table, new stride, kept,
# new weight, new weight stride, new cu_seqlens_k, ws, bytes, stream
_lib.msa_evict_paged.restype = ctypes.c_int
_lib.msa_evict_paged.argtypes = [_P, _vp, _vp, _vp, _i32, _i64, _vp, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _i64, _vp,
                                 _vp, _sz, _vp]
_lib.msa_evict_paged_fp8.restype = ctypes.c_int
_lib.msa_evict_paged_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _i64, _i32, _i32, _vp, _i32, _vp,
                                     _vp, _i64, _vp, _vp, _sz, _vp]
# x, residual, gamma, rows, d_model, eps, sum, y (or y8, y_scale), stream
_lib.msa_add_rms_norm.restype = ctypes.c_int
_lib.msa_add_rms_norm.argtypes = [_vp, _vp, _vp, _i64, _i32, _f32, _vp, _vp, _vp]
_lib.msa_add_rms_norm_fp8.restype = ctypes.c_int
_lib.msa_add_rms_norm_fp8.argtypes = [_vp, _vp, _vp, _i64, _i32, _f32, _vp, _vp, _vp, _vp]
# problem, q, k, v, o, lse, ws, bytes, stream
_lib.msa_dense_attn_prefill.restype = ctypes.c_int
_lib.msa_dense_attn_prefill.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
# problem, q, caches (, scales), block table, stride, pages (, visible, words), o, lse, ws, bytes, stream
_lib.msa_dense_attn_prefill_paged.restype = ctypes.c_int
_lib.msa_dense_attn_prefill_paged.argtypes = [_P, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _sz, _vp]
_lib.msa_dense_attn_prefill_paged_fp8.restype = ctypes.c_int
_lib.msa_dense_attn_prefill_paged_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _sz, _vp]
_lib.msa_tree_attn_paged.restype = ctypes.c_int
_lib.msa_tree_attn_paged.argtypes = [_P, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _i32, _vp, _vp, _vp, _sz, _vp]
_lib.msa_tree_attn_paged_fp8.restype = ctypes.c_int
_lib.msa_tree_attn_paged_fp8.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _i32, _vp, _vp, _vp, _sz,
                                         _vp]
_lib.msa_extend_workspace_size.restype = ctypes.c_int
_lib.msa_extend_workspace_size.argtypes = [_i32, ctypes.POINTER(ctypes.c_size_t)]
# seqs, lengths, new tokens, capacity, free pages, their number, taken, pages, block table, stride, new lengths,
# cu_seqlens_q, cu_seqlens_k, slots, positions, taken_out, ws, bytes, stream
_lib.msa_extend_block_table.restype = ctypes.c_int
_lib.msa_extend_block_table.argtypes = [_i32, _vp, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _sz, _vp]
_lib.msa_append_workspace_size.restype = ctypes.c_int
_lib.msa_append_workspace_size.argtypes = [_i64, ctypes.POINTER(ctypes.c_size_t)]
# k, stride, v, stride, k_idx, stride, slots, tokens, heads, index_dim, caches, pages, ws, bytes, stream
_lib.msa_append_paged.restype = ctypes.c_int
_lib.msa_append_paged.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _sz,
                                  _vp]
# k, stride, v, stride, k_idx, stride, slots, tokens, heads, k, v, scales, k_idx, scale, pages, ws, bytes, stream
_lib.msa_append_paged_fp8.restype = ctypes.c_int
_lib.msa_append_paged_fp8.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _i64, _vp, _sz, _vp]
_lib.msa_read_device_status.restype = ctypes.c_int
_lib.msa_read_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32), _vp]
_lib.msa_set_stage_events.restype = ctypes.c_int
_lib.msa_set_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
_lib.msa_kernel_launch_count.restype = ctypes.c_int64
_lib.msa_last_error_detail.restype = ctypes.c_char_p

EXPORTED = ("msa_workspace_size", "msa_index_pool", "msa_topk_pooled", "msa_index_topk",
            "msa_sparse_attn_prefill", "msa_sparse_attn_decode", "msa_forward",
            "msa_read_device_status", "msa_status_string", "msa_abi_version", "msa_set_stage_events",
            "msa_kernel_launch_count", "msa_last_error_detail", "msa_sparse_attn_decode_static",
            "msa_forward_decode_paged", "msa_quantize_kv_fp8", "msa_sparse_attn_prefill_fp8",
            "msa_sparse_attn_decode_fp8", "msa_forward_fp8", "msa_index_prologue",
            "msa_forward_decode_paged_fp8", "msa_quantize_index_fp8", "msa_index_pool_fp8", "msa_index_topk_fp8",
            "msa_forward_fp8_index", "msa_forward_decode_paged_fp8_index",
            "msa_dense_attn_decode_paged", "msa_dense_attn_decode_paged_fp8", "msa_evict_workspace_size",
            "msa_evict_paged", "msa_evict_paged_fp8", "msa_add_rms_norm", "msa_add_rms_norm_fp8",
            "msa_dense_attn_prefill", "msa_dense_attn_prefill_paged", "msa_dense_attn_prefill_paged_fp8",
            "msa_tree_attn_paged", "msa_tree_attn_paged_fp8", "msa_extend_workspace_size", "msa_extend_block_table",
            "msa_append_workspace_size", "msa_append_paged", "msa_append_paged_fp8")

STAGES = ("plan", "index", "topk", "schedule", "attn", "combine")


@dataclasses.dataclass
class Problem:
    """Sizes of one packed batch.  ``cu_q`` / ``cu_k`` are int32 device tensors."""
    cu_q: torch.Tensor
    cu_k: torch.Tensor
    total_q: int
    total_k: int
    max_q: int
    max_k: int
    hq: int
    hkv: int
    d_idx: int
    topk: int
    head_dim: int = 128
    block: int = 128
    scale: float = 0.0

    @property
    def num_seqs(self) -> int:
        return int(self.cu_q.numel()) - 1

    def c(self) -> MsaProblem:
        return MsaProblem(self.num_seqs, _ptr(self.cu_q), _ptr(self.cu_k), self.total_q, self.total_k,
                          self.max_q, self.max_k, self.hq, self.hkv, self.head_dim, self.d_idx, self.block,
                          self.topk, self.scale)


def problem_from_seqlens(q_lens, kv_lens, hq, hkv, d_idx, topk, device="cuda", scale=0.0) -> Problem:
    """Builds the prefix sums from per-sequence lengths (host lists)."""
    cu_q = [0]
    cu_k = [0]
    for a, b in zip(q_lens, kv_lens):
        cu_q.append(cu_q[-1] + int(a))
        cu_k.append(cu_k[-1] + int(b))
    return Problem(torch.tensor(cu_q, dtype=torch.int32, device=device),
                   torch.tensor(cu_k, dtype=torch.int32, device=device), cu_q[-1], cu_k[-1],
                   max(q_lens) if len(q_lens) else 0, max(kv_lens) if len(kv_lens) else 0, hq, hkv, d_idx, topk,
                   scale=scale)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise MsaError(status, where)


def _need(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def msa_workspace_size(problem: Problem, op: Op) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.msa_workspace_size(ctypes.byref(problem.c()), int(op), ctypes.byref(n)), "msa_workspace_size")
    return int(n.value)


def workspace(problem: Problem, op: Op, device=None) -> torch.Tensor:
    """A device buffer large enough for ``op`` (256-byte aligned by the caching allocator)."""
    nbytes = max(msa_workspace_size(problem, op), 256)
    return torch.empty(nbytes, dtype=torch.uint8, device=device or problem.cu_q.device)


def _ws(problem, op, ws):
    if ws is None:
        ws = workspace(problem, op)
    return ws, ctypes.c_size_t(ws.numel())


def max_blocks(problem: Problem) -> int:
    return max(1, (problem.max_k + problem.block - 1) // problem.block)


def msa_index_pool(problem: Problem, q_idx, k_idx, pooled=None, ws=None):
    """Pooled causal index scores, fp32 [total_q * hkv, ceil(max_k / 128)]; entries past a row's causal end
    are left as they were (NaN when ``pooled`` is allocated here)."""
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(k_idx, torch.bfloat16, "k_idx")
    nb = max_blocks(problem)
    if pooled is None:
        pooled = torch.full((problem.total_q * problem.hkv, nb), float("nan"), dtype=torch.float32,
                            device=q_idx.device)
    ws, nws = _ws(problem, Op.INDEX_POOL, ws)
    _check(_lib.msa_index_pool(ctypes.byref(problem.c()), _ptr(q_idx), _ptr(k_idx), _ptr(pooled),
                               pooled.stride(0), _ptr(ws), nws, _stream()), "msa_index_pool")
    return pooled


def msa_topk_pooled(problem: Problem, pooled, idx=None, ws=None):
    _need(pooled, torch.float32, "pooled")
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=pooled.device)
    ws, nws = _ws(problem, Op.TOPK_POOLED, ws)
    _check(_lib.msa_topk_pooled(ctypes.byref(problem.c()), _ptr(pooled), pooled.stride(0), _ptr(idx), _ptr(ws),
                                nws, _stream()), "msa_topk_pooled")
    return idx


def msa_index_topk(problem: Problem, q_idx, k_idx, idx=None, ws=None):
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(k_idx, torch.bfloat16, "k_idx")
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=q_idx.device)
    ws, nws = _ws(problem, Op.INDEX_TOPK, ws)
    _check(_lib.msa_index_topk(ctypes.byref(problem.c()), _ptr(q_idx), _ptr(k_idx), _ptr(idx), _ptr(ws), nws,
                               _stream()), "msa_index_topk")
    return idx


def _attn(fn, op, where, problem, q, k, v, idx, o, lse, ws):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    _need(idx, torch.int32, "idx")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=q.device)
    ws, nws = _ws(problem, op, ws)
    _check(fn(ctypes.byref(problem.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(o), _ptr(lse), _ptr(ws), nws,
              _stream()), where)
    return o, lse


def msa_sparse_attn_prefill(problem: Problem, q, k, v, idx, o=None, lse=None, ws=None):
    return _attn(_lib.msa_sparse_attn_prefill, Op.SPARSE_ATTN_PREFILL, "msa_sparse_attn_prefill", problem, q, k,
                 v, idx, o, lse, ws)


def msa_sparse_attn_decode(problem: Problem, q, k, v, idx, o=None, lse=None, ws=None):
    return _attn(_lib.msa_sparse_attn_decode, Op.SPARSE_ATTN_DECODE, "msa_sparse_attn_decode", problem, q, k, v,
                 idx, o, lse, ws)


def msa_sparse_attn_decode_static(problem: Problem, q, k, v, idx, o=None, lse=None):
    """The decode Main Branch without a workspace: its scratch is a fixed device array inside the library
    (for callers that cannot allocate device memory; see include/msa.h).  Calls share that array, so calls
    that may overlap on the GPU must be serialised."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    _need(idx, torch.int32, "idx")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=q.device)
    _check(_lib.msa_sparse_attn_decode_static(ctypes.byref(problem.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(idx),
                                              _ptr(o), _ptr(lse), _stream()), "msa_sparse_attn_decode_static")
    return o, lse


def msa_forward(problem: Problem, q, k, v, q_idx, k_idx, idx=None, o=None, lse=None, ws=None):
    """Both branches.  Returns (idx [T, Hkv, k] int32, o [T, Hq, 128] bf16, lse [T, Hq] fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (q_idx, "q_idx"), (k_idx, "k_idx")):
        _need(t, torch.bfloat16, n)
    dev = q.device
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.FORWARD, ws)
    _check(_lib.msa_forward(ctypes.byref(problem.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(q_idx), _ptr(k_idx),
                            _ptr(idx), _ptr(o), _ptr(lse), _ptr(ws), nws, _stream()), "msa_forward")
    return idx, o, lse


def msa_forward_decode_paged(problem: Problem, q, k_cache, v_cache, q_idx, k_idx_cache, block_table, idx=None,
                             o=None, lse=None, ws=None):
    """Decode from paged caches ([num_pages * 128, ...] rows, block_table int32 [num_seqs, max_blocks]).
    Returns (idx, o, lse) as msa_forward."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (q_idx, "q_idx"), (k_idx_cache, "k_idx_cache")):
        _need(t, torch.bfloat16, n)
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or k_cache.shape[0] % 128:
        raise ValueError("block_table must be [num_seqs, max_blocks] and the caches whole pages of 128 rows")
    dev = q.device
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.FORWARD, ws)
    _check(_lib.msa_forward_decode_paged(ctypes.byref(problem.c()), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                         _ptr(q_idx), _ptr(k_idx_cache), _ptr(block_table), block_table.shape[1],
                                         k_cache.shape[0] // 128, _ptr(idx), _ptr(o), _ptr(lse), _ptr(ws), nws,
                                         _stream()), "msa_forward_decode_paged")
    return idx, o, lse


# ---------------------------------------------------------------- index prologue
def msa_index_prologue(problem: Problem, x, w_q, w_k, gamma_q, gamma_k, k_idx, q_idx=None, ws=None):
    """Hidden states x [total_q, d_model] -> Q_idx [total_q, Hkv, 128] (returned) and the new tokens' rows
    k_start + pos(i) of the index-key cache k_idx [total_k, 128] (written in place): projection, RMSNorm,
    RoPE on dims 0..63."""
    for t, n in ((x, "x"), (w_q, "w_q"), (w_k, "w_k"), (gamma_q, "gamma_q"), (gamma_k, "gamma_k"), (k_idx, "k_idx")):
        _need(t, torch.bfloat16, n)
    if q_idx is None:
        q_idx = torch.empty((problem.total_q, problem.hkv, problem.d_idx), dtype=torch.bfloat16, device=x.device)
    ws, nws = _ws(problem, Op.INDEX_PROLOGUE, ws)
    _check(_lib.msa_index_prologue(ctypes.byref(problem.c()), _ptr(x), int(x.shape[1]), _ptr(w_q), _ptr(w_k),
                                   _ptr(gamma_q), _ptr(gamma_k), _ptr(q_idx), _ptr(k_idx), _ptr(ws), nws, _stream()),
           "msa_index_prologue")
    return q_idx


# ---------------------------------------------------------------- dense decode attention, eviction, norm
# The current device and stream as plain numbers: torch's own accessors, without the objects that torch.cuda's
# functions make around them (3 us a call on the host, as much as a small kernel takes).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _refuse(t, dtype, shape, dev, name):
    _need(t, dtype, name)
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")
    raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")


def _is(t, dtype, shape, dev, name):
    """The address of a contiguous tensor of this type and shape on the current CUDA device `dev`."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    _refuse(t, dtype, shape, dev, name)


def _c_paged(problem):
    """Problem.c() for the calls below, checked (every field that they read), with plain integers for the pointers."""
    cu_q, cu_k = problem.cu_q, problem.cu_k
    if not cu_q.is_cuda:
        _need(cu_q, torch.int32, "cu_q")
    n = cu_q.shape[0] - 1
    dev = _current_device()
    _is(cu_q, torch.int32, (n + 1,), dev, "cu_q")
    at_k = _is(cu_k, torch.int32, (n + 1,), dev, "cu_k")
    return n, dev, MsaProblem(n, cu_q.data_ptr(), at_k, problem.total_q, problem.total_k, problem.max_q, problem.max_k,
                              problem.hq, problem.hkv, problem.head_dim, problem.d_idx, problem.block, problem.topk,
                              problem.scale)


def _table(t, n, dev, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected [num_seqs, max_blocks], got {list(t.shape)}")
    return _is(t, torch.int32, (n, t.shape[1]), dev, name)


def _pages(problem, dev, dtype, k_cache, v_cache, scales):
    """Checks a paged cache; returns the number of pages and the addresses of the caches and scales."""
    rows = k_cache.shape[0]
    shape = (rows, problem.hkv, 128)
    at = (_is(k_cache, dtype, shape, dev, "k_cache"), _is(v_cache, dtype, shape, dev, "v_cache"))
    if rows % 128:
        raise ValueError("the caches must be whole pages of 128 rows")
    if scales:
        shape = (rows // 128, problem.hkv)
        at += (_is(scales[0], torch.float32, shape, dev, "k_scale"), _is(scales[1], torch.float32, shape, dev, "v_scale"))
    return rows // 128, at


def _weight(t, n, hkv, dev, name):
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [num_seqs, num_kv_heads, tokens], got {list(t.shape)}")
    return _is(t, torch.float32, (n, hkv, t.shape[2]), dev, name)


def _space(ws, nbytes, dev):
    """The workspace's address and size; a buffer of its own where the caller gives none."""
    if ws is None:
        ws = torch.empty(nbytes(), dtype=torch.uint8, device=f"cuda:{dev}")
    elif ws.get_device() != dev or not ws.is_contiguous():
        _refuse(ws, ws.dtype, ws.shape, dev, "ws")
    return ws, ws.data_ptr(), ws.nbytes


def _dense(problem, q, k, v, scales, block_table, weight, o, lse, ws):
    S, dev, c = _c_paged(problem)
    pages, caches = _pages(problem, dev, torch.uint8 if scales else torch.bfloat16, k, v, scales)
    shape = (S, problem.hq, 128)
    at_q, at_table = _is(q, torch.bfloat16, shape, dev, "q"), _table(block_table, S, dev, "block_table")
    at_weight, stride, op = None, 0, Op.DENSE_ATTN_DECODE
    if weight is not None:
        at_weight, stride = _weight(weight, S, problem.hkv, dev, "weight"), weight.shape[2]
        op = Op.DENSE_ATTN_DECODE_WEIGHT
    if o is None:
        o = torch.empty_like(q)
        at_o = o.data_ptr()
    else:
        at_o = _is(o, torch.bfloat16, shape, dev, "o")
    if lse is None:
        lse = torch.empty((S, shape[1]), dtype=torch.float32, device=q.device)
        at_lse = lse.data_ptr()
    else:
        at_lse = _is(lse, torch.float32, (S, shape[1]), dev, "lse")
    ws, at_ws, nws = _space(ws, lambda: msa_workspace_size(problem, op), dev)
    fn, where = ((_lib.msa_dense_attn_decode_paged_fp8, "msa_dense_attn_decode_paged_fp8") if scales else
                 (_lib.msa_dense_attn_decode_paged, "msa_dense_attn_decode_paged"))
    status = fn(c, at_q, *caches, at_table, block_table.shape[1], pages, at_weight, stride, at_o, at_lse, at_ws, nws,
                _raw_stream(dev))
    if status:
        raise MsaError(status, where)
    return o, lse


def msa_dense_attn_decode_paged(problem: Problem, q, k_cache, v_cache, block_table, weight=None, o=None, lse=None,
                                ws=None):
    """Attention of one new token per sequence over every key of its paged cache ([num_pages * 128, Hkv, 128] rows,
    block_table int32 [num_seqs, max_blocks]); any group size up to 128, cached lengths from 0 (o = 0, lse = -inf).
    ``weight`` (fp32 [num_seqs, Hkv, >= max_k]) is added to in place: each cached key's attention weight, summed over
    the group's heads.  Returns (o [num_seqs, Hq, 128] bf16, lse [num_seqs, Hq] fp32).  Workspace: op
    DENSE_ATTN_DECODE, or DENSE_ATTN_DECODE_WEIGHT with a weight."""
    return _dense(problem, q, k_cache, v_cache, None, block_table, weight, o, lse, ws)


def msa_dense_attn_decode_paged_fp8(problem: Problem, q, k8_cache, v8_cache, k_scale, v_scale, block_table,
                                    weight=None, o=None, lse=None, ws=None):
    """msa_dense_attn_decode_paged over E4M3 pages (uint8 codes) with k_scale / v_scale [num_pages, Hkv]."""
    return _dense(problem, q, k8_cache, v8_cache, (k_scale, v_scale), block_table, weight, o, lse, ws)


def _int32(x, name):
    if not -2 ** 31 <= x < 2 ** 31:  # ctypes would cut it off
        raise ValueError(f"{name}: {x} does not fit 32 bits")


def msa_evict_workspace_size(problem: Problem, budget: int, num_pages: int) -> int:
    _int32(budget, "budget")
    n = ctypes.c_size_t(0)
    _check(_lib.msa_evict_workspace_size(problem.c(), budget, num_pages, ctypes.byref(n)), "msa_evict_workspace_size")
    return int(n.value)


def evict_workspace(problem: Problem, budget: int, num_pages: int, device=None) -> torch.Tensor:
    """A device buffer for msa_evict_paged and msa_evict_paged_fp8 over caches of ``num_pages`` pages."""
    return torch.empty(msa_evict_workspace_size(problem, budget, num_pages), dtype=torch.uint8,
                       device=device or problem.cu_k.device)


def _evict(problem, k, v, scales, block_table, weight, new_block_table, budget, recent, kept, new_weight, new_cu_k, ws):
    _int32(budget, "budget")
    _int32(recent, "recent")
    S, dev, c = _c_paged(problem)
    hkv = problem.hkv
    pages, caches = _pages(problem, dev, torch.uint8 if scales else torch.bfloat16, k, v, scales)
    at_table, at_new = _table(block_table, S, dev, "block_table"), _table(new_block_table, S, dev, "new_block_table")
    at_weight = _weight(weight, S, hkv, dev, "weight")
    device = k.device
    if kept is None:
        kept = torch.empty((S, hkv, budget), dtype=torch.int32, device=device)
        at_kept = kept.data_ptr()
    else:
        at_kept = _is(kept, torch.int32, (S, hkv, budget), dev, "kept")
    if new_weight is None:
        new_weight = torch.zeros((S, hkv, budget), dtype=torch.float32, device=device)
    at_new_weight = _weight(new_weight, S, hkv, dev, "new_weight")
    if new_cu_k is None:
        new_cu_k = torch.empty(S + 1, dtype=torch.int32, device=device)
        at_cu = new_cu_k.data_ptr()
    else:
        at_cu = _is(new_cu_k, torch.int32, (S + 1,), dev, "new_cu_k")
    ws, at_ws, nws = _space(ws, lambda: msa_evict_workspace_size(problem, budget, pages), dev)
    fn, where = ((_lib.msa_evict_paged_fp8, "msa_evict_paged_fp8") if scales else
                 (_lib.msa_evict_paged, "msa_evict_paged"))
    status = fn(c, *caches, at_table, block_table.shape[1], pages, at_weight, weight.shape[2], budget, recent, at_new,
                new_block_table.shape[1], at_kept, at_new_weight, new_weight.shape[2], at_cu, at_ws, nws,
                _raw_stream(dev))
    if status:
        raise MsaError(status, where)
    return kept, new_weight, new_cu_k


def msa_evict_paged(problem: Problem, k_cache, v_cache, block_table, weight, new_block_table, budget: int,
                    recent: int = 0, kept=None, new_weight=None, new_cu_k=None, ws=None):
    """Eviction by accumulated attention weight: per (sequence, KV head) the last ``recent`` slots and the others with
    the largest ``weight`` (equal weights to the lower slot), ``budget`` in all, gathered in order into the pages of
    ``new_block_table`` (pages of the same caches, apart from those of ``block_table``).  Returns (kept slots int32
    [num_seqs, Hkv, budget], -1 padded; their weights [num_seqs, Hkv, budget], zeros behind the new length; prefix
    sums of the new lengths int32 [num_seqs + 1]).  Workspace: evict_workspace."""
    return _evict(problem, k_cache, v_cache, None, block_table, weight, new_block_table, budget, recent, kept,
                  new_weight, new_cu_k, ws)


def msa_evict_paged_fp8(problem: Problem, k8_cache, v8_cache, k_scale, v_scale, block_table, weight, new_block_table,
                        budget: int, recent: int = 0, kept=None, new_weight=None, new_cu_k=None, ws=None):
    """msa_evict_paged over E4M3 pages: the rows of a new page are rounded again at its scale (written to k_scale and
    v_scale [num_pages, Hkv])."""
    return _evict(problem, k8_cache, v8_cache, (k_scale, v_scale), block_table, weight, new_block_table, budget,
                  recent, kept, new_weight, new_cu_k, ws)


def _norm_args(x, gamma, residual, sum_out):
    """Checked inputs: (device, sum, (x, residual, gamma, rows, width), address of sum)."""
    if not x.is_cuda:
        _need(x, torch.bfloat16, "x")
    shape, dev = x.shape, _current_device()
    if not shape:
        raise ValueError("x: needs a dimension to normalise")
    width = shape[-1]
    at_x, at_gamma = _is(x, torch.bfloat16, shape, dev, "x"), _is(gamma, torch.bfloat16, (width,), dev, "gamma")
    at_residual = None if residual is None else _is(residual, torch.bfloat16, shape, dev, "residual")
    if sum_out is None:
        sum_out = torch.empty_like(x)
        at_sum = sum_out.data_ptr()
    else:
        at_sum = _is(sum_out, torch.bfloat16, shape, dev, "sum_out")
    return dev, sum_out, (at_x, at_residual, at_gamma, x.numel() // width if width else 0, width), at_sum


def msa_add_rms_norm(x, gamma, residual=None, eps: float = 1e-6, sum_out=None, y=None):
    """h = x + residual in fp32; returns (bf16(h), bf16(h / sqrt(mean(h^2) + eps) * gamma)) over the last dimension.
    ``sum_out`` may be x or residual (in place), and ``y`` the other one."""
    dev, sum_out, args, at_sum = _norm_args(x, gamma, residual, sum_out)
    if y is None:
        y = torch.empty_like(x)
        at_y = y.data_ptr()
    else:
        at_y = _is(y, torch.bfloat16, x.shape, dev, "y")
    status = _lib.msa_add_rms_norm(*args, eps, at_sum, at_y, _raw_stream(dev))
    if status:
        raise MsaError(status, "msa_add_rms_norm")
    return sum_out, y


def msa_add_rms_norm_fp8(x, gamma, residual=None, eps: float = 1e-6, sum_out=None, y8=None, y_scale=None):
    """msa_add_rms_norm with the norm as E4M3 codes (uint8) and one fp32 scale per row (max |y| / 448, 1 when 0).
    Returns (sum, y8, y_scale)."""
    dev, sum_out, args, at_sum = _norm_args(x, gamma, residual, sum_out)
    shape = x.shape
    if y8 is None:
        y8 = torch.empty(shape, dtype=torch.uint8, device=x.device)
        at_y8 = y8.data_ptr()
    else:
        at_y8 = _is(y8, torch.uint8, shape, dev, "y8")
    if y_scale is None:
        y_scale = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        at_scale = y_scale.data_ptr()
    else:
        at_scale = _is(y_scale, torch.float32, shape[:-1], dev, "y_scale")
    status = _lib.msa_add_rms_norm_fp8(*args, eps, at_sum, at_y8, at_scale, _raw_stream(dev))
    if status:
        raise MsaError(status, "msa_add_rms_norm_fp8")
    return sum_out, y8, y_scale


# ---------------------------------------------------------------- prompts, drafted trees, cache tables and rows
def _prompt(where, op, problem, q, k, v, scales, block_table, visible, o, lse, ws):
    S, dev, c = _c_paged(problem)
    T, hq = problem.total_q, problem.hq
    args = ()
    if block_table is None:
        shape = (problem.total_k, problem.hkv, 128)
        caches = (_is(k, torch.bfloat16, shape, dev, "k"), _is(v, torch.bfloat16, shape, dev, "v"))
    else:
        pages, caches = _pages(problem, dev, torch.uint8 if scales else torch.bfloat16, k, v, scales)
        args = (_table(block_table, S, dev, "block_table"), block_table.shape[1], pages)
    if op is Op.TREE_ATTN:
        if visible.dim() != 2:
            raise ValueError(f"visible: expected [total_q, words], got {list(visible.shape)}")
        args += (_is(visible, torch.int32, (T, visible.shape[1]), dev, "visible"), visible.shape[1])
    at_q = _is(q, torch.bfloat16, (T, hq, 128), dev, "q")
    if o is None:
        o = torch.empty_like(q)
        at_o = o.data_ptr()
    else:
        at_o = _is(o, torch.bfloat16, (T, hq, 128), dev, "o")
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
        at_lse = lse.data_ptr()
    else:
        at_lse = _is(lse, torch.float32, (T, hq), dev, "lse")
    ws, at_ws, nws = _space(ws, lambda: msa_workspace_size(problem, op), dev)
    status = getattr(_lib, where)(c, at_q, *caches, *args, at_o, at_lse, at_ws, nws, _raw_stream(dev))
    if status:
        raise MsaError(status, where)
    return o, lse


def msa_dense_attn_prefill(problem: Problem, q, k, v, o=None, lse=None, ws=None):
    """Causal attention of prompts and prompt chunks over every key: packed q [total_q, Hq, 128] and k, v [total_k, Hkv,
    128], the queries the last q_len positions of their sequences; any group size up to 128, lengths from 0.  Returns (o
    [total_q, Hq, 128] bf16, lse [total_q, Hq] fp32).  Workspace: op DENSE_ATTN_PREFILL."""
    return _prompt("msa_dense_attn_prefill", Op.DENSE_ATTN_PREFILL, problem, q, k, v, None, None, None, o, lse, ws)


def msa_dense_attn_prefill_paged(problem: Problem, q, k_cache, v_cache, block_table, o=None, lse=None, ws=None):
    """msa_dense_attn_prefill over a paged cache ([num_pages * 128, Hkv, 128] rows, block_table int32 [num_seqs,
    max_blocks]) that holds the new tokens' rows already."""
    return _prompt("msa_dense_attn_prefill_paged", Op.DENSE_ATTN_PREFILL, problem, q, k_cache, v_cache, None,
                   block_table, None, o, lse, ws)


def msa_dense_attn_prefill_paged_fp8(problem: Problem, q, k8_cache, v8_cache, k_scale, v_scale, block_table, o=None,
                                     lse=None, ws=None):
    """msa_dense_attn_prefill_paged over E4M3 pages (uint8 codes) with k_scale / v_scale [num_pages, Hkv]."""
    return _prompt("msa_dense_attn_prefill_paged_fp8", Op.DENSE_ATTN_PREFILL, problem, q, k8_cache, v8_cache,
                   (k_scale, v_scale), block_table, None, o, lse, ws)


def msa_tree_attn_paged(problem: Problem, q, k_cache, v_cache, block_table, visible, o=None, lse=None, ws=None):
    """Attention of a tree of drafted tokens: the q_len new tokens of each sequence (in the cache's last q_len slots) see
    every cached key before them and the drafts whose bit is set in their row of ``visible`` (int32 [total_q, words], bit
    d % 32 of word d / 32 for draft d of the sequence).  Returns (o, lse) as msa_dense_attn_prefill; a draft that sees no
    key has o = 0, lse = -inf.  Workspace: op TREE_ATTN."""
    return _prompt("msa_tree_attn_paged", Op.TREE_ATTN, problem, q, k_cache, v_cache, None, block_table, visible, o, lse,
                   ws)


def msa_tree_attn_paged_fp8(problem: Problem, q, k8_cache, v8_cache, k_scale, v_scale, block_table, visible, o=None,
                            lse=None, ws=None):
    """msa_tree_attn_paged over E4M3 pages (uint8 codes) with k_scale / v_scale [num_pages, Hkv]."""
    return _prompt("msa_tree_attn_paged_fp8", Op.TREE_ATTN, problem, q, k8_cache, v8_cache, (k_scale, v_scale),
                   block_table, visible, o, lse, ws)


def msa_extend_workspace_size(num_seqs: int) -> int:
    _int32(num_seqs, "num_seqs")
    n = ctypes.c_size_t(0)
    _check(_lib.msa_extend_workspace_size(num_seqs, ctypes.byref(n)), "msa_extend_workspace_size")
    return int(n.value)


def extend_workspace(num_seqs: int, device="cuda") -> torch.Tensor:
    """A device buffer for msa_extend_block_table over batches of ``num_seqs`` sequences."""
    return torch.empty(msa_extend_workspace_size(num_seqs), dtype=torch.uint8, device=device)


def _out(t, dtype, shape, dev, name):
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _is(t, dtype, shape, dev, name)


def msa_extend_block_table(lengths, new_tokens, free_pages, block_table, capacity: int, taken=None, new_lengths=None,
                           num_pages: int = (1 << 24) - 1, cu_q=None, cu_k=None, slots=None, positions=None,
                           taken_out=None, ws=None):
    """Pages for the new tokens of a batch: ``lengths`` and ``new_tokens`` int32 [num_seqs], ``free_pages`` int32 (the
    first ``taken`` [1] of which are gone), ``block_table`` int32 [num_seqs, max_blocks], whose entries of the new blocks
    are written.  Returns (cu_q, cu_k, slots int64 [capacity], positions int32 [capacity], taken_out int32 [1]): the grown
    batch's prefix sums, and each new token's cache row (-1 past the last token) and place in its sequence.
    ``new_lengths`` (may be ``lengths``) and ``taken_out`` (may be ``taken``) let a captured step advance by itself.
    Workspace: extend_workspace."""
    _int32(capacity, "capacity")
    _int32(num_pages, "num_pages")
    if not lengths.is_cuda:
        _need(lengths, torch.int32, "lengths")
    dev = _current_device()
    S = lengths.numel()
    at_len, at_new = _is(lengths, torch.int32, (S,), dev, "lengths"), _is(new_tokens, torch.int32, (S,), dev, "new_tokens")
    at_free = _is(free_pages, torch.int32, (free_pages.numel(),), dev, "free_pages")
    at_table = _table(block_table, S, dev, "block_table")
    at_taken = None if taken is None else _is(taken, torch.int32, (1,), dev, "taken")
    at_grown = None if new_lengths is None else _is(new_lengths, torch.int32, (S,), dev, "new_lengths")
    room = max(capacity, 0)
    cu_q, at_q = _out(cu_q, torch.int32, (S + 1,), dev, "cu_q")
    cu_k, at_k = _out(cu_k, torch.int32, (S + 1,), dev, "cu_k")
    slots, at_slots = _out(slots, torch.int64, (room,), dev, "slots")
    positions, at_pos = _out(positions, torch.int32, (room,), dev, "positions")
    taken_out, at_out = _out(taken_out, torch.int32, (1,), dev, "taken_out")
    ws, at_ws, nws = _space(ws, lambda: msa_extend_workspace_size(S), dev)
    status = _lib.msa_extend_block_table(S, at_len, at_new, capacity, at_free, free_pages.numel(), at_taken, num_pages,
                                         at_table, block_table.shape[1], at_grown, at_q, at_k, at_slots, at_pos, at_out,
                                         at_ws, nws, _raw_stream(dev))
    if status:
        raise MsaError(status, "msa_extend_block_table")
    return cu_q, cu_k, slots, positions, taken_out


def msa_append_workspace_size(num_pages: int) -> int:
    _int32(num_pages, "num_pages")
    n = ctypes.c_size_t(0)
    _check(_lib.msa_append_workspace_size(num_pages, ctypes.byref(n)), "msa_append_workspace_size")
    return int(n.value)


def append_workspace(num_pages: int, device="cuda") -> torch.Tensor:
    """A device buffer for msa_append_paged_fp8 (and msa_append_paged, which needs none) over caches of ``num_pages``."""
    return torch.empty(msa_append_workspace_size(num_pages), dtype=torch.uint8, device=device)


def _rows(t, tokens, inner, dev, name):
    """The address and token stride of new rows: contiguous but for the distance between tokens."""
    if t.dtype is torch.bfloat16 and t.get_device() == dev and t.shape == (tokens, *inner):
        strides, n = t.stride(), 1
        if tokens > 1 and strides[-1] == 1 and (len(inner) == 1 or strides[1] == 128):  # (a head's row has 128)
            return t.data_ptr(), strides[0]
        for size, stride in zip(inner[::-1], strides[:0:-1]):
            if stride != n and size != 1:
                raise ValueError(f"{name}: a token's row must be contiguous, got strides {list(strides)}")
            n *= size
        return t.data_ptr(), n if tokens <= 1 else strides[0]
    if t.dtype is not torch.bfloat16 or not t.is_cuda:
        _need(t, torch.bfloat16, name)
    _refuse(t.contiguous(), torch.bfloat16, (tokens, *inner), dev, name)


def _append(where, k, v, slots, k_cache, v_cache, scales, k_idx, k_idx_cache, k_idx_scale, ws):
    if not slots.is_cuda:
        _need(slots, torch.int64, "slots")
    dev = _current_device()
    dtype = torch.uint8 if scales else torch.bfloat16
    N = slots.numel()
    at_slots = _is(slots, torch.int64, (N,), dev, "slots")
    if (k_idx is None) != (k_idx_cache is None):
        raise ValueError("k_idx and its cache come together")
    if k is None and v is None and k_cache is None and v_cache is None and k_idx is not None and not scales:
        rows, hkv = k_idx_cache.shape[0], 0
        if k_idx_cache.dim() != 2 or rows % 128:
            raise ValueError("the cache must be whole pages of 128 rows, [num_pages * 128, d_idx]")
        (at_k, stride_k), (at_v, stride_v), caches = (None, 0), (None, 0), (None, None)
    else:
        for t, name in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache")):
            if t is None:
                raise ValueError(f"{name}: needed (k, v and their caches are left out together, for bf16 k_idx alone)")
        if k_cache.dim() != 3 or k_cache.shape[0] % 128:
            raise ValueError("the caches must be whole pages of 128 rows, [num_pages * 128, num_kv_heads, 128]")
        rows, hkv = k_cache.shape[0], k_cache.shape[1]
        at_k, stride_k = _rows(k, N, (hkv, 128), dev, "k")
        at_v, stride_v = _rows(v, N, (hkv, 128), dev, "v")
        caches = (_is(k_cache, dtype, (rows, hkv, 128), dev, "k_cache"), _is(v_cache, dtype, (rows, hkv, 128), dev, "v_cache"))
    at_i, stride_i, at_ic, at_is, d = None, 0, None, None, 128
    if k_idx is not None:
        d = k_idx_cache.shape[-1]
        at_i, stride_i = _rows(k_idx, N, (d,), dev, "k_idx")
        at_ic = _is(k_idx_cache, dtype, (rows, 128 if scales else d), dev, "k_idx_cache")
    at_ws, nws = None, 0
    if scales:
        shape = (rows // 128, hkv)
        at_scales = (_is(scales[0], torch.float32, shape, dev, "k_scale"), _is(scales[1], torch.float32, shape, dev, "v_scale"))
        if k_idx is not None:
            if k_idx_scale is None:
                raise ValueError("k_idx_scale: needed with k_idx")
            at_is = _is(k_idx_scale, torch.float32, (rows // 128,), dev, "k_idx_scale")
        ws, at_ws, nws = _space(ws, lambda: msa_append_workspace_size(rows // 128), dev)
        status = _lib.msa_append_paged_fp8(at_k, stride_k, at_v, stride_v, at_i, stride_i, at_slots, N, hkv, *caches,
                                           *at_scales, at_ic, at_is, rows // 128, at_ws, nws, _raw_stream(dev))
    else:
        if ws is not None:
            ws, at_ws, nws = _space(ws, None, dev)
        status = _lib.msa_append_paged(at_k, stride_k, at_v, stride_v, at_i, stride_i, at_slots, N, hkv, d, *caches, at_ic,
                                       rows // 128, at_ws, nws, _raw_stream(dev))
    if status:
        raise MsaError(status, where)


def msa_append_paged(k, v, slots, k_cache, v_cache, k_idx=None, k_idx_cache=None, ws=None):
    """Writes new tokens' rows k, v [tokens, Hkv, 128] (and k_idx [tokens, d_idx]), which may be slices of wider rows, to
    rows ``slots`` (int64, distinct, -1: none) of the caches.  k, v and their caches may all be None: k_idx alone (bf16 index
    pages beside K and V in E4M3 pages).  ``ws`` (256 bytes) is for device flags only."""
    _append("msa_append_paged", k, v, slots, k_cache, v_cache, None, k_idx, k_idx_cache, None, ws)


def msa_append_paged_fp8(k, v, slots, k8_cache, v8_cache, k_scale, v_scale, k_idx=None, k_idx8_cache=None,
                         k_idx_scale=None, ws=None):
    """msa_append_paged into E4M3 pages: k_scale / v_scale [num_pages, Hkv] (k_idx_scale [num_pages]) grow where the new
    rows need it, and the rows that a page holds already are then rounded again.  A page's tokens follow one another in
    ``slots``.  Workspace: append_workspace."""
    _append("msa_append_paged_fp8", k, v, slots, k8_cache, v8_cache, (k_scale, v_scale), k_idx, k_idx8_cache, k_idx_scale,
            ws)


# ---------------------------------------------------------------- fp8 K/V
def fp8_scale_rows(problem: Problem) -> int:
    """Rows to allocate for a scale array: total_k / 128 + num_seqs bounds the number of key blocks."""
    return problem.total_k // problem.block + problem.num_seqs


def msa_quantize_kv_fp8(problem: Problem, k, v, k8=None, v8=None, k_scale=None, v_scale=None, ws=None):
    """bf16 K, V -> E4M3 codes (uint8, same shape) and fp32 scales [key blocks, Hkv] (rows past the sequences'
    key blocks are left as they were).  Returns (k8, v8, k_scale, v_scale)."""
    _need(k, torch.bfloat16, "k")
    _need(v, torch.bfloat16, "v")
    dev = k.device
    if k8 is None:
        k8 = torch.empty(k.shape, dtype=torch.uint8, device=dev)
    if v8 is None:
        v8 = torch.empty(v.shape, dtype=torch.uint8, device=dev)
    rows = (fp8_scale_rows(problem), problem.hkv)
    if k_scale is None:
        k_scale = torch.zeros(rows, dtype=torch.float32, device=dev)
    if v_scale is None:
        v_scale = torch.zeros(rows, dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.QUANTIZE_KV_FP8, ws)
    _check(_lib.msa_quantize_kv_fp8(ctypes.byref(problem.c()), _ptr(k), _ptr(v), _ptr(k8), _ptr(v8), _ptr(k_scale),
                                    _ptr(v_scale), _ptr(ws), nws, _stream()), "msa_quantize_kv_fp8")
    return k8, v8, k_scale, v_scale


def _attn_fp8(fn, op, where, problem, q, k8, v8, k_scale, v_scale, idx, o, lse, ws):
    _need(q, torch.bfloat16, "q")
    _need(k8, torch.uint8, "k8")
    _need(v8, torch.uint8, "v8")
    _need(k_scale, torch.float32, "k_scale")
    _need(v_scale, torch.float32, "v_scale")
    _need(idx, torch.int32, "idx")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=q.device)
    ws, nws = _ws(problem, op, ws)
    _check(fn(ctypes.byref(problem.c()), _ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale), _ptr(v_scale), _ptr(idx),
              _ptr(o), _ptr(lse), _ptr(ws), nws, _stream()), where)
    return o, lse


def msa_sparse_attn_prefill_fp8(problem: Problem, q, k8, v8, k_scale, v_scale, idx, o=None, lse=None, ws=None):
    return _attn_fp8(_lib.msa_sparse_attn_prefill_fp8, Op.SPARSE_ATTN_PREFILL_FP8, "msa_sparse_attn_prefill_fp8",
                     problem, q, k8, v8, k_scale, v_scale, idx, o, lse, ws)


def msa_sparse_attn_decode_fp8(problem: Problem, q, k8, v8, k_scale, v_scale, idx, o=None, lse=None, ws=None):
    return _attn_fp8(_lib.msa_sparse_attn_decode_fp8, Op.SPARSE_ATTN_DECODE_FP8, "msa_sparse_attn_decode_fp8",
                     problem, q, k8, v8, k_scale, v_scale, idx, o, lse, ws)


def msa_forward_fp8(problem: Problem, q, k8, v8, k_scale, v_scale, q_idx, k_idx, idx=None, o=None, lse=None,
                    ws=None):
    """msa_forward with fp8 K/V for the Main Branch.  Returns (idx, o, lse)."""
    for t, n in ((q, "q"), (q_idx, "q_idx"), (k_idx, "k_idx")):
        _need(t, torch.bfloat16, n)
    for t, n in ((k8, "k8"), (v8, "v8")):
        _need(t, torch.uint8, n)
    _need(k_scale, torch.float32, "k_scale")
    _need(v_scale, torch.float32, "v_scale")
    dev = q.device
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.FORWARD_FP8, ws)
    _check(_lib.msa_forward_fp8(ctypes.byref(problem.c()), _ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale), _ptr(v_scale),
                                _ptr(q_idx), _ptr(k_idx), _ptr(idx), _ptr(o), _ptr(lse), _ptr(ws), nws, _stream()),
           "msa_forward_fp8")
    return idx, o, lse


def msa_forward_decode_paged_fp8(problem: Problem, q, k8_cache, v8_cache, k_scale, v_scale, q_idx, k_idx_cache,
                                 block_table, idx=None, o=None, lse=None, ws=None):
    """Decode from paged fp8 caches: E4M3 codes [num_pages * 128, hkv, 128] with one scale row per page
    (k_scale / v_scale [num_pages, hkv]); bf16 q, q_idx and index-key cache; block_table int32
    [num_seqs, max_blocks].  Returns (idx, o, lse) as msa_forward."""
    for t, n in ((q, "q"), (q_idx, "q_idx"), (k_idx_cache, "k_idx_cache")):
        _need(t, torch.bfloat16, n)
    for t, n in ((k8_cache, "k8_cache"), (v8_cache, "v8_cache")):
        _need(t, torch.uint8, n)
    _need(k_scale, torch.float32, "k_scale")
    _need(v_scale, torch.float32, "v_scale")
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or k8_cache.shape[0] % 128:
        raise ValueError("block_table must be [num_seqs, max_blocks] and the caches whole pages of 128 rows")
    n_pages = k8_cache.shape[0] // 128
    if k_scale.numel() < n_pages * problem.hkv or v_scale.numel() < n_pages * problem.hkv:
        raise ValueError("k_scale and v_scale need one row of num_kv_heads scales per page")
    dev = q.device
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.FORWARD_FP8, ws)
    _check(_lib.msa_forward_decode_paged_fp8(ctypes.byref(problem.c()), _ptr(q), _ptr(k8_cache), _ptr(v8_cache),
                                             _ptr(k_scale), _ptr(v_scale), _ptr(q_idx), _ptr(k_idx_cache),
                                             _ptr(block_table), block_table.shape[1], n_pages, _ptr(idx), _ptr(o),
                                             _ptr(lse), _ptr(ws), nws, _stream()), "msa_forward_decode_paged_fp8")
    return idx, o, lse


def msa_quantize_index_fp8(problem: Problem, q_idx=None, k_idx=None, q_idx8=None, q_idx_scale=None, k_idx8=None,
                           k_idx_scale=None, ws=None):
    """bf16 Q_idx [total_q, Hkv, 128] and/or K_idx [total_k, 128] -> E4M3 codes (uint8, same shapes) with fp32
    scales: q_idx_scale [total_q, Hkv] (one per query row and group), k_idx_scale [key blocks] (one per key block
    of a sequence).  Either input may be None (that side is skipped and its outputs returned as None unless given).
    Returns (q_idx8, q_idx_scale, k_idx8, k_idx_scale)."""
    if q_idx is None and k_idx is None:
        raise ValueError("nothing to quantize: q_idx and k_idx are both None")
    if q_idx is not None:
        _need(q_idx, torch.bfloat16, "q_idx")
        dev = q_idx.device
        if q_idx8 is None:
            q_idx8 = torch.empty(q_idx.shape, dtype=torch.uint8, device=dev)
        if q_idx_scale is None:
            q_idx_scale = torch.empty(q_idx.shape[:2], dtype=torch.float32, device=dev)
    if k_idx is not None:
        _need(k_idx, torch.bfloat16, "k_idx")
        dev = k_idx.device
        if k_idx8 is None:
            k_idx8 = torch.empty(k_idx.shape, dtype=torch.uint8, device=dev)
        if k_idx_scale is None:
            k_idx_scale = torch.zeros(fp8_scale_rows(problem), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.QUANTIZE_INDEX_FP8, ws)
    _check(_lib.msa_quantize_index_fp8(ctypes.byref(problem.c()), _ptr(q_idx), _ptr(k_idx),
                                       _ptr(q_idx8 if q_idx is not None else None),
                                       _ptr(q_idx_scale if q_idx is not None else None),
                                       _ptr(k_idx8 if k_idx is not None else None),
                                       _ptr(k_idx_scale if k_idx is not None else None), _ptr(ws), nws, _stream()),
           "msa_quantize_index_fp8")
    return q_idx8, q_idx_scale, k_idx8, k_idx_scale


def _need_fp8_index(q_idx8, q_idx_scale, k_idx8, k_idx_scale):
    _need(q_idx8, torch.uint8, "q_idx8")
    _need(k_idx8, torch.uint8, "k_idx8")
    _need(q_idx_scale, torch.float32, "q_idx_scale")
    _need(k_idx_scale, torch.float32, "k_idx_scale")


def msa_index_pool_fp8(problem: Problem, q_idx8, q_idx_scale, k_idx8, k_idx_scale, pooled=None, ws=None):
    """msa_index_pool over fp8 index inputs: pooled fp32 [total_q * hkv, ceil(max_k / 128)] (entries past a row's
    causal end are left as they were, NaN when ``pooled`` is allocated here)."""
    _need_fp8_index(q_idx8, q_idx_scale, k_idx8, k_idx_scale)
    if pooled is None:
        pooled = torch.full((problem.total_q * problem.hkv, max_blocks(problem)), float("nan"), dtype=torch.float32,
                            device=q_idx8.device)
    ws, nws = _ws(problem, Op.INDEX_POOL, ws)
    _check(_lib.msa_index_pool_fp8(ctypes.byref(problem.c()), _ptr(q_idx8), _ptr(q_idx_scale), _ptr(k_idx8),
                                   _ptr(k_idx_scale), _ptr(pooled), pooled.stride(0), _ptr(ws), nws, _stream()),
           "msa_index_pool_fp8")
    return pooled


def msa_index_topk_fp8(problem: Problem, q_idx8, q_idx_scale, k_idx8, k_idx_scale, idx=None, ws=None):
    """msa_index_topk over fp8 index inputs.  Returns idx [total_q, Hkv, topk] int32."""
    _need_fp8_index(q_idx8, q_idx_scale, k_idx8, k_idx_scale)
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=q_idx8.device)
    _need(idx, torch.int32, "idx")
    ws, nws = _ws(problem, Op.INDEX_TOPK, ws)
    _check(_lib.msa_index_topk_fp8(ctypes.byref(problem.c()), _ptr(q_idx8), _ptr(q_idx_scale), _ptr(k_idx8),
                                   _ptr(k_idx_scale), _ptr(idx), _ptr(ws), nws, _stream()), "msa_index_topk_fp8")
    return idx


def msa_forward_fp8_index(problem: Problem, q, k8, v8, k_scale, v_scale, q_idx8, q_idx_scale, k_idx8, k_idx_scale,
                          idx=None, o=None, lse=None, ws=None):
    """msa_forward_fp8 with the Index Branch on fp8 inputs too.  Returns (idx, o, lse)."""
    _need(q, torch.bfloat16, "q")
    for t, n in ((k8, "k8"), (v8, "v8")):
        _need(t, torch.uint8, n)
    _need(k_scale, torch.float32, "k_scale")
    _need(v_scale, torch.float32, "v_scale")
    _need_fp8_index(q_idx8, q_idx_scale, k_idx8, k_idx_scale)
    dev = q.device
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.FORWARD_FP8, ws)
    _check(_lib.msa_forward_fp8_index(ctypes.byref(problem.c()), _ptr(q), _ptr(k8), _ptr(v8), _ptr(k_scale),
                                      _ptr(v_scale), _ptr(q_idx8), _ptr(q_idx_scale), _ptr(k_idx8), _ptr(k_idx_scale),
                                      _ptr(idx), _ptr(o), _ptr(lse), _ptr(ws), nws, _stream()),
           "msa_forward_fp8_index")
    return idx, o, lse


def msa_forward_decode_paged_fp8_index(problem: Problem, q, k8_cache, v8_cache, k_scale, v_scale, q_idx8,
                                       q_idx_scale, k_idx8_cache, k_idx_scale, block_table, idx=None, o=None,
                                       lse=None, ws=None):
    """Decode from paged fp8 caches with the index keys in fp8 too: K/V codes [num_pages * 128, hkv, 128] with
    scales [num_pages, hkv]; index-key codes [num_pages * 128, 128] with scales [num_pages]; q_idx8 / q_idx_scale
    for the queries; block_table int32 [num_seqs, max_blocks].  Returns (idx, o, lse) as msa_forward."""
    _need(q, torch.bfloat16, "q")
    for t, n in ((k8_cache, "k8_cache"), (v8_cache, "v8_cache")):
        _need(t, torch.uint8, n)
    _need(k_scale, torch.float32, "k_scale")
    _need(v_scale, torch.float32, "v_scale")
    _need_fp8_index(q_idx8, q_idx_scale, k_idx8_cache, k_idx_scale)
    _need(block_table, torch.int32, "block_table")
    if block_table.dim() != 2 or k8_cache.shape[0] % 128 or k_idx8_cache.shape[0] != k8_cache.shape[0]:
        raise ValueError("block_table must be [num_seqs, max_blocks] and the caches whole pages of 128 rows")
    n_pages = k8_cache.shape[0] // 128
    if k_scale.numel() < n_pages * problem.hkv or v_scale.numel() < n_pages * problem.hkv or \
            k_idx_scale.numel() < n_pages:
        raise ValueError("the scale arrays need one row per page")
    dev = q.device
    if idx is None:
        idx = torch.empty((problem.total_q, problem.hkv, problem.topk), dtype=torch.int32, device=dev)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((problem.total_q, problem.hq), dtype=torch.float32, device=dev)
    ws, nws = _ws(problem, Op.FORWARD_FP8, ws)
    _check(_lib.msa_forward_decode_paged_fp8_index(
        ctypes.byref(problem.c()), _ptr(q), _ptr(k8_cache), _ptr(v8_cache), _ptr(k_scale), _ptr(v_scale), _ptr(q_idx8),
        _ptr(q_idx_scale), _ptr(k_idx8_cache), _ptr(k_idx_scale), _ptr(block_table), block_table.shape[1], n_pages,
        _ptr(idx), _ptr(o), _ptr(lse), _ptr(ws), nws, _stream()), "msa_forward_decode_paged_fp8_index")
    return idx, o, lse


def msa_read_device_status(ws: Optional[torch.Tensor]) -> int:
    """MSA_DEVICE_* flags of the last call on workspace ``ws`` (None: of the last
    msa_sparse_attn_decode_static call on the current device).  Synchronises the stream."""
    flags = ctypes.c_uint32(0)
    _check(_lib.msa_read_device_status(_ptr(ws), ctypes.byref(flags), _stream()), "msa_read_device_status")
    return int(flags.value)


def abi_version() -> int:
    return int(_lib.msa_abi_version())


def kernel_launch_count() -> int:
    """Kernels (and memsets) the library has enqueued in this process."""
    return int(_lib.msa_kernel_launch_count())


class StageTimer:
    """Per-stage CUDA events recorded by the library on the call's stream.

    Use as a context manager around calls; ``elapsed_ms()`` after a
    synchronize gives {stage: ms} for the stages of the last call.
    """

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * len(STAGES))]
        s = torch.cuda.current_stream()
        for e in self.events:      # materialise the underlying cudaEvent_t handles
            e.record(s)
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])
        self.marks = set()

    def __enter__(self):
        _check(_lib.msa_set_stage_events(self._arr), "msa_set_stage_events")
        return self

    def __exit__(self, *exc):
        _lib.msa_set_stage_events(None)
        return False

    def elapsed_ms(self, stages=STAGES):
        out = {}
        for j, name in enumerate(STAGES):
            if name in stages:
                try:
                    out[name] = self.events[2 * j].elapsed_time(self.events[2 * j + 1])
                except RuntimeError:
                    pass
        return out
