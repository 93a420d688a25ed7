// evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head) with n cached keys, budget b and window r <= b: when
// n <= b every slot is kept; else the last r slots and, of the n - r others, the
// b - r with the largest weight (equal weights to the lower slot, NaN below
// everything).  The kept slots, in their order, become slots 0 .. min(n, b) - 1
// of the sequence's pages in a second block table.
//
// Two kernels: the selection reads each weight a few times from L2 (4 bytes a
// cached key), the gather reads and writes each kept key's K and V rows once
// (512 bytes in bf16) and bounds the call.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

constexpr int kSelThreads = 1024;
constexpr uint32_t kMarkNew = 256u;  // page marks: 1 = a page of the batch's table, + 256 per entry of the new one

// Larger key = larger weight; -0 = +0; NaN below -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of v over the CTA's threads before this one; `total` gets the sum over all.  sm: 33 words.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t& total, uint32_t* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // sm free
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  uint32_t w = sm[lane];  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const uint32_t before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) & 31);
  return incl - v + (warp ? before : 0u);
}

// One CTA per (sequence, KV head).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t sm[33];
  __shared__ uint32_t pick[2];
  const int t = threadIdx.x;
  const int s = blockIdx.x / p.hkv, g = blockIdx.x % p.hkv;

  // every CTA checks all lengths: a call whose lengths are wrong is skipped as a whole
  bool bad = t == 0 && (p.cu_k[0] != 0 || p.cu_k[p.num_seqs] != p.total_k);
  for (int i = t; i < p.num_seqs; i += kSelThreads) {
    const int a = p.cu_k[i], b = p.cu_k[i + 1];
    bad |= a < 0 || b < a || b - a > p.max_k;
  }
  if (__syncthreads_or(bad)) {
    if (t == 0 && blockIdx.x == 0) atomicOr(&p.hdr->status, kFlagBadSeqlens);
    return;
  }
  if (blockIdx.x == 0) {  // prefix sums of the new lengths
    uint32_t base = 0;
    for (int i0 = 0; i0 < p.num_seqs; i0 += kSelThreads) {
      const int i = i0 + t;
      const uint32_t n = i < p.num_seqs ? min(p.cu_k[i + 1] - p.cu_k[i], p.budget) : 0;
      uint32_t total;
      const uint32_t before = block_exclusive(n, total, sm);
      if (i < p.num_seqs) p.new_cu_k[i + 1] = static_cast<int32_t>(base + before + n);
      base += total;
    }
    if (t == 0) p.new_cu_k[0] = 0;
  }

  const int n = p.cu_k[s + 1] - p.cu_k[s], m = min(n, p.budget);
  if (g == 0) {
    for (int b = t; b < (n + kBlock - 1) / kBlock; b += kSelThreads) {
      const int e = p.block_table[static_cast<long long>(s) * p.bt_stride + b];
      if (e >= 0 && e < p.n_pages) atomicOr(&p.marks[e], 1u);
    }
    for (int b = t; b < (m + kBlock - 1) / kBlock; b += kSelThreads) {
      const int e = p.new_table[static_cast<long long>(s) * p.new_stride + b];
      if (e >= 0 && e < p.n_pages) atomicAdd(&p.marks[e], kMarkNew);
    }
  }

  const float* w = p.weight + (static_cast<long long>(s) * p.hkv + g) * p.weight_stride;
  float* nw = p.new_weight + (static_cast<long long>(s) * p.hkv + g) * p.new_weight_stride;
  int32_t* kept = p.kept + (static_cast<long long>(s) * p.hkv + g) * p.budget;
  for (int i = m + t; i < p.budget; i += kSelThreads) kept[i] = -1;
  if (n <= p.budget) {
    for (int i = t; i < n; i += kSelThreads) {
      kept[i] = i;
      nw[i] = w[i];
    }
    return;
  }
  const int free_n = n - p.recent, take = p.budget - p.recent;  // free_n > take

  // radix select of the take-th largest key: 11, 11 and 10 bits from the top
  uint32_t prefix = 0, mask = 0;
  uint32_t want = take;  // how many of the keys with this prefix are taken
  if (take > 0) {
    const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = shifts[pass], bins = 1 << bits[pass];
      for (int i = t; i < bins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = t; i < free_n; i += kSelThreads) {
        const uint32_t k = weight_key(w[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // thread t takes the bins from the top: bins - 1 - (2 t) and the one below (one bin for 10 bits)
      const int per = bins / kSelThreads;
      const int top = bins - 1 - per * t;
      const uint32_t c0 = hist[top], c1 = per > 1 ? hist[top - 1] : 0u;
      uint32_t total;
      const uint32_t above = block_exclusive(c0 + c1, total, sm);
      if (above < want && want <= above + c0 + c1) {
        const bool second = want > above + c0;
        pick[0] = second ? top - 1 : top;
        pick[1] = want - above - (second ? c0 : 0u);
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      want = pick[1];
      __syncthreads();
    }
  }

  // ordered compaction: keys above the threshold, the first `want` equal to it, and the window
  uint32_t base = 0, ties = 0;
  for (int i0 = 0; i0 < n; i0 += 4 * kSelThreads) {
    float v[4];
    uint32_t above = 0, equal = 0;  // bits
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 4 * t + j;
      v[j] = i < n ? w[i] : 0.0f;
      if (i < n) {
        if (i >= free_n) {
          above |= 1u << j;
        } else if (take > 0) {
          const uint32_t k = weight_key(v[j]);
          if (k > prefix) above |= 1u << j;
          if (k == prefix) equal |= 1u << j;
        }
      }
    }
    uint32_t total;
    const uint32_t x = block_exclusive(__popc(above) | (__popc(equal) << 16), total, sm);
    uint32_t na = base + (x & 0xFFFFu), ne = ties + (x >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool a = (above >> j) & 1u, e = (equal >> j) & 1u;
      if (a || (e && ne < want)) {
        const uint32_t at = na + min(ne, want);
        kept[at] = i0 + 4 * t + j;
        nw[at] = v[j];
      }
      na += a;
      ne += e;
    }
    base += total & 0xFFFFu;
    ties += total >> 16;
  }
}

// Checks one entry of the new table: inside the cache, not a page of the batch's own table and named once.
__device__ __forceinline__ bool new_page_fine(const EvictParams& p, int page) {
  return page >= 0 && page < p.n_pages && p.marks[page] == kMarkNew;
}

__device__ __forceinline__ void flag_page(const EvictParams& p, int page) {
  if (atomicCAS(&p.hdr->bad_site, 0u, 602u) == 0u) {
    p.hdr->bad_index = page;
    p.hdr->bad_bound = p.n_pages;
  }
  atomicOr(&p.hdr->status, kFlagBadIndex);
}

// Source rows of a new page's slots for up to kHeads heads; -1 for a page outside the cache (reads as zeros).
constexpr int kHeads = 8;
constexpr int kGatherThreads = 256;

__device__ __forceinline__ void source_rows(const EvictParams& p, int s, int page_slot, int rows, int h0, int heads,
                                            int n, int (*src)[kBlock]) {
  for (int i = threadIdx.x; i < heads * kBlock; i += kGatherThreads) {
    const int h = i / kBlock, r = i % kBlock;
    if (r >= rows) continue;
    const int slot =
        p.kept[(static_cast<long long>(s) * p.hkv + h0 + h) * p.budget + static_cast<long long>(page_slot) * kBlock + r];
    int row = -1;
    if (slot >= 0 && slot < n) {
      const int e = p.block_table[static_cast<long long>(s) * p.bt_stride + slot / kBlock];
      if (e >= 0 && e < p.n_pages) row = e * kBlock + slot % kBlock;
      else flag_page(p, e);
    }
    src[h][r] = row;
  }
}

// CTA (sequence, page of the new table, 8 heads), bf16: warp per row, K in the lower half of the lanes, V in the upper.
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(EvictParams p) {
  __shared__ int src[kHeads][kBlock];
  griddep_wait();
  if (p.hdr->status & kFlagBadSeqlens) return;
  const int s = blockIdx.x / p.new_blocks, b = blockIdx.x % p.new_blocks;
  const int n = p.cu_k[s + 1] - p.cu_k[s], m = min(n, p.budget);
  const int rows = min(kBlock, m - b * kBlock);
  if (rows <= 0) return;
  const int page = p.new_table[static_cast<long long>(s) * p.new_stride + b];
  if (!new_page_fine(p, page)) {
    if (threadIdx.x == 0) flag_page(p, page);
    return;
  }
  const int h0 = blockIdx.y * kHeads, heads = min(kHeads, p.hkv - h0);
  source_rows(p, s, b, rows, h0, heads, n, src);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint4* cache = reinterpret_cast<uint4*>(lane < 16 ? p.k : p.v);
  const int col = lane & 15;
  const int items = rows * heads;
#pragma unroll 4
  for (int i = warp; i < items; i += kGatherThreads / 32) {
    const int r = i / heads, h = i % heads;
    const int from = src[h][r];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (from >= 0) v = cache[(static_cast<long long>(from) * p.hkv + h0 + h) * 16 + col];
    cache[((static_cast<long long>(page) * kBlock + r) * p.hkv + h0 + h) * 16 + col] = v;
  }
}

// fp8: a new page has one scale per head, so its rows are gathered, their
// largest value taken, and the codes rounded again.  A value is code * scale of
// its old page, the new code the rounding of code * ratio with ratio = old scale
// * 448 / max.  Codes and scales of few significant bits meet midpoints of
// E4M3 exactly, so the product is rounded once and from more bits than fp32's;
// a page that keeps its largest value keeps its codes.
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {  // of two codes
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
}

// x * (hi + lo), x and hi >= 0, as a float that rounds to fewer bits the way the exact product does: truncated, with
// the lowest bit set when that left something.  hi + lo has 45 bits or more; the product of a code (4 bits) and a
// quotient of (24-bit scale * 448) by (4-bit code * 24-bit scale) is a midpoint or at least 2^-33 of itself away
// from one, so a remainder below 2^-40 is none.
__device__ __forceinline__ float mul_to_odd(float x, float hi, float lo) {
  const float q0 = x * hi, e0 = fmaf(x, lo, fmaf(x, hi, -q0));
  const float q = q0 + e0, e = e0 - (q - q0);  // |e| at most half a step of q
  if (!(fabsf(e) > q * 0x1p-40f)) return q;  // NaN too
  return __uint_as_float((e < 0.0f ? __float_as_uint(q) - 1u : __float_as_uint(q)) | 1u);
}

struct PageScale {
  unsigned long long key[kGatherThreads / 32];
  float inv_hi, inv_lo;  // 448 / max
};

template <bool V>
__device__ __forceinline__ void gather_fp8(const EvictParams& p, int page, int rows, int h, const int* src,
                                           PageScale& sm) {
  const uint4* cache = reinterpret_cast<const uint4*>(V ? p.v : p.k);
  float* scales = V ? p.v_scale : p.k_scale;
  uint4 c[4];
  float sc[4];
  unsigned long long top = 0;  // largest |value|: the exact product of code and scale as two floats, by their bits
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 128 rows x 8 chunks of 16 codes over 256 threads
    const int at = i * kGatherThreads + threadIdx.x, r = at >> 3, col = at & 7;
    c[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0.0f;
    if (r < rows && src[r] >= 0) {
      c[i] = cache[(static_cast<long long>(src[r]) * p.hkv + h) * 8 + col];
      sc[i] = scales[static_cast<long long>(src[r] / kBlock) * p.hkv + h];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    uint32_t m = 0;  // largest |code|, NaN (0x7F) left out
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = w[j] & 0x7F7F7F7Fu;
      m = __vmaxu4(m, a & ~__vcmpeq4(a, 0x7F7F7F7Fu));
    }
    m = max(max(m & 0xFFu, (m >> 8) & 0xFFu), max((m >> 16) & 0xFFu, m >> 24));
    const float x = e4m3_values(m).x;
    const float hi = __fmul_rz(x, sc[i]), lo = fmaf(x, sc[i], -hi);  // lo >= 0
    const unsigned long long key = (static_cast<unsigned long long>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
    top = key > top ? key : top;
  }
  top = warp_max_u64(top);
  if ((threadIdx.x & 31) == 0) sm.key[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kGatherThreads / 32; ++w) top = sm.key[w] > top ? sm.key[w] : top;
    const double value = static_cast<double>(__uint_as_float(static_cast<uint32_t>(top >> 32))) +
                         static_cast<double>(__uint_as_float(static_cast<uint32_t>(top)));
    const bool some = value >= 0x1p-118;  // below, 448 / value is no fp32 number: codes 0
    scales[static_cast<long long>(page) * p.hkv + h] = some ? static_cast<float>(value / 448.0) : 1.0f;
    const double inv = some ? 448.0 / value : 0.0;
    sm.inv_hi = static_cast<float>(inv);
    sm.inv_lo = static_cast<float>(inv - static_cast<double>(sm.inv_hi));
  }
  __syncthreads();
  const float ih = sm.inv_hi, il = sm.inv_lo;
  uint4* out = reinterpret_cast<uint4*>(V ? p.v : p.k);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i * kGatherThreads + threadIdx.x, r = at >> 3, col = at & 7;
    if (r >= rows) continue;
    float hi = sc[i] * ih, lo = fmaf(sc[i], il, fmaf(sc[i], ih, -hi));
    if (!(hi < 1e30f)) hi = 1e30f, lo = 0.0f;  // a scale so far above the values that their codes are 0
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    uint32_t q[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t pair = w[j >> 1] >> (16 * (j & 1));
      const float2 f = e4m3_values(pair & 0x7F7Fu);
      const float2 y = make_float2(mul_to_odd(f.x, hi, lo), mul_to_odd(f.y, hi, lo));
      const uint32_t code = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
      q[j >> 1] |= (code | (pair & 0x8080u)) << (16 * (j & 1));
    }
    out[((static_cast<long long>(page) * kBlock + r) * p.hkv + h) * 8 + col] = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_fp8_kernel(EvictParams p) {
  __shared__ int src[kHeads][kBlock];
  __shared__ PageScale scale[2];
  griddep_wait();
  if (p.hdr->status & kFlagBadSeqlens) return;
  const int s = blockIdx.x / p.new_blocks, b = blockIdx.x % p.new_blocks;
  const int n = p.cu_k[s + 1] - p.cu_k[s], m = min(n, p.budget);
  const int rows = min(kBlock, m - b * kBlock);
  if (rows <= 0) return;
  const int page = p.new_table[static_cast<long long>(s) * p.new_stride + b];
  if (!new_page_fine(p, page)) {
    if (threadIdx.x == 0) flag_page(p, page);
    return;
  }
  const int h0 = blockIdx.y * kHeads, heads = min(kHeads, p.hkv - h0);
  source_rows(p, s, b, rows, h0, heads, n, src);
  __syncthreads();
  for (int h = 0; h < heads; ++h) {
    gather_fp8<false>(p, page, rows, h0 + h, src[h], scale[0]);
    gather_fp8<true>(p, page, rows, h0 + h, src[h], scale[1]);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, bool fp8, cudaStream_t stream) {
  // the header's status and the marks behind it start at zero
  cudaError_t e = cudaMemsetAsync(p.hdr, 0, p.clear_bytes, stream);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<p.num_seqs * p.hkv, kSelThreads, 0, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launches(2);
  if (p.new_blocks == 0) return cudaSuccess;  // no cached key anywhere
  const dim3 grid(static_cast<unsigned>(p.num_seqs) * p.new_blocks, (p.hkv + kHeads - 1) / kHeads);
  e = launch_pdl(fp8 ? evict_gather_fp8_kernel : evict_gather_kernel, grid, dim3(kGatherThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaSuccess;
}

}  // namespace msa
