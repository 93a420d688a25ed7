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

// The first digit holds sign, exponent and two bits: the weights of a cache fall into a few dozen of its bins, so a
// warp's counts would meet in the same words.  Four lane groups count into copies of their own.
constexpr int kCopies = 4;

// A word of the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(smem_u32(p)), "r"(rank)
               : "memory");
  return v;
}

// A cluster of `cs` CTAs per (sequence, KV head), each over its share of the
// slots.  The threshold (the key of the last slot taken by weight) comes from
// three digits of a radix select; the CTAs' digit counts are added through
// distributed shared memory, and each CTA finds the same digit.  What lies above
// the threshold in a CTA's share follows from its own counts, so the kept slots
// are written in one more pass.  Every pass reads the weights from L2, 16 bytes a
// load, or from registers when a share fits them.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p, int cs) {
  __shared__ uint32_t hist[3][2048];
  __shared__ uint32_t spread[2048 * (kCopies - 1)];
  __shared__ uint32_t sm[33];
  __shared__ uint32_t pick[3][2];
  __shared__ uint32_t mine[2];  // kept for sure and equal to the threshold, in this CTA's share
  const int t = threadIdx.x;
  const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int row = blockIdx.x / cs, s = row / p.hkv, g = row % p.hkv;
  auto sync_all = [&] {
    __syncwarp();  // the cluster barrier wants whole warps
    if (cs > 1) cluster_sync(); else __syncthreads();
  };

  // every CTA checks all lengths: a call whose lengths are wrong is skipped as a whole
  bool bad = t == 0 && (p.cu_k[0] != 0 || p.cu_k[p.num_seqs] != p.total_k);
  for (int i = t; i < p.num_seqs; i += kSelThreads) {
    const int a = p.cu_k[i], b = p.cu_k[i + 1];
    bad |= a < 0 || b < a || b - a > p.max_k;
  }
  for (int i = t; i < 3 * 2048; i += kSelThreads) hist[0][i] = 0;
  for (int i = t; i < 2048 * (kCopies - 1); i += kSelThreads) spread[i] = 0;
  uint32_t* const own_first = t % kCopies ? spread + (t % kCopies - 1) * 2048 : hist[0];
  if (__syncthreads_or(bad)) {
    if (t == 0 && blockIdx.x == 0) atomicOr(&p.hdr->status, kFlagBadSeqlens);
    return;  // the whole cluster
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
    const int at = rank * kSelThreads + t, step = cs * kSelThreads;
    for (int b = at; b < (n + kBlock - 1) / kBlock; b += step) {
      const int e = p.block_table[static_cast<long long>(s) * p.bt_stride + b];
      if (e >= 0 && e < p.n_pages) atomicOr(&p.marks[e], 1u);
    }
    for (int b = at; b < (m + kBlock - 1) / kBlock; b += step) {
      const int e = p.new_table[static_cast<long long>(s) * p.new_stride + b];
      if (e >= 0 && e < p.n_pages) atomicAdd(&p.marks[e], kMarkNew);
    }
  }

  const float* w = p.weight + static_cast<long long>(row) * p.weight_stride;
  float* nw = p.new_weight + static_cast<long long>(row) * p.new_weight_stride;
  int32_t* kept = p.kept + static_cast<long long>(row) * p.budget;
  for (int i = m + rank * kSelThreads + t; i < p.budget; i += cs * kSelThreads) kept[i] = -1;
  if (n <= p.budget) {  // uniform in the cluster
    for (int i = rank * kSelThreads + t; i < n; i += cs * kSelThreads) {
      kept[i] = i;
      nw[i] = w[i];
    }
    return;
  }
  const int free_n = n - p.recent, take = p.budget - p.recent;  // free_n > take

  // this CTA's slots [c0, c1), four at a time
  const int share = ((n + cs - 1) / cs + 3) & ~3;
  const int c0 = min(n, rank * share), c1 = min(n, c0 + share);
  const bool vec = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
  auto load4 = [&](int i) {  // slots i .. i + 3; past the share anything
    if (vec && i + 4 <= c1) return *reinterpret_cast<const float4*>(w + i);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < c1) v.x = w[i];
    if (i + 1 < c1) v.y = w[i + 1];
    if (i + 2 < c1) v.z = w[i + 2];
    if (i + 3 < c1) v.w = w[i + 3];
    return v;
  };
  const bool once = c1 - c0 <= 4 * kSelThreads;
  float4 held = make_float4(0.f, 0.f, 0.f, 0.f);
  if (once && c0 + 4 * t < c1) held = load4(c0 + 4 * t);

  uint32_t prefix = 0, mask = 0;
  uint32_t want = take;   // how many of the keys with this prefix are taken
  uint32_t above = 0;     // this thread's count of keys in the share that lie above the prefix
  uint32_t equal = 0;     // keys of the share equal to the threshold (after the last digit)
  if (take > 0) {
    const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
    const int end = min(c1, free_n);
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = shifts[pass], bins = 1 << bits[pass];
      auto count4 = [&](const float4& v, int i) {
        const float f[4] = {v.x, v.y, v.z, v.w};
        uint32_t* const counts = pass == 0 ? own_first : hist[pass];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t k = weight_key(f[j]);
          if (i + j < end && (k & mask) == prefix) atomicAdd(&counts[(k >> shift) & (bins - 1)], 1u);
        }
      };
      if (once) {
        count4(held, c0 + 4 * t);
      } else {
        int i = c0 + 4 * t;
        for (; i + 12 * kSelThreads < end; i += 16 * kSelThreads) {  // four loads in flight
          float4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = load4(i + 4 * u * kSelThreads);
#pragma unroll
          for (int u = 0; u < 4; ++u) count4(v[u], i + 4 * u * kSelThreads);
        }
        for (; i < end; i += 4 * kSelThreads) count4(load4(i), i);
      }
      if (pass == 0) {
        __syncthreads();
        for (int i = t; i < 2048; i += kSelThreads) hist[0][i] += spread[i] + spread[2048 + i] + spread[4096 + i];
      }
      sync_all();
      // thread t takes the bins from the top: bins - 1 - (2 t) and the one below (one bin for 10 bits)
      const int per = bins / kSelThreads;
      const int top = bins - 1 - per * t;
      const uint32_t own0 = hist[pass][top], own1 = per > 1 ? hist[pass][top - 1] : 0u;
      uint32_t n0 = own0, n1 = own1;
      for (int r = 0; r < cs; ++r) {
        if (r == rank) continue;
        n0 += cluster_word(&hist[pass][top], r);
        if (per > 1) n1 += cluster_word(&hist[pass][top - 1], r);
      }
      uint32_t total;
      const uint32_t before = block_exclusive(n0 + n1, total, sm);
      if (before < want && want <= before + n0 + n1) {
        const bool second = want > before + n0;
        pick[pass][0] = second ? top - 1 : top;
        pick[pass][1] = want - before - (second ? n0 : 0u);
      }
      __syncthreads();
      const int digit = static_cast<int>(pick[pass][0]);
      above += (top > digit ? own0 : 0u) + (per > 1 && top - 1 > digit ? own1 : 0u);
      equal = hist[pass][digit];
      prefix |= static_cast<uint32_t>(digit) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      want = pick[pass][1];
    }
  }
  // what the CTAs before this one keep
  uint32_t base = 0, ties = 0;
  if (cs > 1) {
    uint32_t total;
    block_exclusive(above, total, sm);
    if (t == 0) {
      mine[0] = total + max(0, c1 - max(c0, free_n));
      mine[1] = equal;
    }
    sync_all();
    for (int r = 0; r < rank; ++r) {
      base += cluster_word(&mine[0], r);
      ties += cluster_word(&mine[1], r);
    }
    sync_all();  // nobody leaves before its words are read
  }

  // ordered compaction: keys above the threshold, the first `want` equal to it, and the window
  for (int i0 = c0; i0 < c1; i0 += 4 * kSelThreads) {
    const int i = i0 + 4 * t;
    const float4 v4 = once ? held : (i < c1 ? load4(i) : make_float4(0.f, 0.f, 0.f, 0.f));
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
    uint32_t sure = 0, same = 0;  // bits
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j >= c1) continue;
      if (i + j >= free_n) {
        sure |= 1u << j;
      } else if (take > 0) {
        const uint32_t k = weight_key(v[j]);
        if (k > prefix) sure |= 1u << j;
        if (k == prefix) same |= 1u << j;
      }
    }
    uint32_t total;
    const uint32_t x = block_exclusive(__popc(sure) | (__popc(same) << 16), total, sm);
    uint32_t na = base + (x & 0xFFFFu), ne = ties + (x >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool a = (sure >> j) & 1u, e = (same >> j) & 1u;
      if (a || (e && ne < want)) {
        const uint32_t at = na + min(ne, want);
        kept[at] = i + j;
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

// Row of the cache that holds a kept slot; -1 for a page outside the cache (reads as zeros).
__device__ __forceinline__ int source_row(const EvictParams& p, int s, int n, long long kept_at) {
  const int slot = p.kept[kept_at];
  if (slot < 0 || slot >= n) return -1;
  const int e = p.block_table[static_cast<long long>(s) * p.bt_stride + slot / kBlock];
  if (e >= 0 && e < p.n_pages) return e * kBlock + slot % kBlock;
  flag_page(p, e);
  return -1;
}

// The new page that a CTA fills, from its number among the batch's; rows = 0: nothing to do.  The loads that do not
// wait for one another come first: the launch is a chain of dependent loads.
struct NewPage {
  int s, b, n, rows, page;
};
__device__ __forceinline__ NewPage new_page(const EvictParams& p, int number) {
  NewPage x;
  x.s = number / p.new_blocks;
  x.b = number % p.new_blocks;
  const uint32_t status = *reinterpret_cast<volatile uint32_t*>(&p.hdr->status);
  const int c0 = p.cu_k[x.s], c1 = p.cu_k[x.s + 1];
  x.page = p.new_table[static_cast<long long>(x.s) * p.new_stride + x.b];
  x.n = c1 - c0;
  x.rows = (status & kFlagBadSeqlens) ? 0 : max(0, min(kBlock, min(x.n, p.budget) - x.b * kBlock));
  return x;
}
// False, and the page reported, when the call may not write it.
__device__ __forceinline__ bool page_fine(const EvictParams& p, const NewPage& x) {
  if (new_page_fine(p, x.page)) return true;
  if (threadIdx.x == 0) flag_page(p, x.page);
  return false;
}

constexpr int kHeads = 8;
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 32;

// bf16: CTA (new page, 32 of its rows, 8 heads); a warp per row and head, K in
// the lower half of its lanes and V in the upper, eight rows in flight.
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(EvictParams p) {
  __shared__ int src[kGatherRows * kHeads];
  griddep_wait();
  const NewPage x = new_page(p, blockIdx.x / (kBlock / kGatherRows));
  const int r0 = blockIdx.x % (kBlock / kGatherRows) * kGatherRows, rows = min(kGatherRows, x.rows - r0);
  if (rows <= 0) return;
  const int h0 = blockIdx.y * kHeads, heads = min(kHeads, p.hkv - h0);
  const int items = rows * heads;  // row by row, as the caches lie
  if (threadIdx.x < items) {
    const int r = threadIdx.x / heads, h = threadIdx.x % heads;
    src[threadIdx.x] =
        source_row(p, x.s, x.n, (static_cast<long long>(x.s) * p.hkv + h0 + h) * p.budget + x.b * kBlock + r0 + r);
  }
  if (!page_fine(p, x)) return;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint4* cache = reinterpret_cast<uint4*>(lane < 16 ? p.k : p.v);
  const int col = lane & 15;
  const long long to = (static_cast<long long>(x.page) * kBlock + r0) * p.hkv + h0;
  constexpr int kFlight = 8, kStep = kGatherThreads / 32;
  for (int i0 = warp; i0 < items; i0 += kFlight * kStep) {
    uint4 v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int i = i0 + u * kStep;
      v[u] = make_uint4(0, 0, 0, 0);
      if (i < items && src[i] >= 0) v[u] = cache[(static_cast<long long>(src[i]) * p.hkv + h0 + i % heads) * 16 + col];
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int i = i0 + u * kStep;
      if (i < items) cache[(to + static_cast<long long>(i / heads) * p.hkv + i % heads) * 16 + col] = v[u];
    }
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

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
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

// One page and head of K or V in the CTA's registers: 128 rows x 8 chunks of 16 codes over 256 threads.
struct Codes {
  uint4 c[4];
  float sc[4];  // the old pages' scales
};

__device__ __forceinline__ void load_codes(const EvictParams& p, const void* cache, const float* scales, int rows, int h,
                                           const int* src, Codes& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i * kGatherThreads + threadIdx.x, r = at >> 3;
    x.c[i] = make_uint4(0, 0, 0, 0);
    x.sc[i] = 0.0f;
    if (r < rows && src[r] >= 0) {
      x.c[i] = static_cast<const uint4*>(cache)[(static_cast<long long>(src[r]) * p.hkv + h) * 8 + (at & 7)];
      x.sc[i] = scales[static_cast<long long>(src[r] / kBlock) * p.hkv + h];
    }
  }
}

// The thread's largest |value|: the exact product of code and scale as two floats, by their bits.
__device__ __forceinline__ unsigned long long largest(const Codes& x) {
  unsigned long long top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w};
    uint32_t m = 0;  // largest |code|, NaN (0x7F) left out
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = w[j] & 0x7F7F7F7Fu;
      m = __vmaxu4(m, a & ~__vcmpeq4(a, 0x7F7F7F7Fu));
    }
    m = max(max(m & 0xFFu, (m >> 8) & 0xFFu), max((m >> 16) & 0xFFu, m >> 24));
    const float v = e4m3_values(m).x;
    const float hi = __fmul_rz(v, x.sc[i]), lo = fmaf(v, x.sc[i], -hi);  // lo >= 0
    const unsigned long long key = (static_cast<unsigned long long>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
    top = key > top ? key : top;
  }
  return top;
}

__device__ __forceinline__ void store_codes(const EvictParams& p, void* cache, long long row0, int rows, int h,
                                            float inv_hi, float inv_lo, const Codes& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i * kGatherThreads + threadIdx.x, r = at >> 3;
    if (r >= rows) continue;
    float hi = x.sc[i] * inv_hi, lo = fmaf(x.sc[i], inv_lo, fmaf(x.sc[i], inv_hi, -hi));
    if (!(hi < 1e30f)) hi = 1e30f, lo = 0.0f;  // a scale so far above the values that their codes are 0
    // A product just below and one just above the exact one round alike unless a midpoint lies between: only then,
    // four codes at a time, the exact way.
    const float under = hi * (1.0f - 0x1p-21f), over = hi * (1.0f + 0x1p-21f);
    const uint32_t w[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w};
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3_values(w[j] & 0x7F7Fu), b = e4m3_values((w[j] >> 16) & 0x7F7Fu);
      q[j] = e4m3x4(a.x * under, a.y * under, b.x * under, b.y * under);
      if (q[j] != e4m3x4(a.x * over, a.y * over, b.x * over, b.y * over))
        q[j] = e4m3x4(mul_to_odd(a.x, hi, lo), mul_to_odd(a.y, hi, lo), mul_to_odd(b.x, hi, lo), mul_to_odd(b.y, hi, lo));
      q[j] |= w[j] & 0x80808080u;
    }
    static_cast<uint4*>(cache)[((row0 + r) * p.hkv + h) * 8 + (at & 7)] = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// CTA (new page, KV head).
__global__ void __launch_bounds__(kGatherThreads, 4) evict_gather_fp8_kernel(EvictParams p) {
  __shared__ int src[kBlock];
  __shared__ unsigned long long keys[2][kGatherThreads / 32];
  __shared__ float2 inv[2];  // 448 / max as two floats
  griddep_wait();
  const NewPage x = new_page(p, blockIdx.x);
  if (x.rows <= 0) return;
  const int h = blockIdx.y;
  if (threadIdx.x < x.rows)
    src[threadIdx.x] = source_row(p, x.s, x.n, (static_cast<long long>(x.s) * p.hkv + h) * p.budget + x.b * kBlock + threadIdx.x);
  if (!page_fine(p, x)) return;
  __syncthreads();
  Codes k, v;
  load_codes(p, p.k, p.k_scale, x.rows, h, src, k);
  load_codes(p, p.v, p.v_scale, x.rows, h, src, v);
  const unsigned long long tk = warp_max_u64(largest(k)), tv = warp_max_u64(largest(v));
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    keys[0][warp] = tk;
    keys[1][warp] = tv;
  }
  __syncthreads();
  if (threadIdx.x < 64 && (threadIdx.x & 31) == 0) {  // one thread each for K and V
    unsigned long long top = 0;
#pragma unroll
    for (int i = 0; i < kGatherThreads / 32; ++i) top = keys[warp][i] > top ? keys[warp][i] : top;
    const double value = static_cast<double>(__uint_as_float(static_cast<uint32_t>(top >> 32))) +
                         static_cast<double>(__uint_as_float(static_cast<uint32_t>(top)));
    const bool some = value >= 0x1p-118;  // below, 448 / value is no fp32 number: codes 0
    (warp ? p.v_scale : p.k_scale)[static_cast<long long>(x.page) * p.hkv + h] =
        some ? static_cast<float>(value / 448.0) : 1.0f;
    const double q = some ? 448.0 / value : 0.0;
    const float hi = static_cast<float>(q);
    inv[warp] = make_float2(hi, static_cast<float>(q - static_cast<double>(hi)));
  }
  __syncthreads();
  const long long row0 = static_cast<long long>(x.page) * kBlock;
  store_codes(p, p.k, row0, x.rows, h, inv[0].x, inv[0].y, k);
  store_codes(p, p.v, row0, x.rows, h, inv[1].x, inv[1].y, v);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, bool fp8, int sms, cudaStream_t stream) {
  // the header's status and the marks behind it start at zero
  cudaError_t e = cudaMemsetAsync(p.hdr, 0, p.clear_bytes, stream);
  if (e != cudaSuccess) return e;
  // CTAs per (sequence, head): one while those fill the GPU or a share would fall under 4,096 slots (one load per
  // thread, held in registers); up to eight for few long sequences
  int cs = 1;
  while (cs < 8 && 2ll * cs * p.num_seqs * p.hkv <= sms && p.max_k / (2 * cs) >= 4 * kSelThreads) cs *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * p.hkv * cs);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(cs), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cs);
  if (e != cudaSuccess) return e;
  note_launches(2);
  if (p.new_blocks == 0) return cudaSuccess;  // no cached key anywhere
  const unsigned pages = static_cast<unsigned>(p.num_seqs) * p.new_blocks;
  if (fp8)
    e = launch_pdl(evict_gather_fp8_kernel, dim3(pages, p.hkv), dim3(kGatherThreads), 0, stream, p);
  else
    e = launch_pdl(evict_gather_kernel, dim3(pages * (kBlock / kGatherRows), (p.hkv + kHeads - 1) / kHeads),
                   dim3(kGatherThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaSuccess;
}

}  // namespace msa
