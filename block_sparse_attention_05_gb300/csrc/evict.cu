// evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head) with n cached keys, budget b and window r <= b: when
// n <= b every slot is kept; else the last r slots and, of the n - r others, the
// b - r with the largest weight (equal weights to the lower slot, NaN below
// everything).  The kept slots, in their order, become slots 0 .. min(n, b) - 1
// of the sequence's pages in a second block table.
//
// Three kernels, set up under one another's ends: a clear of the workspace's
// header and page marks, the selection, which reads each weight once (4 bytes a
// cached key), and the gather, which reads and writes each kept key's K and V
// rows once (512 bytes in bf16) and bounds the call.  Measured: 12 sequences of
// 65,536 keys to 32,768 (4 KV heads, bf16) 273 us, 6.0 TB/s, of which the gather
// 241; the 12 in E4M3 226 us (123 for the bytes), 16 ragged ones of up to 9,001 to
// 4,096 in E4M3 39 to 41 us (13 for the bytes: the gather, which rounds every code
// again, 27); one of 700 to 512 16 us, three launches of dependent loads.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

constexpr int kSelThreads = 1024;
constexpr uint32_t kMarkNew = 256u;  // page marks: 1 = a page of the batch's table, + 256 per entry of the new one

// Larger key = larger weight; -0 = +0 (the addition makes them one); NaN below -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return w != w ? 0u : k;
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

// A word of the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(smem_u32(p)), "r"(rank));
  return v;
}

// The sum of a shared memory word over the cluster's other CTAs.
__device__ __forceinline__ uint32_t others(const uint32_t* p, int cs, int rank) {
  uint32_t v[7], sum = 0;  // all in flight at once
#pragma unroll
  for (int r = 1; r < 8; ++r) v[r - 1] = r < cs ? cluster_word(p, rank + r < cs ? rank + r : rank + r - cs) : 0u;
#pragma unroll
  for (int r = 0; r < 7; ++r) sum += v[r];
  return sum;
}

// The lane in which the sum of n over the lanes so far reaches `want` (some lane's does), which becomes what is wanted
// of that lane's n.  Called by a whole warp.
__device__ __forceinline__ int crossing_lane(uint32_t n, uint32_t& want) {
  const int lane = threadIdx.x & 31;
  uint32_t incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  const uint32_t reached = __ballot_sync(0xFFFFFFFFu, incl >= want);
  const int hit = reached ? __ffs(reached) - 1 : 31;
  want -= __shfl_sync(0xFFFFFFFFu, incl - n, hit);
  return hit;
}

// A cluster of `cs` CTAs per (sequence, KV head), each over its share of the
// slots.  The threshold (the key of the last slot taken by weight) comes from
// three digits of a radix select; the CTAs' digit counts are added through
// distributed shared memory, and each CTA finds the same digit.  What lies above
// the threshold in a CTA's share follows from its own counts, so the kept slots
// are written in one more pass.  Each weight is read once, a kept one again: its
// key stays in shared memory (CACHED, shares of up to kSelKeys slots; larger ones read the
// weights again for each pass).  What bounds it: 32,768 slots to a CTA take 5 us
// to read and count, 4 for each further digit (2 of them the exchange) and 10 for
// the compaction; 8,192 on each of eight CTAs 15 us in all.
constexpr int kSelKeys = 48 * 1024;
constexpr uint32_t kLate = 0xFFFFFFFFu;  // the key of a slot of the window: above every weight's

template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p, int cs) {
  extern __shared__ __align__(16) uint32_t keys[];  // CACHED: this CTA's share, in slot order
  __shared__ uint32_t hist[2 * 2048 + 1024];
  __shared__ uint32_t sm[33];
  __shared__ uint32_t coarse[3][32];  // counts of a digit's 32 groups of bins, the highest first
  __shared__ uint32_t pick[3][2];
  __shared__ __align__(8) uint32_t mine[2];  // kept for sure and equal to the threshold, in this CTA's share
  __shared__ uint32_t ahead[2];              // the same of the CTAs before this one
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int row = blockIdx.x / cs, s = row / p.hkv, g = row % p.hkv;
  auto sync_all = [&] {
    __syncwarp();  // the cluster barrier wants whole warps
    if (cs > 1) cluster_sync(); else __syncthreads();
  };

  griddep_wait();
  // every CTA checks all lengths: a call whose lengths are wrong is skipped as a whole
  bool bad = t == 0 && (p.cu_k[0] != 0 || p.cu_k[p.num_seqs] != p.total_k);
  for (int i = t; i < p.num_seqs; i += kSelThreads) {
    const int a = p.cu_k[i], b = p.cu_k[i + 1];
    bad |= a < 0 || b < a || b - a > p.max_k;
  }
  for (int i = t; i < 2 * 2048 + 1024; i += kSelThreads) hist[i] = 0;
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
  for (uint32_t i = m + rank * kSelThreads + t; i < static_cast<uint32_t>(p.budget); i += cs * kSelThreads)
    kept[i] = -1;  // unsigned: the index passes 2^31 on the way out when the budget is near it
  if (n <= p.budget) {  // uniform in the cluster
    for (int i = rank * kSelThreads + t; i < n; i += cs * kSelThreads) {
      kept[i] = i;
      nw[i] = w[i];
    }
    return;
  }
  const int free_n = n - p.recent, take = p.budget - p.recent;  // free_n > take

  // this CTA's slots [c0, c1), c0 a multiple of 16; those before `end` are chosen by weight
  const int share = ((n + cs - 1) / cs + 15) & ~15;
  const int c0 = min(n, rank * share), c1 = min(n, c0 + share);
  const int end = max(c0, min(c1, free_n));
  const bool vec = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
  // the keys of slots i .. i + 3; kLate in the window and past the share
  auto load4 = [&](int i) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (vec && i + 4 <= c1) {
      v = *reinterpret_cast<const float4*>(w + i);
    } else {
      if (i < c1) v.x = w[i];
      if (i + 1 < c1) v.y = w[i + 1];
      if (i + 2 < c1) v.z = w[i + 2];
      if (i + 3 < c1) v.w = w[i + 3];
    }
    return make_uint4(i < end ? weight_key(v.x) : kLate, i + 1 < end ? weight_key(v.y) : kLate,
                      i + 2 < end ? weight_key(v.z) : kLate, i + 3 < end ? weight_key(v.w) : kLate);
  };

  uint32_t prefix = kLate - 1, mask = 0;  // no weight counts when the window takes the whole budget
  uint32_t want = 0;                      // how many of the keys with this prefix are taken
  uint32_t above = 0;                     // this thread's count of keys in the share that lie above the prefix
  uint32_t equal = 0;                     // keys of the share equal to the threshold (after the last digit)
  if (CACHED && take == 0) {
    for (int i = c0 + 4 * t; i < c1; i += 4 * kSelThreads) *reinterpret_cast<uint4*>(keys + (i - c0)) = load4(i);
    __syncthreads();
  }
  if (take > 0) {
    prefix = 0;
    want = take;
    const int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = shifts[pass], bins = 1 << bits[pass];
      uint32_t* const counts = hist + 2048 * pass;
      auto count = [&](uint32_t k) {
        // the window's keys have all digits set, the first of them that of a NaN with its sign clear: no weight's
        if (pass == 0 ? k != kLate : (k & mask) == prefix) atomicAdd(&counts[(k >> shift) & (bins - 1)], 1u);
      };
      auto count4 = [&](const uint4& k) {
        count(k.x);
        count(k.y);
        count(k.z);
        count(k.w);
      };
      if (pass == 0 || !CACHED) {
        int i = c0 + 4 * t;
        for (; i + 12 * kSelThreads < c1; i += 16 * kSelThreads) {  // four loads in flight
          uint4 k[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) k[u] = load4(i + 4 * u * kSelThreads);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (CACHED) *reinterpret_cast<uint4*>(keys + (i - c0 + 4 * u * kSelThreads)) = k[u];
            count4(k[u]);
          }
        }
        for (; i < c1; i += 4 * kSelThreads) {
          const uint4 k = load4(i);
          if (CACHED) *reinterpret_cast<uint4*>(keys + (i - c0)) = k;
          count4(k);
        }
      } else {
#pragma unroll 2
        for (int i = 4 * t; i < c1 - c0; i += 4 * kSelThreads) count4(*reinterpret_cast<const uint4*>(keys + i));
      }
      // The digit where the taken keys end, counted from the top.  One CTA or two: a thread for one or two bins.  More:
      // first the digit's group of bins, then the bin, both found by warp 0 from the counts of all CTAs, a word or two
      // per lane and CTA (reading every bin of seven other CTAs took 3.5 us a digit: 21 us for 65,536 slots on eight
      // CTAs, now 15; on two CTAs the groups take 1 us longer than 28).
      const bool by_group = cs > 2;
      const int in_group = bins / 32;  // 64 or 32
      uint32_t own0 = 0, own1 = 0;
      int top = 0;
      if (!by_group) {
        sync_all();
        const int per = bins / kSelThreads;
        top = bins - 1 - per * t;
        own0 = counts[top];
        own1 = per > 1 ? counts[top - 1] : 0u;
        uint32_t n0 = own0, n1 = own1;
        if (cs > 1) {
          n0 += cluster_word(&counts[top], rank ^ 1);
          if (per > 1) n1 += cluster_word(&counts[top - 1], rank ^ 1);
        }
        uint32_t total;
        const uint32_t before = block_exclusive(n0 + n1, total, sm);
        if (before < want && want <= before + n0 + n1) {
          const bool second = want > before + n0;
          pick[pass][0] = second ? top - 1 : top;
          pick[pass][1] = want - before - (second ? n0 : 0u);
        }
      } else {
        __syncthreads();
        const uint32_t* const b = counts + bins - (warp + 1) * in_group;
        const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, b[lane] + (in_group > 32 ? b[32 + lane] : 0u));
        if (lane == 0) coarse[pass][warp] = sum;
        sync_all();
      }
      if (by_group && warp == 0) {
        const uint32_t own = coarse[pass][lane];
        uint32_t at = want, all = own + others(&coarse[pass][lane], cs, rank);
        const int group = crossing_lane(all, at);
        above += lane < group ? own : 0u;
        const int per = in_group / 32;  // bins of a lane, the highest first
        top = bins - 1 - group * in_group - per * lane;
        own0 = counts[top];
        own1 = per > 1 ? counts[top - 1] : 0u;
        uint32_t n0 = own0 + others(&counts[top], cs, rank), n1 = own1;
        if (per > 1) n1 += others(&counts[top - 1], cs, rank);
        all = n0 + n1;
        const int hit = crossing_lane(all, at);
        const bool second = at > n0;  // in lane `hit`
        if (lane == hit) {
          pick[pass][0] = second ? top - 1 : top;
          pick[pass][1] = at - (second ? n0 : 0u);
        }
      }
      __syncthreads();
      const int digit = static_cast<int>(pick[pass][0]);
      above += (top > digit ? own0 : 0u) + (top - 1 > digit ? own1 : 0u);
      equal = counts[digit];
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
      mine[0] = total + (c1 - end);
      mine[1] = equal;
    }
    sync_all();
    if (warp == 0) {
      uint2 x = make_uint2(0, 0);
      if (lane < rank) x = make_uint2(cluster_word(&mine[0], lane), cluster_word(&mine[1], lane));
      x.x = __reduce_add_sync(0xFFFFFFFFu, x.x);
      x.y = __reduce_add_sync(0xFFFFFFFFu, x.y);
      if (lane == 0) {
        ahead[0] = x.x;
        ahead[1] = x.y;
      }
    }
    sync_all();  // nobody leaves before its words are read
    base = ahead[0];
    ties = ahead[1];
  }

  // Ordered compaction: keys above the threshold (the window's among them) and the first `want` equal to it.  A thread
  // takes eight neighbours; the places come from a scan of the threads' counts, and the kept slots go through shared
  // memory (the counts' place), so that they and their weights are written side by side: about 25 instructions for 32
  // keys, where ballots over rows of 32 took 55.
  constexpr int kPer = 8;
  uint16_t* const stage = reinterpret_cast<uint16_t*>(hist);
  static_assert(kPer * kSelThreads * 2 <= static_cast<int>(sizeof hist), "a turn's slots fit");
  __syncthreads();  // the counts are read
  for (int i0 = c0; i0 < c1; i0 += kPer * kSelThreads) {
    const int i = i0 + kPer * t;
    uint32_t sure = 0, same = 0;  // a bit per key
#pragma unroll
    for (int q = 0; q < kPer; q += 4) {
      if (i + q >= c1) continue;
      const uint4 k = CACHED ? *reinterpret_cast<const uint4*>(keys + (i + q - c0)) : load4(i + q);
      const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + q + j >= c1) continue;
        sure |= static_cast<uint32_t>(ks[j] > prefix) << (q + j);
        same |= static_cast<uint32_t>(ks[j] == prefix) << (q + j);
      }
    }
    uint32_t total;
    const uint32_t x = block_exclusive(__popc(sure) | (__popc(same) << 16), total, sm);
    const uint32_t out0 = min(ties, want);  // ties that went before this turn
    uint32_t to = (x & 0xFFFFu) + min(ties + (x >> 16), want) - out0, tie = ties + (x >> 16);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool equal_kept = ((same >> j) & 1u) && tie < want;
      if (((sure >> j) & 1u) || equal_kept) stage[to++] = static_cast<uint16_t>(i - i0 + j);
      tie += (same >> j) & 1u;
    }
    __syncthreads();
    const int count = static_cast<int>((total & 0xFFFFu) + min(ties + (total >> 16), want) - out0);
    const uint32_t at = base + out0;
#pragma unroll 4
    for (int q = t; q < count; q += kSelThreads) {
      const int slot = i0 + stage[q];
      kept[at + q] = slot;
      nw[at + q] = w[slot];
    }
    base += total & 0xFFFFu;
    ties += total >> 16;
  }
}

// Zeroes the header and the marks behind it: a kernel in place of a memset, so that the three launches can be set up
// under one another's ends.
__global__ void __launch_bounds__(256) evict_clear_kernel(EvictParams p) {
  griddep_wait();
  uint4* to = reinterpret_cast<uint4*>(p.hdr);
  const size_t n = p.clear_bytes / 16, step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = blockIdx.x * static_cast<size_t>(256) + threadIdx.x; i < n; i += step) to[i] = make_uint4(0, 0, 0, 0);
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
// a page that keeps its largest value keeps its codes when that one's code is 448
// (as the quantizers' pages have it).
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

// Largest magnitude among 16 codes, NaN (0x7F) left out.
__device__ __forceinline__ uint32_t largest_code(const uint4& c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = __vimax3_u16x2(m, w[j] & 0x007F007Fu, (w[j] >> 8) & 0x007F007Fu);
  m = max(m & 0xFFFFu, m >> 16);
  if (m == 0x7Fu) {
    m = 0;
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = (w[i >> 2] >> (8 * (i & 3))) & 0x7Fu;
      if (a != 0x7Fu) m = max(m, a);
    }
  }
  return m;
}

// The thread's largest |value|: the exact product of code and scale as two floats, by their bits.
__device__ __forceinline__ unsigned long long largest(const Codes& x) {
  unsigned long long top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = e4m3_values(largest_code(x.c[i])).x;
    const float hi = __fmul_rz(v, x.sc[i]), lo = fmaf(v, x.sc[i], -hi);  // lo >= 0
    const unsigned long long key = (static_cast<unsigned long long>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
    top = key > top ? key : top;
  }
  return top;
}

// The new code of every magnitude, for each old page that the rows come from: rounding a code takes a dozen
// instructions, looking it up in 128 bytes of shared memory (a word per bank) three.
__device__ __forceinline__ void fill_table(uint8_t (*table)[128], const float* page_scale, int pages, float2 inv) {
  for (int i = threadIdx.x; i < pages * 128; i += kGatherThreads) {
    const float sc = page_scale[i >> 7];
    const int code = i & 127;
    float hi = sc * inv.x, lo = fmaf(sc, inv.y, fmaf(sc, inv.x, -hi));
    if (!(hi < 1e30f)) hi = 1e30f, lo = 0.0f;  // a scale so far above the values that their codes are 0
    const float y = mul_to_odd(e4m3_values(code).x, hi, lo);
    table[i >> 7][code] = code == 127 ? 127 : __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  }
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void store_codes(const EvictParams& p, void* cache, long long row0, int rows, int h,
                                            const uint8_t (*table)[128], const uint8_t* which, const Codes& x) {
  const uint32_t tables = smem_u32(table);  // each on a 128-byte boundary: an entry's address is the two or'ed
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i * kGatherThreads + threadIdx.x, r = at >> 3;
    if (r >= rows) continue;
    const uint32_t tab = tables + which[r] * 128u;
    const uint32_t w[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w};
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = lds_u8((w[j] & 0x7Fu) | tab), b = lds_u8(((w[j] >> 8) & 0x7Fu) | tab),
                     c = lds_u8(((w[j] >> 16) & 0x7Fu) | tab), d = lds_u8(((w[j] >> 24) & 0x7Fu) | tab);
      q[j] = __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410) | (w[j] & 0x80808080u);
    }
    static_cast<uint4*>(cache)[((row0 + r) * p.hkv + h) * 8 + (at & 7)] = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// CTA (new page, KV head).
__global__ void __launch_bounds__(kGatherThreads, 4) evict_gather_fp8_kernel(EvictParams p) {
  __shared__ int src[kBlock];
  __shared__ uint8_t which[kBlock];             // the row's old page, numbered in order
  __shared__ int changes[kBlock / 32];
  __shared__ float page_scale[2][kBlock];       // K and V scale of each old page
  __shared__ unsigned long long keys[2][kGatherThreads / 32];
  __shared__ float2 inv[2];                     // 448 / max as two floats
  __shared__ __align__(128) uint8_t table[2][kBlock][128];
  griddep_wait();
  const NewPage x = new_page(p, blockIdx.x);
  if (x.rows <= 0) return;
  const int h = blockIdx.y, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t < kBlock)
    src[t] = t < x.rows
                 ? source_row(p, x.s, x.n, (static_cast<long long>(x.s) * p.hkv + h) * p.budget + x.b * kBlock + t)
                 : -1;
  if (!page_fine(p, x)) return;
  __syncthreads();
  Codes k, v;
  load_codes(p, p.k, p.k_scale, x.rows, h, src, k);
  load_codes(p, p.v, p.v_scale, x.rows, h, src, v);
  // number the old pages: kept slots ascend, so a page's rows are neighbours
  const int old = t < kBlock && src[t] >= 0 ? src[t] / kBlock : -1;
  const bool change = t > 0 && t < x.rows && old != (src[t - 1] >= 0 ? src[t - 1] / kBlock : -1);
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, change);
  if (warp < kBlock / 32 && lane == 0) changes[warp] = __popc(mask);
  const unsigned long long tk = warp_max_u64(largest(k)), tv = warp_max_u64(largest(v));
  if (lane == 0) {
    keys[0][warp] = tk;
    keys[1][warp] = tv;
  }
  __syncthreads();
  int pages = 1;
#pragma unroll
  for (int i = 0; i < kBlock / 32; ++i) pages += changes[i];
  if (t < x.rows) {
    int number = __popc(mask & (0xFFFFFFFFu >> (31 - lane)));
    for (int i = 0; i < warp; ++i) number += changes[i];
    which[t] = static_cast<uint8_t>(number);
    if (change || t == 0) {
      page_scale[0][number] = old >= 0 ? p.k_scale[static_cast<long long>(old) * p.hkv + h] : 0.0f;
      page_scale[1][number] = old >= 0 ? p.v_scale[static_cast<long long>(old) * p.hkv + h] : 0.0f;
    }
  } else if (t >= kGatherThreads - 64 && lane == 0) {  // the last two warps: a thread each for K and V
    const int kv = warp & 1;
    unsigned long long top = 0;
#pragma unroll
    for (int i = 0; i < kGatherThreads / 32; ++i) top = keys[kv][i] > top ? keys[kv][i] : top;
    const double value = static_cast<double>(__uint_as_float(static_cast<uint32_t>(top >> 32))) +
                         static_cast<double>(__uint_as_float(static_cast<uint32_t>(top)));
    const bool some = value >= 0x1p-118;  // below, 448 / value is no fp32 number: codes 0
    (kv ? p.v_scale : p.k_scale)[static_cast<long long>(x.page) * p.hkv + h] =
        some ? static_cast<float>(value / 448.0) : 1.0f;
    const double q = some ? 448.0 / value : 0.0;
    const float hi = static_cast<float>(q);
    inv[kv] = make_float2(hi, static_cast<float>(q - static_cast<double>(hi)));
  }
  __syncthreads();
  fill_table(table[0], page_scale[0], pages, inv[0]);
  fill_table(table[1], page_scale[1], pages, inv[1]);
  __syncthreads();
  const long long row0 = static_cast<long long>(x.page) * kBlock;
  store_codes(p, p.k, row0, x.rows, h, table[0], which, k);
  store_codes(p, p.v, row0, x.rows, h, table[1], which, v);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, bool fp8, int sms, cudaStream_t stream) {
  const size_t clear = (p.clear_bytes / 16 + 1023) / 1024;  // CTAs, four pieces a thread
  cudaError_t e = launch_pdl(evict_clear_kernel, dim3(static_cast<unsigned>(clear < 4096 ? clear : 4096)), dim3(256), 0,
                             stream, p);
  if (e != cudaSuccess) return e;
  // CTAs per (sequence, head): at most eight (a portable cluster), none with a share under 8,192 slots (the cluster's
  // barriers and reads cost about 4 us), and only as many as run at once: a cluster's CTAs, one to an SM, share one
  // of the GPU's eight or so SM groups, so larger clusters leave more SMs over (16 clusters of 8 took two turns, 49 us
  // against 25 us for 4 clusters, at 65,536 slots).
  const long long rows = static_cast<long long>(p.num_seqs) * p.hkv;
  int cs = rows <= sms / 19 ? 8 : rows <= sms / 6 ? 4 : rows <= sms / 2 ? 2 : 1;
  while (cs > 1 && p.max_k / cs < 8 * kSelThreads) cs /= 2;
  const int share = ((p.max_k + cs - 1) / cs + 15) & ~15;  // the largest
  const bool cached = share <= kSelKeys;
  auto* fn = cached ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cs);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = cached ? static_cast<size_t>(share) * 4 : 0;
  cfg.stream = stream;
  if (cfg.dynamicSmemBytes > 16 * 1024) {  // with the static part more than the default limit
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cs), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, fn, p, cs);
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
