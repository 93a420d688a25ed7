// cache.cu -- filling a paged cache: block tables and slot maps from the requests' lengths, and the new tokens' K, V and
// K_idx rows into their slots.
//
// Tables.  A sequence of n cached tokens that gets m new ones needs ceil((n + m) / 128) - ceil(n / 128) more pages; they
// are taken from a list of free pages, sequence by sequence, so the result does not depend on timing.  One CTA scans the
// lengths; then every new token finds its sequence in the prefix sums and its page in the table or the list, and the
// token at a block's first position writes the block's entry.  The CTA that scanned does that too where the tokens are few.
//
// Rows.  bf16: a copy, a warp per token and tensor.  E4M3: a page has one scale per head, so the new rows of a page are
// taken together: the tokens that follow one another into one page (a run), per head.  Their largest value may ask for a
// larger scale than the page has; the rows that the page holds already (those before the run's first) are then rounded
// again.
#include <cuda_fp8.h>

#include <cstddef>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

// ---------------------------------------------------------------- tables
constexpr int kTableThreads = 1024;
constexpr int kPlaceMost = 4096;  // tokens that the scanning CTA places itself: a second kernel takes 3 us more, 1,000 tokens 0.4

struct Sums {
  long long tokens, keys, pages;
};
// Exclusive scan of three numbers over the CTA's kTableThreads threads.
__device__ __forceinline__ Sums table_scan(Sums v, Sums* sh, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto warp_scan = [&](Sums x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y{__shfl_up_sync(0xFFFFFFFFu, x.tokens, o), __shfl_up_sync(0xFFFFFFFFu, x.keys, o),
                   __shfl_up_sync(0xFFFFFFFFu, x.pages, o)};
      if (lane >= o) {
        x.tokens += y.tokens;
        x.keys += y.keys;
        x.pages += y.pages;
      }
    }
    return x;
  };
  const Sums x = warp_scan(v);
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) sh[lane] = warp_scan(sh[lane]);
  __syncthreads();
  const Sums before = warp > 0 ? sh[warp - 1] : Sums{0, 0, 0};
  *total = sh[31];
  __syncthreads();
  return {before.tokens + x.tokens - v.tokens, before.keys + x.keys - v.keys, before.pages + x.pages - v.pages};
}

// New token i, the `t`-th of sequence s, which had `len`: its slot and position, and its block's table entry when it is the
// block's first token.
__device__ __forceinline__ void place_token(const ExtendParams& p, long long i, int s, int len, int t, int page_base) {
  const int pos = len + t, block = pos >> 7, held = (len + 127) >> 7;
  int page = -1;
  if (block < held) {
    page = p.block_table[static_cast<long long>(s) * p.bt_stride + block];
  } else {
    const long long at = static_cast<long long>(page_base) + block - held;
    if (at < p.num_free) page = p.free_pages[at];
  }
  if (page < 0 || page >= p.n_pages) {
    page = -1;
    atomicOr(&p.hdr->status, kFlagBadIndex);
  }
  if ((pos & 127) == 0) p.block_table[static_cast<long long>(s) * p.bt_stride + block] = page;
  p.slots[i] = page < 0 ? -1 : static_cast<long long>(page) * 128 + (pos & 127);
  p.positions[i] = pos;
}

__global__ void __launch_bounds__(kTableThreads) extend_plan_kernel(ExtendParams p, bool place) {
  __shared__ Sums sh[32];
  __shared__ int s_bad;
  __shared__ int first[kTableThreads + 1], length[kTableThreads], pages[kTableThreads];  // of up to kTableThreads sequences
  if (threadIdx.x == 0) s_bad = 0;
  griddep_wait();
  const int taken = p.taken ? *p.taken : 0;
  // lengths that cannot be, or that pass the buffers: nothing is taken, every slot is -1
  bool bad = taken < 0 || taken > p.num_free;
  Sums carry{0, 0, taken};
  for (int base = 0; base < p.num_seqs; base += kTableThreads) {
    const int s = base + threadIdx.x;
    long long n = 0, m = 0;
    if (s < p.num_seqs) {
      n = p.lengths[s];
      m = p.new_tokens[s];
      if (n < 0 || m < 0 || n + m > p.max_len) {
        bad = true;
        n = m = 0;
      }
    }
    Sums t;
    const Sums at = table_scan({m, n + m, ((n + m + 127) >> 7) - ((n + 127) >> 7)}, sh, &t);
    if (s < p.num_seqs) {
      const int q = static_cast<int>(carry.tokens + at.tokens), pg = static_cast<int>(carry.pages + at.pages);
      p.cu_q[s + 1] = q + static_cast<int>(m);
      p.cu_k[s + 1] = static_cast<int>(carry.keys + at.keys + n + m);
      p.page_base[s] = pg;
      if (base == 0) {
        first[threadIdx.x] = q;
        length[threadIdx.x] = static_cast<int>(n);
        pages[threadIdx.x] = pg;
      }
    }
    carry.tokens += t.tokens;
    carry.keys += t.keys;
    carry.pages += t.pages;
  }
  if (bad) s_bad = 1;
  __syncthreads();
  bad = s_bad || carry.tokens > p.capacity || carry.keys > 0x7FFFFFFFLL;
  if (bad) carry.tokens = 0;
  for (int s = threadIdx.x; s < p.num_seqs; s += kTableThreads) {
    if (bad) {
      p.cu_q[s + 1] = 0;
      p.cu_k[s + 1] = 0;
    } else if (p.new_lengths) {
      p.new_lengths[s] = p.lengths[s] + p.new_tokens[s];
    }
  }
  if (threadIdx.x < sizeof(WsHeader) / 4)
    reinterpret_cast<uint32_t*>(p.hdr)[threadIdx.x] = threadIdx.x == 0 && bad ? kFlagBadSeqlens : 0u;
  static_assert(offsetof(WsHeader, status) == 0, "the first word");
  if (threadIdx.x == 0) {
    p.cu_q[0] = 0;
    p.cu_k[0] = 0;
    *p.taken_out = bad ? taken : static_cast<int>(carry.pages < p.num_free ? carry.pages : p.num_free);
  }
  if (!place) return;
  __syncthreads();  // the header, before flags are raised in it
  const int tokens = static_cast<int>(carry.tokens);
  for (int i = threadIdx.x; i < p.capacity; i += kTableThreads) {
    if (i >= tokens) {
      p.slots[i] = -1;
      p.positions[i] = 0;
      continue;
    }
    const int s = find_seq(first, p.num_seqs, i);  // num_seqs <= kTableThreads
    place_token(p, i, s, length[s], i - first[s], pages[s]);
  }
}

// Tokens 32 i .. of a warp lie in few sequences: the warp finds the first one's, 32 places at a time, and each lane goes on
// from there.
constexpr int kPlaceThreads = 256;
__global__ void __launch_bounds__(kPlaceThreads) extend_place_kernel(ExtendParams p) {
  griddep_wait();
  const int tokens = p.cu_q[p.num_seqs], lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (kPlaceThreads / 32);
  for (long long i0 = (blockIdx.x * static_cast<long long>(kPlaceThreads / 32) + (threadIdx.x >> 5)) * 128; i0 < p.capacity;
       i0 += warps * 128) {
    // the last sequence that begins at or before token i0, with an empty one's successors behind it
    int lo = 0, n = p.num_seqs;
    while (i0 < tokens && n > 1) {
      const int step = (n + 31) / 32;
      const int at = lo + lane * step;
      const bool begun = lane * step < n && p.cu_q[at] <= i0;
      const int k = __popc(__ballot_sync(0xFFFFFFFFu, begun)) - 1;  // lane 0's has begun
      lo += k * step;
      n = min(step, n - k * step);
    }
    int s = lo, q0 = 0, q1 = 0, len = 0, base = 0;
    bool known = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long i = i0 + u * 32 + lane;
      if (i >= p.capacity) continue;
      if (i >= tokens) {
        p.slots[i] = -1;
        p.positions[i] = 0;
        continue;
      }
      if (!known || i >= q1) {
        while (p.cu_q[s + 1] <= i) ++s;
        q0 = p.cu_q[s];
        q1 = p.cu_q[s + 1];
        len = (p.cu_k[s + 1] - p.cu_k[s]) - (q1 - q0);
        base = p.page_base[s];
        known = true;
      }
      place_token(p, i, s, len, static_cast<int>(i) - q0, base);
    }
  }
}

// ---------------------------------------------------------------- rows, bf16
// HBM: 31,800 tokens of 4 heads and K_idx (147 MB) take 25.7 us, 84 % of a copy's rate.
constexpr int kAppendWarps = 8;
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(AppendParams p) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long n = p.tokens * p.planes;
  for (long long i = blockIdx.x * static_cast<long long>(kAppendWarps) + (threadIdx.x >> 5); i < n;
       i += static_cast<long long>(gridDim.x) * kAppendWarps) {
    const long long token = i / p.planes;
    const AppendPlane& a = p.plane[i - token * p.planes];
    const long long slot = p.slots[token];
    if (slot < 0 || slot >= p.n_pages * 128) {
      if (slot != -1 && p.hdr && lane == 0) atomicOr(&p.hdr->status, kFlagBadIndex);
      continue;
    }
    const uint4* from = reinterpret_cast<const uint4*>(a.x + token * a.stride);
    uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.cache) + slot * a.width);
    for (int c = lane; c < a.width / 8; c += 32) to[c] = from[c];
  }
}

// ---------------------------------------------------------------- rows, E4M3
constexpr int kRunThreads = 256;
constexpr float kZeroBelow = 3.0092655e-36f;  // 2^-118: rows below are zeros.  Its scale, 2^-126.8, is off by 2^-23 at most

__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(__half2(h));
}

// What a run does to its page's scale, and its rows' quotients.
struct RunScale {
  float was, now;
  float up, down, inv;  // a code is that of x * up / down; 1 / down
  bool plain;           // by division
};
__device__ __forceinline__ RunScale run_scale(float was, float amax, bool live) {
  RunScale r;
  const float fresh = amax >= kZeroBelow ? __fdiv_rn(amax, 448.0f) : 0.0f;
  r.was = was;
  r.now = live ? fmaxf(was, fresh) : fresh;
  if (r.now == 0.0f) r.now = 1.0f;
  // A value's code is that of the exact quotient: where the new rows set the scale (amax / 448, rounded) that is x * 448 /
  // amax, and x * 448 has 11 significant bits.  bf16 values meet the middle between two codes often (one in 40 of a
  // normal distribution's), and a rounded scale would put them on either side.
  const bool ours = fresh > 0.0f && r.now == fresh;
  // powers of two that keep products and remainders normal numbers
  const float shift = amax > 1.26765060e30f ? 5.42101086e-20f : amax < 8.8817842e-16f ? 1.84467441e19f : 1.0f;
  r.up = ours ? 448.0f * shift : 1.0f;
  r.down = ours ? amax * shift : r.now;
  r.plain = !(r.down >= 7.8886091e-31f && r.down <= 1.26765060e30f);  // a scale of the caller's outside 2^-100 .. 2^100
  r.inv = __fdiv_rn(1.0f, r.down);
  return r;
}
// fp32(x / down), correctly rounded, of two numbers given as -x: with 1 / down correctly rounded, one step from the remainder,
// which an fma gives exactly (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  From -x the remainder has the sign with which a zero keeps its own through the last sum.  With a division for
// each value the kernel ran 45 instructions a value.  Not for inf and NaN.
__device__ __forceinline__ float2 quotients(float2 minus_x, const RunScale& r) {
  const float2 minus_inv = make_float2(-r.inv, -r.inv), q = fmul2(minus_x, minus_inv);
  return ffma2(ffma2(q, make_float2(r.down, r.down), minus_x), minus_inv, q);
}
__device__ __forceinline__ float2 divided(float2 minus_x, const RunScale& r) {
  return make_float2(__fdiv_rn(-minus_x.x, r.down), __fdiv_rn(-minus_x.y, r.down));
}
template <bool PLAIN>
__device__ __forceinline__ uint2 codes_of(const uint4& v, const RunScale& r) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = fmul2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), make_float2(-r.up, -r.up));
    const float2 q = PLAIN ? divided(x, r) : quotients(x, r);
    c[j] = to_e4m3x2(q.x, q.y);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// Out of line: where a scale is outside 2^-100 .. 2^100, or a value is inf or NaN.
__device__ __noinline__ uint2 codes_of_any(uint4 v, RunScale r) { return codes_of<true>(v, r); }
// Eight codes of a row that was there before, at the new scale.
template <bool PLAIN>
__device__ __forceinline__ uint2 codes_again(const uint2& old, const RunScale& r) {
  const uint32_t w[4] = {old.x & 0xFFFFu, old.x >> 16, old.y & 0xFFFFu, old.y >> 16};
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = fmul2(fmul2(from_e4m3x2(w[j]), make_float2(-r.up, -r.up)), make_float2(r.was, r.was));
    const float2 q = PLAIN ? divided(x, r) : quotients(x, r);
    c[j] = to_e4m3x2(q.x, q.y);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
__device__ __noinline__ uint2 codes_again_any(uint2 old, RunScale r) { return codes_again<true>(old, r); }
// |x| as bits, two values to a word: the largest of eight and of m.
__device__ __forceinline__ uint32_t bf16x8_max(const uint4& v, uint32_t m) {
  return __vmaxu2(__vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)), m);
}
// The same of finite values, where there are others.
__device__ __noinline__ uint32_t bf16x8_max_finite(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = w[j >> 1] >> (j & 1) * 16 & 0x7FFFu;
    if (b < 0x7F80u) m = max(m, b);
  }
  return m;
}

// A CTA: the runs that begin among the tokens of a chunk, one head of the planes.  16 threads take a row, 8
// values each.  A short run is one warp's, two rows at a time; a longer one all warps', 16 rows at a time; its rows stay in
// registers between their maximum and their codes.  Slots are read once, those of the longest run behind the chunk
// among them.
// 31,800 tokens of 6 prompts, 9 heads (110 MB): 31.8 us, 3.5 TB/s; some 17 instructions a value issue in half of the cycles,
// the rest waits for rows and barriers (two CTAs an SM: 36.8 us; four, whose registers do not hold a run's rows: 35.6).  256
// runs of one token, 16 heads: 5.0 us, the latency of slots, scale and row one after another.
constexpr int kShortRun = 16;
constexpr int kMostChunk = 128;
__global__ void __launch_bounds__(kRunThreads, 3) append_fp8_kernel(AppendParams p, int chunk, uint32_t all_heads) {
  __shared__ int s_page[2 + kMostChunk + 128];  // page of tokens lo - 1 .. lo + chunk + 127, -1: none
  __shared__ uint8_t s_row[2 + kMostChunk + 128];
  __shared__ int2 s_long[kMostChunk / kShortRun + 1];  // runs for all warps: first token, length
  __shared__ int s_count;
  __shared__ uint32_t s_max[kRunThreads / 32];
  __shared__ int s_low[kRunThreads / 32];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int head = static_cast<int>(blockIdx.x % all_heads), pl = 0;  // the heads of a chunk run together: their rows share pages of DRAM
  const bool marks = head == 0;
  while (head >= p.plane[pl].width / 128) head -= p.plane[pl++].width / 128;
  const AppendPlane& a = p.plane[pl];
  const int heads = a.width / 128;
  const long long rows = p.n_pages * 128, row_bytes = static_cast<long long>(heads) * 128;
  const long long lo = static_cast<long long>(blockIdx.x / all_heads) * chunk;
  const int n = static_cast<int>(min(static_cast<long long>(chunk), p.tokens - lo));
  for (int t = tid; t < 1 + chunk + 128; t += kRunThreads) {
    const long long i = lo - 1 + t;
    long long slot = -1;
    if (i >= 0 && i < p.tokens) slot = p.slots[i];
    const bool there = slot >= 0 && slot < rows;
    if (!there && slot != -1 && marks) atomicOr(&p.hdr->status, kFlagBadIndex);
    s_page[t] = there ? static_cast<int>(slot >> 7) : -1;
    s_row[t] = static_cast<uint8_t>(slot & 127);
  }
  if (tid == 0) s_count = 0;
  __syncthreads();
  const int sub = lane & 15, half = lane >> 4;
  const __nv_bfloat16* const x0 = a.x + lo * a.stride + head * 128 + sub * 8;
  // the warp's share of the chunk's tokens, one to a lane: which are a run's first
  constexpr int kWarps = kRunThreads / 32;
  static_assert(kMostChunk <= 32 * kWarps, "a lane per token");
  const int at = warp + lane * kWarps;
  uint32_t starts = __ballot_sync(0xFFFFFFFFu, at < n && s_page[min(1 + at, 1 + kMostChunk)] >= 0 &&
                                                   s_page[min(at, kMostChunk)] != s_page[min(1 + at, 1 + kMostChunk)]);
  for (; starts; starts &= starts - 1) {
    const int t = warp + (__ffs(starts) - 1) * kWarps, page = s_page[1 + t];
    int len = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t same = __ballot_sync(0xFFFFFFFFu, s_page[1 + t + u * 32 + lane] == page);
      if (len == u * 32) len += same == 0xFFFFFFFFu ? 32 : __ffs(~same) - 1;
    }
    if (marks && lane == 0) {
      // a page's rows come in one run of at most 128 tokens
      const bool more = len == 128 && s_page[1 + t + 128] == page;  // t < chunk: within what was read
      if (atomicExch(&p.marks[page], 1u) != 0u || more) atomicOr(&p.hdr->status, kFlagBadIndex);
    }
    if (len > kShortRun) {
      if (lane == 0) s_long[atomicAdd(&s_count, 1)] = make_int2(t, len);  // at most one in kShortRun tokens begins one
      continue;
    }
    float* const scale_at = a.scale + static_cast<long long>(page) * heads + head;
    const float was = *scale_at;
    uint4 v[kShortRun / 2];
    uint32_t m = 0;
    int low = 127;
#pragma unroll
    for (int k = 0; k < kShortRun / 2; ++k) {
      const int r = k * 2 + half;
      v[k] = make_uint4(0, 0, 0, 0);
      if (r < len) {
        v[k] = *reinterpret_cast<const uint4*>(x0 + (t + r) * a.stride);
        low = min(low, static_cast<int>(s_row[1 + t + r]));
      }
    }
#pragma unroll
    for (int k = 0; k < kShortRun / 2; ++k) m = bf16x8_max(v[k], m);
    m = max(m & 0xFFFFu, m >> 16);
    const bool odd = __any_sync(0xFFFFFFFFu, m >= 0x7F80u);  // an inf or NaN
    if (odd) {
      m = 0;
#pragma unroll
      for (int k = 0; k < kShortRun / 2; ++k) m = bf16x8_max_finite(v[k], m);
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    const RunScale r = run_scale(was, __uint_as_float(m << 16), low > 0);
    uint8_t* const cache = static_cast<uint8_t*>(a.cache) + (static_cast<long long>(page) * 128 * heads + head) * 128 + sub * 8;
    __syncwarp();  // every lane has read the scale
    if (lane == 0) *scale_at = r.now;
    if (low > 0 && r.now != was) {
      for (int row = half; row < low; row += 16) {
        uint2 old[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (row + 2 * k < low) old[k] = *reinterpret_cast<const uint2*>(cache + (row + 2 * k) * row_bytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (row + 2 * k < low) *reinterpret_cast<uint2*>(cache + (row + 2 * k) * row_bytes) =
                r.plain ? codes_again_any(old[k], r) : codes_again<false>(old[k], r);
      }
    }
    const bool any = r.plain || odd;
#pragma unroll
    for (int k = 0; k < kShortRun / 2; ++k) {
      const int q = k * 2 + half;
      if (q < len)
        *reinterpret_cast<uint2*>(cache + s_row[1 + t + q] * row_bytes) = any ? codes_of_any(v[k], r) : codes_of<false>(v[k], r);
    }
  }
  __syncthreads();
  const int r0 = tid >> 4;
  for (int j = 0; j < s_count; ++j) {
    const int t = s_long[j].x, len = s_long[j].y;
    const int page = s_page[1 + t];
    float* const scale_at = a.scale + static_cast<long long>(page) * heads + head;
    const float was = *scale_at;
    const __nv_bfloat16* const from = x0 + (t + r0) * a.stride;
    const long long step = 16 * a.stride;
    uint4 v[8];
    uint32_t m = 0;
    int low = 127;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int q = k * 16 + r0;
      v[k] = make_uint4(0, 0, 0, 0);
      if (q < len) {
        v[k] = *reinterpret_cast<const uint4*>(from + k * step);
        low = min(low, static_cast<int>(s_row[1 + t + q]));
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = bf16x8_max(v[k], m);
    m = max(m & 0xFFFFu, m >> 16);
    const bool odd = __any_sync(0xFFFFFFFFu, m >= 0x7F80u);  // an inf or NaN among the warp's rows
    if (odd) {
      m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = bf16x8_max_finite(v[k], m);
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    if (lane == 0) {
      s_max[warp] = m;
      s_low[warp] = low;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRunThreads / 32; ++w) {
      m = max(m, s_max[w]);
      low = min(low, s_low[w]);
    }
    const RunScale r = run_scale(was, __uint_as_float(m << 16), low > 0);
    uint8_t* const cache = static_cast<uint8_t*>(a.cache) + (static_cast<long long>(page) * 128 * heads + head) * 128 + sub * 8;
    __syncthreads();  // every thread has read the scale, and the maxima
    if (tid == 0) *scale_at = r.now;
    if (low > 0 && r.now != was) {
      for (int row = r0; row < low; row += 128) {
        uint2 old[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (row + 16 * k < low) old[k] = *reinterpret_cast<const uint2*>(cache + (row + 16 * k) * row_bytes);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (row + 16 * k < low) *reinterpret_cast<uint2*>(cache + (row + 16 * k) * row_bytes) =
                r.plain ? codes_again_any(old[k], r) : codes_again<false>(old[k], r);
      }
    }
    const bool any = r.plain || odd;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int q = k * 16 + r0;
      if (q < len)
        *reinterpret_cast<uint2*>(cache + s_row[1 + t + q] * row_bytes) = any ? codes_of_any(v[k], r) : codes_of<false>(v[k], r);
    }
  }
}

constexpr int kClearThreads = 256;
__global__ void __launch_bounds__(kClearThreads) clear_kernel(uint4* at, long long n) {
  griddep_wait();
  for (long long i = blockIdx.x * static_cast<long long>(kClearThreads) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kClearThreads)
    at[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

cudaError_t launch_extend(const ExtendParams& p, int sms, cudaStream_t stream) {
  const bool place = p.capacity <= kPlaceMost && p.num_seqs <= kTableThreads;
  cudaError_t e = launch_pdl(extend_plan_kernel, dim3(1), dim3(kTableThreads), 0, stream, p, place);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (place) return cudaSuccess;
  long long ctas = (p.capacity + 4 * kPlaceThreads - 1) / (4 * kPlaceThreads);
  if (ctas > sms * 8) ctas = sms * 8;
  if (ctas < 1) ctas = 1;
  e = launch_pdl(extend_place_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPlaceThreads), 0, stream, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream) {
  if (p.hdr) {
    const cudaError_t e = cudaMemsetAsync(p.hdr, 0, sizeof(WsHeader), stream);
    if (e != cudaSuccess) return e;
    note_launches(1);
  }
  if (p.tokens == 0) return cudaSuccess;
  long long ctas = (p.tokens * p.planes + kAppendWarps - 1) / kAppendWarps;
  if (ctas > sms * 8) ctas = sms * 8;
  const cudaError_t e = launch_pdl(append_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kAppendWarps * 32), 0, stream, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

cudaError_t launch_append_fp8(const AppendParams& p, size_t clear_bytes, int sms, cudaStream_t stream) {
  const long long words = static_cast<long long>(clear_bytes / 16);  // the workspace's parts are multiples of 256 bytes
  long long clear_ctas = (words + 4 * kClearThreads - 1) / (4 * kClearThreads);
  if (clear_ctas > sms) clear_ctas = sms;
  cudaError_t e = launch_pdl(clear_kernel, dim3(static_cast<unsigned>(clear_ctas)), dim3(kClearThreads), 0, stream,
                             reinterpret_cast<uint4*>(p.hdr), words);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (p.tokens == 0) return cudaSuccess;
  // Few tokens are mostly runs of their own (a decode step), one to a warp; many are prompts with a run per page, about one
  // to the largest chunk (31,800 tokens: 31.8 us, with half of it 35.4, a quarter 44.8).  4,096 runs of one token, 8 heads:
  // 19.4 us with chunks of 32, 23.4 with 8.
  int chunk = kRunThreads / 32;
  while (chunk < kMostChunk && p.tokens > 128LL * chunk) chunk *= 2;
  int heads = 0;
  for (int i = 0; i < p.planes; ++i) heads += p.plane[i].width / 128;
  e = launch_pdl(append_fp8_kernel, dim3(static_cast<unsigned>((p.tokens + chunk - 1) / chunk * heads)), dim3(kRunThreads), 0,
                 stream, p, chunk, static_cast<uint32_t>(heads));
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace msa
