// cache.cu -- filling a paged cache: block tables and slot maps from the requests' lengths, and the new tokens' K, V and
// K_idx rows into their slots.
//
// Tables.  A sequence of n cached tokens that gets m new ones needs ceil((n + m) / 128) - ceil(n / 128) more pages; they
// are taken from a list of free pages, sequence by sequence, so the result does not depend on timing.  A plan kernel (one
// CTA) scans the lengths; then every new token finds its sequence in the prefix sums and its page in the table or the
// list, and the token at a block's first position writes the block's entry.
//
// Rows.  bf16: a copy, a warp per token and tensor.  E4M3: a page has one scale per head, so the new rows of a page are
// taken together: the tokens that follow one another into one page (a run) by one CTA per head, read once into
// registers.  Their largest value may ask for a larger scale than the page has; the rows that the page holds already (those
// before the run's first) are then rounded again.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

// ---------------------------------------------------------------- tables
constexpr int kTableThreads = 1024;

// Exclusive scan over the CTA's kTableThreads threads.
__device__ long long table_scan(long long v, long long* sh, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    sh[lane] = w;
  }
  __syncthreads();
  const long long before = x - v + (warp > 0 ? sh[warp - 1] : 0);
  *total = sh[31];
  __syncthreads();
  return before;
}

// Token i of the call: its slot and position, and its block's table entry when it is the block's first token.
__device__ __forceinline__ void place_token(const ExtendParams& p, long long i, int tokens) {
  if (i >= tokens) {
    p.slots[i] = -1;
    p.positions[i] = 0;
    return;
  }
  const int s = find_seq(p.cu_q, p.num_seqs, static_cast<int>(i));
  const int q0 = p.cu_q[s], len = (p.cu_k[s + 1] - p.cu_k[s]) - (p.cu_q[s + 1] - q0);
  const int pos = len + static_cast<int>(i) - q0, block = pos >> 7, held = (len + 127) >> 7;
  int page = -1;
  if (block < held) {
    page = p.block_table[static_cast<long long>(s) * p.bt_stride + block];
  } else {
    const long long at = static_cast<long long>(p.page_base[s]) + block - held;
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

__global__ void __launch_bounds__(kTableThreads) extend_plan_kernel(ExtendParams p) {
  __shared__ long long sh[32];
  __shared__ int s_bad;
  griddep_wait();
  for (int w = threadIdx.x; w < static_cast<int>(sizeof(WsHeader) / 4); w += kTableThreads)
    reinterpret_cast<uint32_t*>(p.hdr)[w] = 0u;
  const int taken = p.taken ? *p.taken : 0;
  // lengths that cannot be, or that pass the buffers: nothing is taken, every slot is -1
  if (threadIdx.x == 0) s_bad = taken < 0 || taken > p.num_free;
  __syncthreads();
  long long tokens = 0, keys = 0;
  for (int base = 0; base < p.num_seqs; base += kTableThreads) {
    const int s = base + threadIdx.x;
    long long n = 0, m = 0;
    if (s < p.num_seqs) {
      n = p.lengths[s];
      m = p.new_tokens[s];
      if (n < 0 || m < 0 || n + m > p.max_len) s_bad = 1;
    }
    long long t;
    table_scan(m, sh, &t);
    tokens += t;
    table_scan(n + m, sh, &t);
    keys += t;
  }
  __syncthreads();
  const bool bad = s_bad || tokens > p.capacity || keys > 0x7FFFFFFFLL;
  long long carry_q = 0, carry_k = 0, carry_p = taken;
  for (int base = 0; base < p.num_seqs; base += kTableThreads) {
    const int s = base + threadIdx.x;
    int n = 0, m = 0;
    if (s < p.num_seqs && !bad) {
      n = p.lengths[s];
      m = p.new_tokens[s];
    }
    const int need = ((n + m + 127) >> 7) - ((n + 127) >> 7);
    long long tq, tk, tp;
    const long long bq = table_scan(m, sh, &tq), bk = table_scan(n + m, sh, &tk), bp = table_scan(need, sh, &tp);
    if (s < p.num_seqs) {
      p.cu_q[s + 1] = static_cast<int>(carry_q + bq + m);
      p.cu_k[s + 1] = static_cast<int>(carry_k + bk + n + m);
      p.page_base[s] = static_cast<int>(carry_p + bp);
      if (p.new_lengths && !bad) p.new_lengths[s] = n + m;
    }
    carry_q += tq;
    carry_k += tk;
    carry_p += tp;
  }
  if (threadIdx.x == 0) {
    p.cu_q[0] = 0;
    p.cu_k[0] = 0;
    *p.taken_out = bad ? taken : static_cast<int>(carry_p < p.num_free ? carry_p : p.num_free);
    if (bad) atomicOr(&p.hdr->status, kFlagBadSeqlens);
  }
}

constexpr int kPlaceThreads = 256;
__global__ void __launch_bounds__(kPlaceThreads) extend_place_kernel(ExtendParams p) {
  griddep_wait();
  const int tokens = p.cu_q[p.num_seqs];
  for (long long i = blockIdx.x * static_cast<long long>(kPlaceThreads) + threadIdx.x; i < p.capacity;
       i += static_cast<long long>(gridDim.x) * kPlaceThreads)
    place_token(p, i, tokens);
}

// ---------------------------------------------------------------- rows, bf16
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
constexpr int kRunThreads = 128;
constexpr float kZeroBelow = 3.0092655e-36f;  // 2^-118: an amax / 448 is a normal number from here on

__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(__half2(h));
}

// CTA (x, y): the runs that begin among tokens [x * chunk, (x + 1) * chunk), head y of the planes.
__global__ void __launch_bounds__(kRunThreads) append_fp8_kernel(AppendParams p, int chunk) {
  __shared__ int s_first, s_len, s_low;
  __shared__ uint32_t s_max[kRunThreads / 32];
  __shared__ int s_row[128];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int head = blockIdx.y, pl = 0;
  while (head >= p.plane[pl].width / 128) head -= p.plane[pl++].width / 128;
  const AppendPlane& a = p.plane[pl];
  const int heads = a.width / 128;
  const long long rows = p.n_pages * 128;
  const long long lo = static_cast<long long>(blockIdx.x) * chunk, hi = min(lo + chunk, p.tokens);
  const bool marks = blockIdx.y == 0;
  auto page_of = [&](long long slot) { return slot < 0 || slot >= rows ? -1LL : slot >> 7; };
  for (long long at = lo; at < hi;) {
    // the first token of the chunk, from `at` on, whose page is not that of the token before it
    if (tid == 0) {
      s_first = kRunThreads;
      s_len = kRunThreads;
      s_low = 128;
    }
    __syncthreads();
    const long long i = at + tid;
    if (i < hi) {
      const long long slot = p.slots[i], page = page_of(slot);
      if (page < 0) {
        if (slot != -1 && marks) atomicOr(&p.hdr->status, kFlagBadIndex);
      } else if (i == 0 || page_of(p.slots[i - 1]) != page) {
        atomicMin(&s_first, tid);
      }
    }
    __syncthreads();
    const int first = s_first;
    if (first == kRunThreads) {
      at += kRunThreads;
      __syncthreads();
      continue;
    }
    const long long start = at + first;
    const long long page = p.slots[start] >> 7;
    {
      const long long j = start + tid;
      const long long slot = j < p.tokens ? p.slots[j] : -1;
      if (page_of(slot) != page) atomicMin(&s_len, tid);
      s_row[tid] = static_cast<int>(slot & 127);
    }
    if (tid == 0 && marks) {
      // a page's rows come in one run of at most 128 tokens
      const bool more = start + 128 < p.tokens && page_of(p.slots[start + 128]) == page && page_of(p.slots[start + 127]) == page;
      if (atomicExch(&p.marks[page], 1u) != 0u || more) atomicOr(&p.hdr->status, kFlagBadIndex);
    }
    __syncthreads();
    const int len = s_len;
    if (tid < len) atomicMin(&s_low, s_row[tid]);
    // 16 threads to a row, 8 values each
    const int sub = tid & 15, r0 = tid >> 4;
    const __nv_bfloat16* x = a.x + start * a.stride + head * 128 + sub * 8;
    uint4 v[16];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      v[k] = make_uint4(0, 0, 0, 0);
      if (k * 8 + r0 < len) v[k] = *reinterpret_cast<const uint4*>(x + (k * 8 + r0) * a.stride);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t l = w[j] & 0x7FFFu, h = (w[j] >> 16) & 0x7FFFu;
        if (l < 0x7F80u) m = max(m, l);  // inf and NaN do not count
        if (h < 0x7F80u) m = max(m, h);
      }
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    const int low = s_low;
    const float amax = __uint_as_float(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])) << 16);
    const float fresh = amax >= kZeroBelow ? __fdiv_rn(amax, 448.0f) : 0.0f;
    float* scale_at = a.scale + page * heads + head;
    const float was = *scale_at;
    float now = low > 0 ? fmaxf(was, fresh) : fresh;
    if (now == 0.0f) now = 1.0f;
    // A value's code is that of the exact quotient: where the new rows set the scale (amax / 448, rounded) that is x * 448 /
    // amax, and x * 448 has 11 significant bits.  bf16 values meet the middle between two codes often (one in 40 of a
    // normal distribution's), and a rounded scale would put them on either side.
    const bool ours = fresh > 0.0f && now == fresh;
    const float shift = amax > 1.26765060e30f ? 5.42101086e-20f : 1.0f;  // 2^100, 2^-64: a product that does not overflow
    const float up = ours ? 448.0f * shift : 1.0f, down = ours ? amax * shift : now;
    uint8_t* cache = static_cast<uint8_t*>(a.cache) + (page * 128 * heads + head) * 128 + sub * 8;
    const long long row_bytes = static_cast<long long>(heads) * 128;
    __syncthreads();  // every thread has read the scale
    if (tid == 0) *scale_at = now;
    if (low > 0 && now != was) {
      for (int r = r0; r < low; r += 8) {
        uint2* c = reinterpret_cast<uint2*>(cache + r * row_bytes);
        const uint2 old = *c;
        const uint32_t w[2] = {old.x, old.y};
        uint32_t out[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f0 = from_e4m3x2(w[j] & 0xFFFFu), f1 = from_e4m3x2(w[j] >> 16);
          auto again = [&](float f) { return __fdiv_rn(f * up * was, down); };
          out[j] = to_e4m3x2(again(f0.x), again(f0.y)) | to_e4m3x2(again(f1.x), again(f1.y)) << 16;
        }
        *c = make_uint2(out[0], out[1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k * 8 + r0 >= len) continue;
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = to_e4m3x2(__fdiv_rn(__uint_as_float(w[j] << 16) * up, down),
                         __fdiv_rn(__uint_as_float(w[j] & 0xFFFF0000u) * up, down));
      *reinterpret_cast<uint2*>(cache + s_row[k * 8 + r0] * row_bytes) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
    at = start + 1;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_extend(const ExtendParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = launch_pdl(extend_plan_kernel, dim3(1), dim3(kTableThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (p.capacity == 0) return cudaSuccess;
  long long ctas = (p.capacity + kPlaceThreads - 1) / kPlaceThreads;
  if (ctas > sms * 8) ctas = sms * 8;
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

cudaError_t launch_append_fp8(const AppendParams& p, size_t clear_bytes, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(p.hdr, 0, clear_bytes, stream);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (p.tokens == 0) return cudaSuccess;
  // few tokens are mostly runs of their own (a decode step), many are prompts with a run per page: the CTAs of a chunk
  // without a run's first token end at once
  int chunk = 1;
  while (chunk < 64 && p.tokens > 512LL * chunk) chunk *= 2;
  int heads = 0;
  for (int i = 0; i < p.planes; ++i) heads += p.plane[i].width / 128;
  e = launch_pdl(append_fp8_kernel, dim3(static_cast<unsigned>((p.tokens + chunk - 1) / chunk), heads), dim3(kRunThreads),
                 0, stream, p, chunk);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace msa
