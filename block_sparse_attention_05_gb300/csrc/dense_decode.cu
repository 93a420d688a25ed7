// dense_decode.cu -- attention of one new token per sequence over every key of
// a paged cache (the full-attention layers beside the sparse ones), and the
// accumulation of each cached key's attention weight.
//
// For query head h of KV head g and cached key j (log2 units, c = scale * log2 e):
//   s[h,j] = c q_h . k_j,  m_h = max_j s,  l_h = sum_j 2^(s - m),
//   o_h = sum_j 2^(s - m) v_j / l_h,  lse_h = (m + log2 l) ln 2,
//   weight[g,j] += sum over the group's heads of 2^(s[h,j] - m_h) / l_h.
//
// Bound: K and V are read once; a key costs 4 * 128 G flops over 512 bytes in
// bf16, G flops a byte (2 G in E4M3).  HBM bounds groups of up to 16 heads.
// Larger ones are bound by what a unit costs its SM: those of 17 to 32 load, and in
// E4M3 widen, every fragment of K and V once per 16 heads (160 MB in bf16 36 us,
// 24 for the bytes; 80 MB in E4M3 34 to 36, 12 for the bytes), those above have the chain
// described at their kernel.
// Measured (16 heads to each of 4 KV heads): one sequence of 1,048,576 keys in
// bf16 314 us (6.8 TB/s), 24 ragged sequences of up to 65,521 in E4M3 123 us
// (5.9 TB/s; issuing the widening and the MMAs of 16 keys at a time is the rest),
// 200 short ones of up to 700 keys (40 heads to 8) 50 us (5.1 TB/s, with about
// 10 us of start, last units and join); 32 sequences of up to 16,384, calls back to
// back in a graph: 79 us, with weights 100 (72 for the bytes of K, V and weights), in
// E4M3 52 and 67: the logits, 64 bytes a key and KV head, are written beside K and V
// and read by a kernel behind the join.
//
// Work split: a unit is 64 keys of one sequence (128 in groups of more than 32
// heads).  All units of the batch, in
// order, are cut into `groups` equal runs and CTA (run, KV head) takes one:
// every CTA streams the same number of bytes whatever the lengths, and the CTAs
// of the KV heads walk the same pages at the same time (a page's rows hold all
// heads).  A sequence that lies inside one run is finished by its CTA; one that
// crosses runs leaves an unnormalised partial (O, m, l) per run, and the join
// kernel merges them.  A run has at most one sequence that continues from the
// run before and one that continues in the next, so two partial slots per CTA
// are enough whatever the batch.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

constexpr int kTile = kDenseTile;  // keys of a unit and of a ring stage (small groups)
constexpr float kLn2 = 0.6931471805599453f;
// A weight is 2^(s c - m) of an exact product and a maximum that is rounded, off by half the maximum's last place: 2^-14
// below this size of a logit in log2 units (710 nats), but without bound above it (2^127 from logits of 2^31).  Rows at or
// above it round their logits first: an fp32 softmax of fp32 logits, like that of the weights kernel, which reads them.
constexpr float kRoundLogits = 1024.0f;
// A product's factor with a page's scale in it, kept a normal number: 0 times a masked -inf, or inf times a product of 0,
// would be NaN.  A scale that is NaN stays it.
__device__ __forceinline__ float normal_factor(float c) {
  return c < 1.17549435e-38f ? 1.17549435e-38f : c > 3.40282347e38f ? 3.40282347e38f : c;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// D += A(16x16, row) * B(16x8, col), bf16 or fp16 inputs, fp32 accumulate.
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^(a - b) with 0 for a = -inf whatever b (b may be -inf too)
__device__ __forceinline__ float exp2_diff(float a, float b) {
  return a == -INFINITY ? 0.0f : exp2_approx(a - b);
}
// 1 / l of a sum of weights; 0 when every weight is 0 (all logits -inf), as for a row without keys
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
// what turns a logit of the row into its weight: (maximum, 1 / sum)
__device__ __forceinline__ float2 row_norm(float m, float l) {
  return make_float2(m == -INFINITY ? 0.0f : m, inverse(l));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// (a, b) >= 0 as a bf16 pair, cut off, plus a bf16 pair of the rest, rounded: 2^-16 of the value is lost at most (the
// rest of a value in [2^e, 2^(e+1)) is below 2^(e-7), half its last place 2^(e-16)).  Cutting off is a byte
// permutation where rounding takes the conversion unit a second time: 0.75 against 1.02 us a unit of 64 keys at 128
// heads.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  hi = __byte_perm(ua, ub, 0x7632);
  const float2 rest = ffma2(make_float2(__uint_as_float(ua & 0xFFFF0000u), __uint_as_float(ub & 0xFFFF0000u)),
                            make_float2(-1.0f, -1.0f), make_float2(a, b));
  lo = pack_bf16(rest.x, rest.y);
}
// two E4M3 codes (low 16 bits) -> fp16 pair; exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(codes)));
  return r;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------- the run of a CTA
struct Run {
  long long lo, hi, total;  // units [lo, hi) of `total`
  int runs;                 // runs that hold units: min(groups, total)
  int seq;                  // sequence of unit lo
  int off;                  // lo's unit within it
};
struct RunSmem {
  int warp_sum[32];
  int seq, off;
};

// Units of `1 << shift` keys in a sequence.
__device__ __forceinline__ int units_of(int len, int shift) { return (len + (1 << shift) - 1) >> shift; }

// Cuts the batch's units and finds run g of `groups`.  Every thread of the CTA
// calls it; returns false (for every thread) when cu_seqlens contradict the host
// sizes.  The CTA has passed a barrier when it returns.
__device__ bool find_run(const DenseDecodeParams& p, int g, RunSmem& sm, Run& r) {
  const int32_t* cu = p.cu_k;
  const int num_seqs = p.num_seqs, groups = p.groups, shift = p.unit_shift;
  const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = T >> 5;
  if (num_seqs <= 32) {  // each warp for itself, a sequence per lane
    const int start = lane < num_seqs ? cu[lane] : 0, stop = lane < num_seqs ? cu[lane + 1] : 0;
    const int len = stop - start;
    const bool bad = start < 0 || stop < start || len > p.max_k || (lane == 0 && start != 0) ||
                     (lane == num_seqs - 1 && stop != p.total_k);
    const int n = units_of(len, shift);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
    r.total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    r.runs = min(groups, static_cast<int>(r.total));
    r.lo = g < r.runs ? r.total * g / r.runs : r.total;
    r.hi = g < r.runs ? r.total * (g + 1) / r.runs : r.total;
    const uint32_t holds = __ballot_sync(0xFFFFFFFFu, incl > r.lo);  // the first such lane's sequence holds unit lo
    r.seq = holds ? __ffs(holds) - 1 : 0;
    r.off = static_cast<int>(r.lo - __shfl_sync(0xFFFFFFFFu, incl - n, r.seq));
    __syncthreads();
    return !any_bad;
  }
  const int per = (num_seqs + T - 1) / T;
  const int s0 = min(num_seqs, t * per), s1 = min(num_seqs, s0 + per);
  int sum = 0;
  bool bad = false;
  int prev = s0 < s1 ? cu[s0] : 0;
  if (t == 0) bad = prev != 0;
  for (int s = s0; s < s1; ++s) {
    const int next = cu[s + 1], len = next - prev;
    bad |= prev < 0 || next < prev || len > p.max_k || (s == num_seqs - 1 && next != p.total_k);
    sum += units_of(len, shift);
    prev = next;
  }
  if (__syncthreads_or(bad)) return false;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    const int v = sm.warp_sum[w];
    if (w < warp) base += v;
    total += v;
  }
  base += incl - sum;  // units before this thread's sequences
  r.total = total;
  r.runs = min(groups, total);
  r.lo = g < r.runs ? r.total * g / r.runs : r.total;
  r.hi = g < r.runs ? r.total * (g + 1) / r.runs : r.total;
  if (r.lo < r.hi && base <= r.lo && r.lo < base + sum) {  // one thread
    int u = base, s = s0;
    for (;; ++s) {
      const int n = units_of(cu[s + 1] - cu[s], shift);
      if (u + n > r.lo) break;
      u += n;
    }
    sm.seq = s;
    sm.off = static_cast<int>(r.lo - u);
  }
  __syncthreads();
  r.seq = sm.seq;
  r.off = sm.off;
  return true;
}

// Writes the empty sequences of a run's share (o = 0, lse = -inf): sequences g, g + groups, ..
__device__ __forceinline__ void write_empty(const DenseDecodeParams& p, int g, int head, int t, int threads) {
  const int G = p.group;
  for (int s = g; s < p.num_seqs; s += p.groups) {
    if (p.cu_k[s + 1] != p.cu_k[s]) continue;
    if (p.by_seq && t == 0) p.meta[s * p.hkv + head].x = -1;
    const long long row0 = (static_cast<long long>(s) * p.hkv + head) * G;
    for (int i = t; i < G * 16; i += threads)
      reinterpret_cast<uint4*>(p.o + row0 * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
    for (int i = t; i < G; i += threads) p.lse[row0 + i] = -INFINITY;
  }
}

// Walks a run's segments: the parts of its sequences that it covers.
struct Segment {
  int seq, len, off, count;  // units [off, off + count) of a sequence of `len` keys
  long long unit;            // the first one's number in the batch
  bool first, last;          // begins / ends the sequence
};
struct Walker {
  const int32_t* cu;
  long long at, hi;
  int seq, off, shift;
  __device__ Walker(const DenseDecodeParams& p, const Run& r)
      : cu(p.cu_k), at(r.lo), hi(r.hi), seq(r.seq), off(r.off), shift(p.unit_shift) {}
  __device__ bool next(Segment& g) {
    if (at >= hi) return false;
    int len, n;
    for (;;) {
      len = cu[seq + 1] - cu[seq];
      n = units_of(len, shift);
      if (off < n) break;
      ++seq;  // an empty sequence
      off = 0;
    }
    const long long left = hi - at;
    g.seq = seq;
    g.len = len;
    g.off = off;
    g.count = static_cast<int>(n - off < left ? n - off : left);
    g.unit = at;
    g.first = off == 0;
    g.last = off + g.count == n;
    at += g.count;
    ++seq;
    off = 0;
    return true;
  }
};

// ---------------------------------------------------------------- split kernel
// MG head tiles of 16 rows, each with KG compute warps, and one warp that feeds
// the ring.  A warp takes NS key tiles of 16 at a time (independent chains of
// MMAs, one softmax update for all of them): a unit's 64 keys are shared by
// 4 / NS of a head tile's warps, and KG / (4 / NS) such teams take the units in
// turn.  A ring stage always falls to the same team (stages are a multiple of
// the teams): a warp that had not waited for a stage's previous fill could take
// an older phase of its barrier for the next one.
template <int MG, bool FP8>
struct SplitCfg {
  static_assert(MG == 1 || MG == 2, "more heads: the tcgen05 kernel");
  static constexpr int kKG = 4;
  static constexpr int kNS = MG == 1 && !FP8 ? 1 : 2;
  static constexpr int kTeam = kTile / 16 / kNS;   // warps of a head tile that share a unit
  static constexpr int kTeams = kKG / kTeam;
  static_assert(kTeam * kTeams == kKG, "every warp belongs to a team");
  static constexpr int kWarps = MG * kKG;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kCtasPerSm = MG == 1 ? 2 : 1;
  static constexpr int kRowBytes = FP8 ? 128 : 256;
  static constexpr int kHalf = kTile * kRowBytes;  // K or V of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = (MG == 1 ? 3 : 6) * (FP8 ? 2 : 1);
  static_assert(kStages % kTeams == 0, "a stage's fills belong to one team");
  static constexpr int kExchange = kKG > 1 ? kWarps * 4096 : 0;  // half of each warp's O
  static constexpr int kMl = kWarps * 16 * 8;
  static constexpr size_t kSmem = kStages * kStage + kExchange + kMl + kStages * 24 + 16 + sizeof(RunSmem);
};

// Byte offset of (row, 16-byte chunk) in a stage's K or V: TMA's 128-byte
// swizzle; bf16 rows are two 64-dim halves, each kTile rows of 128 bytes.
__device__ __forceinline__ uint32_t tile_off(int row, int chunk) {
  return (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int MG, bool FP8, bool LOGITS>
__global__ void __launch_bounds__(SplitCfg<MG, FP8>::kThreads, SplitCfg<MG, FP8>::kCtasPerSm)
    dense_split_kernel(const __grid_constant__ DenseMaps maps, DenseDecodeParams p) {
  using C = SplitCfg<MG, FP8>;
  constexpr int KG = C::kKG, NS = C::kNS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  float* xch = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
  float2* ml = reinterpret_cast<float2*>(smem + C::kStages * C::kStage + C::kExchange);  // [warp][16] (m, l)
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage + C::kExchange + C::kMl);
  uint64_t* empty = full + C::kStages;
  float2* scales = reinterpret_cast<float2*>(empty + C::kStages);  // fp8: the stage's K scale and log2 of its V scale
  int* abort_flag = reinterpret_cast<int*>(scales + C::kStages);
  uint32_t* err = reinterpret_cast<uint32_t*>(abort_flag + 1);
  RunSmem& run_sm = *reinterpret_cast<RunSmem*>(err + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % p.hkv, g = blockIdx.x / p.hkv;
  const int G = p.group;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], MG * C::kTeam);
    }
    *abort_flag = 0;
    *err = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  griddep_wait();  // set up while the kernel before it ends
  Run run;
  const bool fine = find_run(p, g, run_sm, run);  // synchronises
  if (!fine) {
    if (threadIdx.x == 0) {
      p.flags[blockIdx.x] = kFlagBadSeqlens;
      if (!p.by_seq) p.meta[blockIdx.x].x = -1;
    }
    if (p.by_seq && g < p.num_seqs && threadIdx.x == 0) p.meta[g * p.hkv + head].x = -1;  // num_seqs <= groups
    return;
  }

  Walker walk(p, run);
  Segment sg;
  uint32_t issued = 0;  // the feeding lane's fills
  if (warp == C::kWarps) {
    // ------------------------------------------------------------ producer
    uint32_t fills = 0, bad = 0;
    const uint64_t policy = l2_evict_first();  // with logits: K and V pass through, the logits are to stay in L2
    bool stopped = false;
    while (!stopped && walk.next(sg)) {
      const int first_page = sg.off * kTile / kBlock, last_page = (sg.off + sg.count - 1) * kTile / kBlock;
      const int32_t* table = p.block_table + static_cast<long long>(sg.seq) * p.bt_stride;
      int base = first_page;
      int row = 0;
      float sk = 1.0f, sv = 1.0f;
      for (int u = sg.off; u < sg.off + sg.count; ++u) {
        const int page = u * kTile / kBlock;
        if (u == sg.off || page - base >= 32) {  // the next 32 pages' rows and scales, one per lane
          if (u != sg.off) base += 32;
          row = 0;
          if (base + lane <= last_page) {
            const int e = table[base + lane];
            if (e < 0 || e >= p.n_pages) {
              bad = 1;
              row = static_cast<int>(p.n_pages) * kBlock;  // past the cache: TMA reads zeros
            } else {
              row = e * kBlock;
              if (FP8) {
                sk = p.k_scale[static_cast<long long>(e) * p.hkv + head];
                sv = p.v_scale[static_cast<long long>(e) * p.hkv + head];
              }
            }
          }
        }
        const int r = __shfl_sync(0xFFFFFFFFu, row, page - base) + (u * kTile) % kBlock;
        float tk = 1.0f, tv = 1.0f;
        if (FP8) {
          tk = __shfl_sync(0xFFFFFFFFu, sk, page - base);
          tv = __shfl_sync(0xFFFFFFFFu, sv, page - base);
        }
        if (lane == 0) {
          const int st = fills % C::kStages;
          const uint32_t n = fills / C::kStages;
          if (n > 0 && !mbar_wait(&empty[st], (n - 1) & 1, abort_flag)) {
            *abort_flag = 1;
            atomicOr(err, kFlagTimeout);
          } else {
            uint8_t* dk = ring + st * C::kStage;
            uint8_t* dv = dk + C::kHalf;
            if (FP8) scales[st] = make_float2(tk, tv == 0.0f ? -160.0f : log2f(tv));
            auto load = [&](uint8_t* dst, const CUtensorMap* map, int dim, int row) {
              if (LOGITS) tma_load_3d_policy(dst, map, &full[st], dim, head, row, policy);
              else tma_load_3d(dst, map, &full[st], dim, head, row);
            };
            const int valid = sg.len - u * kTile;
            if (valid > kTile - kDenseTail) {
              mbar_arrive_expect_tx(&full[st], C::kStage);
              load(dk, &maps.k, 0, r);
              if (!FP8) load(dk + kTile * 128, &maps.k, 64, r);
              load(dv, &maps.v, 0, r);
              if (!FP8) load(dv + kTile * 128, &maps.v, 64, r);
            } else {  // a sequence's last unit: only as many rows as hold keys, 16 at a time
              const int boxes = (valid + kDenseTail - 1) / kDenseTail;
              mbar_arrive_expect_tx(&full[st], boxes * kDenseTail * 2 * C::kRowBytes);
              for (int b = 0; b < boxes; ++b) {
                const int at = b * kDenseTail * 128, row = r + b * kDenseTail;
                load(dk + at, &maps.k_tail, 0, row);
                if (!FP8) load(dk + kTile * 128 + at, &maps.k_tail, 64, row);
                load(dv + at, &maps.v_tail, 0, row);
                if (!FP8) load(dv + kTile * 128 + at, &maps.v_tail, 64, row);
              }
            }
            ++issued;
          }
        }
        stopped = __any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(abort_flag)) != 0;
        if (stopped) break;
        ++fills;
      }
    }
    if (bad) atomicOr(err, kFlagBadIndex);
  } else {
    // ------------------------------------------------------------ compute
    const int mg = warp / KG, kg = warp % KG;
    const int t4 = lane & 3, r0 = mg * 16 + (lane >> 2), r1 = r0 + 8;  // this thread's two head rows
    write_empty(p, g, head, threadIdx.x, 32 * C::kWarps);
    uint32_t fills = 0;
    bool ok = true;
    const int team = kg / C::kTeam;
    int4 crossing = make_int4(-1, 0, 0, 0);  // the sequence that begins in this run and goes on
    while (walk.next(sg)) {
      // Q fragments (A operand).  bf16: dims 16 kk + 2 t4 (+ 8); fp8: the order
      // in which a 4-byte word of codes widens, dims 16 kk + 4 t4 .. + 3, as
      // fp16 scaled per row by the power of two that brings max |q| to [1, 2)
      // (exact but for values 2^-24 below the row's largest).
      uint32_t qa[8][4];
      float qs0 = p.scale_log2, qs1 = p.scale_log2;
      {
        const __nv_bfloat16* q = p.q + (static_cast<long long>(sg.seq) * p.hkv + head) * G * kHeadDim;
        const uint32_t* q0 = reinterpret_cast<const uint32_t*>(q + r0 * kHeadDim);
        const uint32_t* q1 = reinterpret_cast<const uint32_t*>(q + r1 * kHeadDim);
        if (!FP8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qa[kk][0] = r0 < G ? q0[8 * kk + t4] : 0;
            qa[kk][1] = r1 < G ? q1[8 * kk + t4] : 0;
            qa[kk][2] = r0 < G ? q0[8 * kk + 4 + t4] : 0;
            qa[kk][3] = r1 < G ? q1[8 * kk + 4 + t4] : 0;
          }
        } else {
          uint32_t m0 = 0, m1 = 0;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qa[kk][0] = r0 < G ? q0[8 * kk + 2 * t4] : 0;
            qa[kk][1] = r1 < G ? q1[8 * kk + 2 * t4] : 0;
            qa[kk][2] = r0 < G ? q0[8 * kk + 2 * t4 + 1] : 0;
            qa[kk][3] = r1 < G ? q1[8 * kk + 2 * t4 + 1] : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t w = max(qa[kk][j] & 0x7FFFu, (qa[kk][j] >> 16) & 0x7FFFu);
              if (j & 1) m1 = max(m1, w); else m0 = max(m0, w);
            }
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            m0 = max(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
            m1 = max(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, o));
          }
          // exponent of the row's largest value, 0 for zero, subnormal, inf or NaN rows
          const int x0 = static_cast<int>(m0 >> 7), x1 = static_cast<int>(m1 >> 7);
          const int e0 = (x0 > 0 && x0 < 255) ? min(max(x0 - 127, -120), 120) : 0;
          const int e1 = (x1 > 0 && x1 < 255) ? min(max(x1 - 127, -120), 120) : 0;
          const float i0 = __uint_as_float(static_cast<uint32_t>(127 - e0) << 23);
          const float i1 = __uint_as_float(static_cast<uint32_t>(127 - e1) << 23);
          qs0 *= __uint_as_float(static_cast<uint32_t>(127 + e0) << 23);
          qs1 *= __uint_as_float(static_cast<uint32_t>(127 + e1) << 23);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = (j & 1) ? i1 : i0;
              qa[kk][j] = pack_f16(__uint_as_float(qa[kk][j] << 16) * f,
                                   __uint_as_float(qa[kk][j] & 0xFFFF0000u) * f);
            }
        }
      }
      float o[16][4];
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      float ref0 = -INFINITY, ref1 = -INFINITY;  // fp8: O's own reference, less m (see below)

      for (int u = sg.off; u < sg.off + sg.count; ++u, ++fills) {
        if (C::kTeams > 1 && static_cast<int>(fills % C::kTeams) != team) continue;
        const int st = fills % C::kStages;
        if (ok && !mbar_wait_warp(&full[st], (fills / C::kStages) & 1, abort_flag)) {
          ok = false;  // keep walking: the segments' barriers below need every warp
          if (lane == 0) {
            *reinterpret_cast<volatile int*>(abort_flag) = 1;
            atomicOr(err, kFlagTimeout);
          }
        }
        if (!ok) continue;
        const uint32_t kt = smem_u32(ring + st * C::kStage), vt = kt + C::kHalf;
        const int key0 = kg % C::kTeam * (NS * 16);
        const int valid = sg.len - u * kTile - key0;  // keys of this warp's share that exist (may exceed it)
        if (valid > 0) {                              // uniform in the warp
          float c0 = qs0, c1 = qs1, lv = 0.0f;
          if (FP8) {
            const float2 sc = scales[st];
            c0 = normal_factor(c0 * sc.x);
            c1 = normal_factor(c1 * sc.x);
            lv = sc.y;
          }
          // s[j]: keys key0 + 8 j + 2 t4 (+ 1) of rows r0 and r1
          float s[2 * NS][4];
#pragma unroll
          for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = 0.0f;
          const int krow = key0 + (lane & 7) + ((lane >> 4) << 3);
          if (!FP8) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                uint32_t b[4];
                ldsm_x4(kt + tile_off(krow + 16 * n, 2 * kk + ((lane >> 3) & 1)), b);
                mma16<false>(s[2 * n], qa[kk], b[0], b[1]);
                mma16<false>(s[2 * n + 1], qa[kk], b[2], b[3]);
              }
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; kk += 2)  // one load: 16-byte chunks kk and kk + 1 of 16 keys
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                uint32_t b[4];
                ldsm_x4(kt + tile_off(krow + 16 * n, kk + ((lane >> 3) & 1)), b);
                mma16<true>(s[2 * n], qa[kk], e4m3x2_to_f16x2(b[0]), e4m3x2_to_f16x2(b[0] >> 16));
                mma16<true>(s[2 * n + 1], qa[kk], e4m3x2_to_f16x2(b[2]), e4m3x2_to_f16x2(b[2] >> 16));
                mma16<true>(s[2 * n], qa[kk + 1], e4m3x2_to_f16x2(b[1]), e4m3x2_to_f16x2(b[1] >> 16));
                mma16<true>(s[2 * n + 1], qa[kk + 1], e4m3x2_to_f16x2(b[3]), e4m3x2_to_f16x2(b[3] >> 16));
              }
          }
          const bool tail = valid < NS * 16;
          if (tail) {
#pragma unroll
            for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (8 * j + 2 * t4 + i >= valid) s[j][i] = s[j][2 + i] = -INFINITY;
          }
          auto round_logits = [&](float f0, float f1) {
#pragma unroll
            for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                s[j][i] = __fmul_rn(s[j][i], f0);
                s[j][2 + i] = __fmul_rn(s[j][2 + i], f1);
              }
          };
          if (LOGITS) {
            round_logits(c0, c1);
            c0 = c1 = 1.0f;
            float* w = p.logits + ((sg.unit + (u - sg.off)) * p.hkv + head) * static_cast<long long>(G) * kTile +
                       key0 + 2 * t4;
#pragma unroll
            for (int j = 0; j < 2 * NS; ++j) {
              if (r0 < G) *reinterpret_cast<float2*>(w + r0 * kTile + 8 * j) = make_float2(s[j][0], s[j][1]);
              if (r1 < G) *reinterpret_cast<float2*>(w + r1 * kTile + 8 * j) = make_float2(s[j][2], s[j][3]);
            }
          } else if (FP8) {
            // Products of a query of less than 2 and a code are below 2^17, logits below 2^16 with a factor under a half
            // (off by 2^-8 at most, which the fp16 weights have room for).  The factor is known ahead of the products; a
            // look at the maximum behind them holds up the exponentials (24 sequences of up to 65,521: 125.1 -> 126.6 us).
            const bool large0 = c0 >= 0.5f, large1 = c1 >= 0.5f;
            if (__any_sync(0xFFFFFFFFu, large0 || large1)) {
              round_logits(large0 ? c0 : 1.0f, large1 ? c1 : 1.0f);
              if (large0) c0 = 1.0f;
              if (large1) c1 = 1.0f;
            }
          }
          float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2 * NS; ++j) {
            x0 = fmax3(x0, s[j][0], s[j][1]);
            x1 = fmax3(x1, s[j][2], s[j][3]);
          }
#pragma unroll
          for (int of = 1; of < 4; of <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, of));
            x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, of));
          }
          const float n0 = fmaxf(m0, x0 * c0), n1 = fmaxf(m1, x1 * c1);  // the factors are positive
          const float e0 = n0 == -INFINITY ? 0.0f : n0, e1 = n1 == -INFINITY ? 0.0f : n1;
          const float d0 = m0 - e0, d1 = m1 - e1;  // -inf while no key counts
          float a0 = exp2_approx(d0), a1 = exp2_approx(d1);
          l0 *= a0;
          l1 *= a1;
          m0 = n0;
          m1 = n1;
          // fp8: O is kept relative to a reference of its own, the running maximum
          // of m + log2(V scale), so that the weights of the codes fit fp16 whatever
          // the pages' scales: at most 2^14, with fp16's full 11 bits down to
          // 2^-28 of the largest.  It is held as its distance from m, a small
          // number that a large m does not round (-inf again after units without
          // a key that counts).
          float f0 = 1.0f, f1 = 1.0f;
          if (FP8) {
            ref0 += d0;
            ref1 += d1;
            const float y0 = fmaxf(ref0, lv), y1 = fmaxf(ref1, lv);
            a0 = exp2_approx(ref0 - y0);
            a1 = exp2_approx(ref1 - y1);
            ref0 = y0;
            ref1 = y1;
            f0 = exp2_approx(lv + 14.0f - y0);
            f1 = exp2_approx(lv + 14.0f - y1);
          }
          const bool look = !LOGITS && !FP8;
          const bool big0 = look && fabsf(n0) >= kRoundLogits, big1 = look && fabsf(n1) >= kRoundLogits;
          if (__any_sync(0xFFFFFFFFu, a0 != 1.0f || a1 != 1.0f || big0 || big1)) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              o[j][0] *= a0; o[j][1] *= a0; o[j][2] *= a1; o[j][3] *= a1;
            }
            if (look && __any_sync(0xFFFFFFFFu, big0 || big1)) {  // rare; each row for itself
              round_logits(big0 ? c0 : 1.0f, big1 ? c1 : 1.0f);
              if (big0) c0 = 1.0f;
              if (big1) c1 = 1.0f;
            }
          }
#pragma unroll
          for (int j = 0; j < 2 * NS; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s[j][i] = exp2_approx(fmaf(s[j][i], c0, -e0));
              s[j][2 + i] = exp2_approx(fmaf(s[j][2 + i], c1, -e1));
            }
            l0 += s[j][0] + s[j][1];
            l1 += s[j][2] + s[j][3];
          }
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            // P as the A operand.  bf16 V: the weights as a bf16 value and the bf16
            // rest (16 significant bits; one bf16 alone would add half as much error
            // again as the output's own rounding).  fp8: one fp16 value.
            uint32_t ph[4], pl[4];
            const float(&w0)[4] = s[2 * n], (&w1)[4] = s[2 * n + 1];
            if (!FP8) {
              split_bf16(w0[0], w0[1], ph[0], pl[0]);
              split_bf16(w0[2], w0[3], ph[1], pl[1]);
              split_bf16(w1[0], w1[1], ph[2], pl[2]);
              split_bf16(w1[2], w1[3], ph[3], pl[3]);
            } else {
              ph[0] = pack_f16(w0[0] * f0, w0[1] * f0);
              ph[1] = pack_f16(w0[2] * f1, w0[3] * f1);
              ph[2] = pack_f16(w1[0] * f0, w1[1] * f0);
              ph[3] = pack_f16(w1[2] * f1, w1[3] * f1);
            }
            // rows past the sequence's end hold anything (0 * NaN): V words of such keys become 0
            uint32_t k0 = 0xFFFFFFFFu, k1 = 0xFFFFFFFFu;
            if (tail) {
              const int a = valid - 16 * n - 2 * t4, b = a - 8;
              k0 = a >= 2 ? 0xFFFFFFFFu : a == 1 ? 0xFFFFu : 0u;
              k1 = b >= 2 ? 0xFFFFFFFFu : b == 1 ? 0xFFFFu : 0u;
            }
            const int vrow = key0 + 16 * n + (lane & 7) + (((lane >> 3) & 1) << 3);
            if (!FP8) {
#pragma unroll
              for (int j = 0; j < 16; j += 2) {  // dims 8 j .. 8 j + 15
                uint32_t b[4];
                ldsm_x4_trans(vt + tile_off(vrow, j + (lane >> 4)), b);
                b[0] &= k0; b[1] &= k1; b[2] &= k0; b[3] &= k1;
                mma16<false>(o[j], ph, b[0], b[1]);
                mma16<false>(o[j + 1], ph, b[2], b[3]);
                mma16<false>(o[j], pl, b[0], b[1]);
                mma16<false>(o[j + 1], pl, b[2], b[3]);
              }
            } else {
              // A 16-bit word of the transposed load is two adjacent dims of one
              // key, so a register holds (key 2 t4: dims d, d + 1; key 2 t4 + 1:
              // d, d + 1) with d = 16 c + 2 (lane / 4): accumulator tile 2 c takes
              // the even dims of chunk c, tile 2 c + 1 the odd ones.
#pragma unroll
              for (int c = 0; c < 8; c += 2) {
                uint32_t b[4];
                ldsm_x4_trans(vt + tile_off(vrow, c + (lane >> 4)), b);
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = __byte_perm(b[i] & ((i & 1) ? k1 : k0), 0, 0x3120);
                mma16<true>(o[2 * c], ph, e4m3x2_to_f16x2(b[0]), e4m3x2_to_f16x2(b[1]));
                mma16<true>(o[2 * c + 1], ph, e4m3x2_to_f16x2(b[0] >> 16), e4m3x2_to_f16x2(b[1] >> 16));
                mma16<true>(o[2 * c + 2], ph, e4m3x2_to_f16x2(b[2]), e4m3x2_to_f16x2(b[3]));
                mma16<true>(o[2 * c + 3], ph, e4m3x2_to_f16x2(b[2] >> 16), e4m3x2_to_f16x2(b[3] >> 16));
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }

      // ---- merge of the segment's KG key shares
#pragma unroll
      for (int of = 1; of < 4; of <<= 1) {
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, of);
        l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, of);
      }
      float b0 = 1.0f, b1 = 1.0f;  // factor of this warp's O
      if (FP8) {
        b0 = exp2_approx(ref0 - 14.0f);
        b1 = exp2_approx(ref1 - 14.0f);
      }
      if (KG > 1) {
        if (t4 == 0) {
          ml[warp * 16 + (lane >> 2)] = make_float2(m0, l0);
          ml[warp * 16 + 8 + (lane >> 2)] = make_float2(m1, l1);
        }
        named_sync(1 + mg, 32 * KG);
        float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          M0 = fmaxf(M0, ml[(mg * KG + k) * 16 + (lane >> 2)].x);
          M1 = fmaxf(M1, ml[(mg * KG + k) * 16 + 8 + (lane >> 2)].x);
        }
        float L0 = 0.0f, L1 = 0.0f;
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const float2 a = ml[(mg * KG + k) * 16 + (lane >> 2)], b = ml[(mg * KG + k) * 16 + 8 + (lane >> 2)];
          L0 += a.y * exp2_diff(a.x, M0);
          L1 += b.y * exp2_diff(b.x, M1);
        }
        b0 *= exp2_diff(m0, M0);
        b1 *= exp2_diff(m1, M1);
        m0 = M0; m1 = M1; l0 = L0; l1 = L1;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= b0; o[j][1] *= b0; o[j][2] *= b1; o[j][3] *= b1;
      }
      // Butterfly: partners swap halves of their accumulator tiles, so that after
      // log2(KG) steps warp kg holds the sums of 16 / KG tiles from `tile0`.
      int tile0 = 0;
      float* mine = xch + warp * 1024 + lane;
      if (KG > 1) {
        constexpr int d = KG / 2;
        const bool upper = (kg & d) != 0;
        const float* theirs = xch + (warp ^ d) * 1024 + lane;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[(j * 4 + i) * 32] = upper ? o[j][i] : o[j + 8][i];
        named_sync(1 + mg, 32 * KG);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] = (upper ? o[j + 8][i] : o[j][i]) + theirs[(j * 4 + i) * 32];
        tile0 = upper ? 8 : 0;
      }
      if (KG > 2) {
        const bool upper = (kg & 1) != 0;
        const float* theirs = xch + (warp ^ 1) * 1024 + lane;
        named_sync(1 + mg, 32 * KG);  // the first step's values are read
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[(j * 4 + i) * 32] = upper ? o[j][i] : o[j + 4][i];
        named_sync(1 + mg, 32 * KG);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] = (upper ? o[j + 4][i] : o[j][i]) + theirs[(j * 4 + i) * 32];
        tile0 += upper ? 4 : 0;
      }

      // ---- the finished output, or this run's partial
      const bool whole = sg.first && sg.last;
      const long long out_row = (static_cast<long long>(sg.seq) * p.hkv + head) * G;
      const long long part_row = (static_cast<long long>(blockIdx.x) * 2 + (sg.first ? 1 : 0)) * G;
      const float v0 = whole ? inverse(l0) : 1.0f, v1 = whole ? inverse(l1) : 1.0f;
#pragma unroll
      for (int j = 0; j < 16 / KG; j += 2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = half ? r1 : r0;
          const float f = half ? v1 : v0;
          // four values and the dims of the first two and the last two
          float w[4];
          int da, db;
          if (!FP8) {
            w[0] = o[j][2 * half] * f; w[1] = o[j][2 * half + 1] * f;
            w[2] = o[j + 1][2 * half] * f; w[3] = o[j + 1][2 * half + 1] * f;
            da = (tile0 + j) * 8 + 2 * t4;
            db = da + 8;
          } else {
            w[0] = o[j][2 * half] * f; w[1] = o[j + 1][2 * half] * f;
            w[2] = o[j][2 * half + 1] * f; w[3] = o[j + 1][2 * half + 1] * f;
            da = (tile0 + j) * 8 + 4 * t4;
            db = da + 2;
          }
          if (r < G) {
            if (whole) {
              uint32_t* d = reinterpret_cast<uint32_t*>(p.o + (out_row + r) * kHeadDim);
              d[da >> 1] = pack_bf16(w[0], w[1]);
              d[db >> 1] = pack_bf16(w[2], w[3]);
            } else {
              float* d = p.part_o + (part_row + r) * kHeadDim;
              *reinterpret_cast<float2*>(d + da) = make_float2(w[0], w[1]);
              *reinterpret_cast<float2*>(d + db) = make_float2(w[2], w[3]);
            }
          }
        }
      }
      if (kg == 0 && t4 == 0) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = half ? r1 : r0;
          const float m = half ? m1 : m0, l = half ? l1 : l0;
          if (r < G) {
            if (whole) {
              p.lse[out_row + r] = (m + log2f(l)) * kLn2;
              if (LOGITS) p.norm[out_row + r] = row_norm(m, l);
            } else {
              p.part_ml[part_row + r] = make_float2(m, l);
            }
          }
        }
      }
      if (sg.first && !sg.last) {
        // the run that holds the sequence's last unit: lo(x) = floor(total x / runs) <= u < lo(x + 1)
        const long long end = sg.unit + units_of(sg.len, p.unit_shift) - 1;
        crossing = make_int4(sg.seq, g, static_cast<int>(((end + 1) * run.runs - 1) / run.total), 0);
      }
      if (p.by_seq && sg.first && warp == 0 && lane == 0)
        p.meta[sg.seq * p.hkv + head] = sg.last ? make_int4(-1, 0, 0, 0) : crossing;
    }
    if (!p.by_seq && warp == 0 && lane == 0) p.meta[blockIdx.x] = crossing;
  }
  __syncthreads();
  if (*abort_flag && issued > 0)  // no copy may land after this CTA has left
    for (uint32_t f = issued > C::kStages ? issued - C::kStages : 0; f < issued; ++f)
      mbar_wait(&full[f % C::kStages], (f / C::kStages) & 1, nullptr);
  if (threadIdx.x == 0) p.flags[blockIdx.x] = *err;
}

// ---------------------------------------------------------------- split kernel, large groups
// Groups of many heads on the 5th-generation tensor cores: the group's heads are
// the 128 rows of the MMAs (rows past the group hold zero queries), a unit's 128
// keys (a page) their columns.
//   S = Q K^T    128 x 128 x 128
//   P = 2^(S c - m)   one row per thread; written over S in TMEM as a bf16 value
//                and the bf16 rest (16 significant bits), the A operand of
//   O += P V     128 x 128 x 128, twice (value and rest), accumulated in TMEM
// m is a row's reference, not its maximum: a whole number, the first unit's maximum
// rounded up, and O and l are rescaled, by an exact power of two, only when a unit's
// maximum passes it by more than 2^8.
//
// Per unit (64 KB of K and V, 1.4 us of an SM's share of HBM) the MMAs take 0.8 us
// alone and a warpgroup's softmax 1.5 us, so two warpgroups take the units in turn,
// each with its own S and O in TMEM (2 x (128 + 128) columns), m and l, merged at
// the end of a segment: one computes P while the other's MMAs run.  What bounds it is
// that chain: under each other's traffic S takes 0.45, the softmax 1.5, P V 1.2 and
// the hand-offs 0.35 us, two chains in flight, a unit every 1.8 us (5.6 TB/s over the
// SMs).  No one link carries it (P V without the rests 8 % faster, the softmax without
// its maximum 5 %, four warpgroups with half the softmax each or P V begun at half of
// P no faster), and TMEM has no columns for a third S beside two O.  200,000 keys of 8 sequences, 128 heads: 33 us, and
// 5 for the join (bytes: 15).
// Units of 64 keys ran at half this rate: an MMA with 64 columns takes as long as
// one with 128, and issuing it and the commits (about 250 clocks each) held up the
// one thread that does; here a unit has two commits, S done (K's stage is free,
// its warpgroup may go on) and P V done (V's stage and S's columns are free).
//
// E4M3 pages: the codes land in a ring of their own (two stages) and each softmax
// warpgroup widens its units' while it waits for its MMAs, K to bf16 (the queries'
// type) and V to fp16, both exact; the weights times the page's V scale are one
// fp16 value, so P V is one product.  Once widened a code meets all heads: 41 us
// for 80 MB of K and V where the small groups' kernel, which widens them for every
// 16 heads, took 87 us at 128 heads and 51 us at 64.
//
// Warps: 0 feeds K and 3 feeds V (TMA), 1 issues the MMAs, 2 owns TMEM and feeds
// Q, 4..7 and 8..11 softmax and output.
template <bool FP8>
struct TcCfg {
  static constexpr int kThreads = 384;
  static constexpr int kKeys = 128;
  static constexpr int kStages = FP8 ? 2 : 3;
  static constexpr int kCodes = kKeys * 128;  // fp8: K or V of a stage as it lands
  static constexpr int kHalf = kKeys * 256;  // K or V of a stage
  static constexpr uint32_t kColS = 0, kColO = 256;
};
struct TcSmem {
  uint64_t k_full[3], v_full[3];
  uint64_t k_empty[2], v_empty[2], k_ready[2], v_ready[2];  // fp8: codes read, values written
  // S done by unit % 6: a stage's and a warpgroup's units each keep to barriers of their own, so every waiter sees
  // every phase of the barriers it uses (one that skipped a phase could take an older one for its own)
  uint64_t s_done[6];
  uint64_t pv_done[3];
  uint64_t p_full[2];
  uint64_t q_full, q_empty, ml_full, o_free, mma_done;
  float2 ml[2][128];  // (m, l) of each warpgroup's rows; m = -inf: no unit of the segment was its own, or no key counts
  short d[2][128];    // fp8: exponent of O
  float scale[2][2];  // fp8: a stage's scales of K and V
  RunSmem run;
  uint32_t tmem_base;
  int abort_flag;
  uint32_t err;
};
constexpr size_t kTcSmemBytes = 7 * 32768 + sizeof(TcSmem);  // three stages and Q; or two, two of codes and Q
static_assert(kTcSmemBytes <= 227 * 1024, "one CTA's shared memory");

// Multiplies this thread's row of O or S (128 TMEM columns) by f.  Rare; out of line to leave the softmax its registers.
__device__ __noinline__ void scale_row(uint32_t addr, float f) {
  for (int c = 0; c < 128; c += 8) {
    uint32_t w[8];
    tmem_ld_8cols(addr + c, w);
    tmem_ld_wait_regs8(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
    tmem_st_8cols(addr + c, w);
  }
  tmem_st_wait();
}

// Element i of lane t4 of four goes to element t4 of lane i.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4], int t4) {
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, t4 & d ? x[i] : x[i | d], d);
      if (t4 & d) x[i] = got;
      else x[i | d] = got;
    }
}

// 16 rows (TMEM lanes, from a multiple of 16) of 32 columns: registers 4 i + {0, 1} hold columns 8 i + 2 (lane % 4) +
// {0, 1} of row lane / 4, registers 4 i + {2, 3} those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16rows_32cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait_regs16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 16-byte pieces of a unit's codes (rows of 128 bytes, TMA's 128-byte swizzle) to 16-bit values in the layout in which
// TMA lands bf16 rows: K as bf16 (the queries' type), V as fp16 (the weights' type), both exact.  128 threads; eight
// lanes read a row, and those of its second half write their pieces in the other order, so that eight lanes' stores
// meet all banks.  Rows from `valid` on become zeros (V: 0 * NaN is NaN).
template <bool BF16>
__device__ __forceinline__ void widen(const uint8_t* codes, uint8_t* to, int thread, int valid) {
  const int chunk = thread & 7, half = chunk >> 2;
  const uint32_t flip = half;
#pragma unroll 1  // two or more at once hold up the MMAs' reads of shared memory (2 to 8 % slower)
  for (int row = thread >> 3; row < 128; row += 16) {
    const int x = row & 7;
    uint4 in = *reinterpret_cast<const uint4*>(codes + row * 128 + ((chunk ^ x) << 4));
    if (row >= valid) in = make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      out[j] = e4m3x2_to_f16x2(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
      if (BF16) {  // four significant bits: the upper half of the value in fp32
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&out[j]));
        out[j] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(to + half * 16384 + row * 128);
    const uint4 a = make_uint4(out[0], out[1], out[2], out[3]), b = make_uint4(out[4], out[5], out[6], out[7]);
    const uint32_t at = 2 * (chunk & 3);
    dst[(at + flip) ^ x] = flip ? b : a;
    dst[(at + 1 - flip) ^ x] = flip ? a : b;
  }
}

template <bool FP8, bool LOGITS>
__global__ void __launch_bounds__(TcCfg<FP8>::kThreads, 1)
    dense_split_tc_kernel(const __grid_constant__ DenseMaps maps, DenseDecodeParams p) {
  using C = TcCfg<FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;                                     // stages of K and V: two 64-dim halves of 128 rows each
  uint8_t* codes = smem + C::kStages * 2 * C::kHalf;        // fp8: stages of K and V as they land
  uint8_t* q_buf = smem + 6 * 32768;                        // as the ring
  TcSmem& sm = *reinterpret_cast<TcSmem*>(q_buf + C::kHalf);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % p.hkv, g = blockIdx.x / p.hkv;
  const int G = p.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < 6; ++i) mbar_init(&sm.s_done[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.k_empty[i], 4);
      mbar_init(&sm.v_empty[i], 4);
      mbar_init(&sm.k_ready[i], 4);
      mbar_init(&sm.v_ready[i], 4);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.ml_full, 8);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.mma_done, 1);
    sm.abort_flag = 0;
    sm.err = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.q);
  }
  // queries of the rows past the group: zero once, the loads write the group's rows only
  for (int i = threadIdx.x; i < (128 - G) * 16; i += C::kThreads)
    reinterpret_cast<uint4*>(q_buf + (i & 8) * 2048)[G * 8 + (i >> 4) * 8 + (i & 7)] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  griddep_wait();  // set up while the kernel before it ends
  Run run;
  const bool fine = find_run(p, g, sm.run, run);  // synchronises
  if (!fine) {
    if (threadIdx.x == 0) {
      p.flags[blockIdx.x] = kFlagBadSeqlens;
      if (!p.by_seq) p.meta[blockIdx.x].x = -1;
    }
    if (p.by_seq && g < p.num_seqs && threadIdx.x == 0) p.meta[g * p.hkv + head].x = -1;  // num_seqs <= groups
    return;
  }
  if (warp == 2) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  auto gave_up = [&] {
    *abort_flag = 1;
    atomicOr(&sm.err, kFlagTimeout);
  };

  Walker walk(p, run);
  Segment sg;
  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ producers: K, V
    const CUtensorMap* map = warp == 0 ? &maps.k : &maps.v;
    uint64_t* full = warp == 0 ? sm.k_full : sm.v_full;
    constexpr int kTileBytes = FP8 ? C::kCodes : C::kHalf;
    uint8_t* const dst0 = (FP8 ? codes : ring) + (warp == 0 ? 0 : kTileBytes);
    uint64_t* const empty = warp == 0 ? sm.k_empty : sm.v_empty;
    const float* const scale = warp == 0 ? p.k_scale : p.v_scale;
    uint32_t fills = 0, issued = 0, bad = 0;
    const uint64_t policy = l2_evict_first();  // with logits: K and V pass through, the logits are to stay in L2
    bool stopped = false;
    while (!stopped && walk.next(sg)) {
      const int32_t* table = p.block_table + static_cast<long long>(sg.seq) * p.bt_stride + sg.off;
      int row = 0;
      float s = 1.0f;
      for (int i = 0; i < sg.count; ++i) {
        if ((i & 31) == 0) {  // the next 32 pages' rows and scales, one per lane
          row = 0;
          s = 1.0f;
          if (i + lane < sg.count) {
            const int e = table[i + lane];
            if (e < 0 || e >= p.n_pages) {
              bad = 1;
              row = static_cast<int>(p.n_pages) * kBlock;  // past the cache: TMA reads zeros
            } else {
              row = e * kBlock;
              if (FP8) s = scale[static_cast<long long>(e) * p.hkv + head];
            }
          }
        }
        const int r = __shfl_sync(0xFFFFFFFFu, row, i & 31);
        const float sc = FP8 ? __shfl_sync(0xFFFFFFFFu, s, i & 31) : 1.0f;
        if (lane == 0) {
          const int st = fills % C::kStages;
          bool free = true;  // the stage's last unit is done with
          if (fills >= C::kStages) {
            const uint32_t u = fills - C::kStages;
            free = FP8         ? mbar_wait(&empty[st], (u / C::kStages) & 1, abort_flag)
                   : warp == 0 ? mbar_wait(&sm.s_done[u % 6], (u / 6) & 1, abort_flag)
                               : mbar_wait(&sm.pv_done[st], (u / C::kStages) & 1, abort_flag);
          }
          if (!free) {
            gave_up();
          } else {
            uint8_t* dst = dst0 + st * 2 * kTileBytes;
            if (FP8) sm.scale[st][warp == 0 ? 0 : 1] = sc;
            mbar_arrive_expect_tx(&full[st], kTileBytes);
#pragma unroll
            for (int half = 0; half < (FP8 ? 1 : 2); ++half) {
              if (LOGITS) tma_load_3d_policy(dst + half * 16384, map, &full[st], half * 64, head, r, policy);
              else tma_load_3d(dst + half * 16384, map, &full[st], half * 64, head, r);
            }
            ++issued;
          }
        }
        __syncwarp();
        stopped = __any_sync(0xFFFFFFFFu, *abort_flag) != 0;
        if (stopped) break;
        ++fills;
      }
    }
    if (bad) atomicOr(&sm.err, kFlagBadIndex);
    if (lane == 0)  // no copy may land after this CTA has left (all have, but after a wait that gave up)
      for (uint32_t f = issued > C::kStages ? issued - C::kStages : 0; f < issued; ++f)
        mbar_wait(&full[f % C::kStages], (f / C::kStages) & 1, nullptr);
  } else if (warp == 2) {
    // ------------------------------------------------------------ Q of each segment, once the one before has its last S
    if (lane == 0) {
      uint32_t segs = 0;
      while (walk.next(sg)) {
        if (segs > 0 && !mbar_wait(&sm.q_empty, (segs - 1) & 1, abort_flag)) {
          gave_up();
          break;
        }
        mbar_arrive_expect_tx(&sm.q_full, G * 256);
        tma_load_3d(q_buf, &maps.q, &sm.q_full, 0, head * G, sg.seq);
        tma_load_3d(q_buf + 16384, &maps.q, &sm.q_full, 64, head * G, sg.seq);
        ++segs;
      }
      if (segs > 0) mbar_wait(&sm.q_full, (segs - 1) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16(128, C::kKeys, false), idesc_o = FP8 ? idesc_f16(128, kHeadDim, true) : idesc_bf16(128, kHeadDim, true);
      uint32_t fs = 0, fp = 0;          // units whose S, whose P V has been issued
      uint32_t segs = 0, pv_segs = 0;   // segments begun on either side
      uint32_t place = 0;               // a byte per warpgroup: its unit's place in the segment (0, 1, 2 and behind)
      int i = 0;                        // the next unit's place
      bool ok = true, more = walk.next(sg);
      // S of unit fs
      auto issue_s = [&] {
        const int st = fs % C::kStages, b = fs & 1;
        if (i == 0 && !mbar_wait(&sm.q_full, segs & 1, abort_flag)) return false;
        // S's columns are free once P V of unit fs - 2 has read its P
        if (fs >= 2 && !mbar_wait(&sm.pv_done[(fs - 2) % C::kStages], ((fs - 2) / C::kStages) & 1, abort_flag)) return false;
        if (!mbar_wait(FP8 ? &sm.k_ready[st] : &sm.k_full[st], (fs / C::kStages) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t qa = smem_u32(q_buf), ka = smem_u32(ring + st * 2 * C::kHalf);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          umma_bf16(tmem + C::kColS + b * 128, sdesc_sw128(qa + off, 16, 1024), sdesc_sw128(ka + off, 16, 1024), idesc_s,
                    kk ? 1u : 0u);
        }
        umma_commit(&sm.s_done[fs % 6]);
        place = (place & ~(0xFFu << (8 * b))) | (static_cast<uint32_t>(i < 2 ? i : 2) << (8 * b));
        ++fs;
        if (++i == sg.count) {
          umma_commit(&sm.q_empty);
          ++segs;
          i = 0;
          more = walk.next(sg);
        }
        return true;
      };
      // O (+)= P V of unit fp, in its warpgroup's accumulator: a new sum for the first two units of a segment, once
      // the segment before has been read out
      auto issue_pv = [&] {
        const int st = fp % C::kStages, b = fp & 1;
        const uint32_t at = (place >> (8 * b)) & 0xFFu;
        if (at == 0) ++pv_segs;
        if (!mbar_wait(&sm.p_full[b], (fp >> 1) & 1, abort_flag) ||
            !mbar_wait(FP8 ? &sm.v_ready[st] : &sm.v_full[st], (fp / C::kStages) & 1, abort_flag) ||
            (at < 2 && pv_segs > 1 && !mbar_wait(&sm.o_free, (pv_segs - 2) & 1, abort_flag)))
          return false;
        tc_fence_after();
        const uint32_t va = smem_u32(ring + st * 2 * C::kHalf + C::kHalf);
        const uint32_t pc = tmem + C::kColS + b * 128, oc = tmem + C::kColO + b * 128;
        // P of keys 32 c .. + 31: the values in columns 32 c .. + 15, the rests in 32 c + 16 .. + 31
#pragma unroll
        for (int part = 0; part < (FP8 ? 1 : 2); ++part)  // fp8: one value
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(oc, pc + (kk >> 1) * 32 + (kk & 1) * 8 + part * 16, sdesc_sw128(va + kk * 2048, 16384, 1024),
                         idesc_o, (at < 2 && part == 0 && kk == 0) ? 0u : 1u);
        umma_commit(&sm.pv_done[st]);
        ++fp;
        return true;
      };
      while (ok && more) {
        // S one unit ahead of P V
        ok = issue_s() && (fs < 2 || issue_pv());
      }
      if (ok && fp < fs) ok = issue_pv();
      if (!ok) gave_up();
      umma_commit(&sm.mma_done);
      mbar_wait(&sm.mma_done, 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    const int b = (warp >> 2) - 1;         // warpgroup: units of this parity
    const int r = (warp & 3) * 32 + lane;  // TMEM lane = head of the group
    const bool busy = (warp & 3) * 32 < G;  // a warp whose rows are all past the group only keeps the barriers going
    const uint32_t la = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = la + C::kColS + b * 128, o_col = la + C::kColO + b * 128;
    uint32_t f = 0, segs = 0;
    bool ok = true;
    int4 crossing = make_int4(-1, 0, 0, 0);  // the sequence that begins in this run and goes on
    write_empty(p, g, head, threadIdx.x - 128, 256);
    auto warp_arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // fp8: this warpgroup widens its units' codes; stages (of codes and of values) are its own.  K of its next unit, at
    // once after a unit (whose S is done): a segment's output waits for P V, which is issued after the next S.  V,
    // once P V of the unit before is done.
    const uint32_t units = static_cast<uint32_t>(run.hi - run.lo);
    float sk = 1.0f;
    auto widen_k = [&](uint32_t n) {  // of unit n
      if (n >= units) return true;
      if (!mbar_wait_warp(&sm.k_full[b], n >> 1 & 1, abort_flag)) return false;
      sk = sm.scale[b][0];
      widen<true>(codes + b * 2 * C::kCodes, ring + b * 2 * C::kHalf, r, C::kKeys);
      fence_proxy_async_smem();
      warp_arrive(&sm.k_empty[b]);
      warp_arrive(&sm.k_ready[b]);
      return true;
    };
    if (FP8) ok = widen_k(b);
    for (; ok && walk.next(sg); ++segs) {
      float m = -INFINITY;
      float d = 0.0f;  // fp8: O is relative to 2^(m + d - 11), d whole
      float2 l2 = make_float2(0.0f, 0.0f);
      for (int i = 0; i < sg.count; ++i, ++f) {
        if (static_cast<int>(f & 1) != b) continue;
        const int valid = sg.len - (sg.off + i) * C::kKeys;
        const bool tail = valid < C::kKeys;  // uniform: the sequence's last unit
        float c = p.scale_log2, sv = 1.0f;
        if (FP8) {
          c = normal_factor(c * sk);
          if ((f >= 2 && !mbar_wait_warp(&sm.pv_done[b], (f >> 1 & 1) ^ 1, abort_flag)) ||
              !mbar_wait_warp(&sm.v_full[b], f >> 1 & 1, abort_flag)) {
            ok = false;
            break;
          }
          sv = sm.scale[b][1];
          widen<false>(codes + b * 2 * C::kCodes + C::kCodes, ring + b * 2 * C::kHalf + C::kHalf, r, valid);
          fence_proxy_async_smem();
          warp_arrive(&sm.v_empty[b]);
          warp_arrive(&sm.v_ready[b]);
        }
        if (!mbar_wait_warp(&sm.s_done[f % 6], (f / 6) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!FP8 && tail) {
          // Its V rows past the end hold anything, and 0 * NaN is NaN: zero them.  (The barrier is past the stage's
          // earlier fills: S of this unit came after P V of the unit before the last.)
          const int st = f % C::kStages;
          if (!mbar_wait_warp(&sm.v_full[st], (f / C::kStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* v = ring + st * 2 * C::kHalf + C::kHalf;
          for (int j = valid * 8 + r; j < C::kKeys * 8; j += 128) {  // 16-byte pieces of the rows' two halves
            reinterpret_cast<uint4*>(v)[j] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(v + 16384)[j] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (busy) {
          // the row's maximum over the unit, then its weights, 32 keys at a time
          uint32_t va[32], vb[32];
          float x = -INFINITY;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float xa, xb;
            tmem_ld_max_32cols(s_col + 64 * q, va, xa);
            tmem_ld_max_32cols(s_col + 64 * q + 32, vb, xb);
            tmem_ld_wait_regs_max(va, xa);
            tmem_regs_written(vb, xb);
            if (tail) {
              xa = xb = -INFINITY;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                if (64 * q + j < valid) xa = fmaxf(xa, __uint_as_float(va[j]));
                if (64 * q + 32 + j < valid) xb = fmaxf(xb, __uint_as_float(vb[j]));
              }
            }
            x = fmax3(x, xa, xb);
          }
          x *= c;
          float to_fp16 = 1.0f;
          // Per lane: the warpgroup's first unit of the segment, or so far no key counts (O and l are 0).
          const bool fresh = i < 2 || m == -INFINITY;
          const float top = ceilf(x);
          if (fresh) m = top;
          const bool rise = x - m > 8.0f;  // not where it is fresh
          const float up = rise ? top - m : 0.0f, k = exp2_approx(-up);
          if (rise) m = top;
          const bool big = fabsf(m) >= kRoundLogits;
          if (FP8) {
            // fp8: the weights times the page's scale are one fp16 value, O relative to an exponent of its own, d above
            // m, which rises when a unit's largest would pass it by more than 2^4: at most 2^15, with fp16's full 11
            // bits down to 2^-25 of the largest, whatever the pages' scales.
            const float lv = log2f(sv), d_new = fminf(fmaxf(ceilf(lv), -160.0f), 160.0f);
            l2.x *= k;
            l2.y *= k;
            d = fresh ? d_new : d - up;
            const float over = x - m + lv - d;
            const bool need = !fresh && over > 4.0f;
            if (__any_sync(0xFFFFFFFFu, need || big)) {  // uniform, as the votes and the rescaling have to be
              if (__any_sync(0xFFFFFFFFu, need)) {  // not a segment's first units; O is complete: its P V has been waited for
                tc_fence_after();
                const float raise = need ? ceilf(over) : 0.0f;
                scale_row(o_col, exp2_approx(-raise));
                d = raise > 150.0f ? d_new : d + raise;  // O is 0 then, and a sum of numbers of that size not exact
              }
              if (__any_sync(0xFFFFFFFFu, big)) scale_row(s_col, big ? c : 1.0f);
            }
            const float part = truncf(0.5f * (11.0f - d));  // in two steps: the exponent may pass fp32's
            to_fp16 = sv * exp2_approx(part) * exp2_approx(11.0f - d - part);
          } else if (__any_sync(0xFFFFFFFFu, rise || big)) {
            if (__any_sync(0xFFFFFFFFu, rise)) {  // not a segment's first units
              // O is complete once P V of this warpgroup's unit before is done
              if (!mbar_wait_warp(&sm.pv_done[(f - 2) % C::kStages], ((f - 2) / C::kStages) & 1, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
              scale_row(o_col, k);
              l2.x *= k;
              l2.y *= k;
            }
            if (__any_sync(0xFFFFFFFFu, big)) scale_row(s_col, big ? c : 1.0f);
          }
          if (big) c = 1.0f;  // S holds the row's logits
          float* logits = nullptr;
          if (LOGITS && r < G)
            logits = p.logits + (((sg.unit + i) * p.hkv + head) * static_cast<long long>(G) + r) * C::kKeys;
          const float off = m == -INFINITY ? 0.0f : -m;  // -inf - -inf is NaN
          const float2 c2 = make_float2(c, c), nm = make_float2(off, off), s2 = make_float2(to_fp16, to_fp16);
          auto weights = [&](uint32_t (&v)[32], int q) {
            if (tail) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (32 * q + j >= valid) v[j] = 0xFF800000u;
            }
            if (LOGITS && logits) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(__uint_as_float(v[j + k]) * c);
                st_global_32b(logits + 32 * q + j, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
              }
            }
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              uint32_t hi[8], lo[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 z = ffma2(make_float2(__uint_as_float(v[h + 2 * j]), __uint_as_float(v[h + 2 * j + 1])), c2, nm);
                const float2 w = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                l2 = fadd2(l2, w);
                if (FP8) {
                  const float2 v16 = fmul2(w, s2);
                  hi[j] = pack_f16(v16.x, v16.y);
                } else {
                  split_bf16(w.x, w.y, hi[j], lo[j]);
                }
              }
              tmem_st_8cols(s_col + 32 * q + h / 2, hi);
              if (!FP8) tmem_st_8cols(s_col + 32 * q + 16 + h / 2, lo);
            }
          };
          tmem_ld_32cols(s_col, va);
          tmem_ld_wait_regs(va);
          tmem_ld_32cols(s_col + 32, vb);
          weights(va, 0);
          tmem_ld_wait_regs(vb);
          tmem_ld_32cols(s_col + 64, va);
          weights(vb, 1);
          tmem_ld_wait_regs(va);
          tmem_ld_32cols(s_col + 96, vb);
          weights(va, 2);
          tmem_ld_wait_regs(vb);
          weights(vb, 3);
          tmem_st_wait();
        } else {
          m = 0.0f;  // O of these rows exists but is nobody's
        }
        tc_fence_before();
        warp_arrive(&sm.p_full[b]);
        if (FP8 && !widen_k(f + 2)) {
          ok = false;
          break;
        }
      }
      if (!ok) break;

      // ---- the segment's output: this warpgroup's last P V done, (m, l) exchanged; each takes half of the dims
      const uint32_t last = f - 1;                                   // the segment's last unit
      const bool some = sg.count > 1 || static_cast<int>(last & 1) == b;
      if (some) {
        const uint32_t own = static_cast<int>(last & 1) == b ? last : last - 1;
        if (!mbar_wait_warp(&sm.pv_done[own % C::kStages], (own / C::kStages) & 1, abort_flag)) {
          ok = false;
          break;
        }
      }
      float l = l2.x + l2.y;
      if (segs > 0 && !mbar_wait_warp(&sm.o_free, (segs - 1) & 1, abort_flag)) {  // the segment before's are read
        ok = false;
        break;
      }
      sm.ml[b][r] = make_float2(m, l);
      if (FP8) sm.d[b][r] = static_cast<short>(d);
      warp_arrive(&sm.ml_full);
      if (!mbar_wait_warp(&sm.ml_full, segs & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float2 other = sm.ml[b ^ 1][r];
      const float top = fmaxf(m, other.x);
      const float k_own = exp2_diff(m, top), k_other = exp2_diff(other.x, top);
      l = b == 0 ? fmaf(l, k_own, other.y * k_other) : fmaf(other.y, k_other, l * k_own);  // the same in both warpgroups
      // fp8: 2^(m + d - 11 - top), the small numbers by themselves
      auto from_d = [&](float m, float d) { return m == -INFINITY ? 0.0f : exp2_approx((m - top) + (d - 11.0f)); };
      const float e_own = FP8 ? from_d(m, d) : k_own;
      const float e_other = FP8 ? from_d(other.x, sm.d[b ^ 1][r]) : k_other;
      m = top;
      const bool whole = sg.first && sg.last;
      const long long out_row0 = (static_cast<long long>(sg.seq) * p.hkv + head) * G;
      const long long part_row0 = (static_cast<long long>(blockIdx.x) * 2 + (sg.first ? 1 : 0)) * G;
      if (busy) {
        // A warpgroup that had no unit of the segment: its O holds an older one.  Uniform, from the segment alone: the
        // rows of O that a lane sums below are other lanes'.  (A row of which no key counts has the factor 0.)
        const bool none_own = !some, none_other = !(sg.count > 1 || static_cast<int>(last & 1) != b);
        const float inv = whole ? inverse(l) : 1.0f;
        const float f_own = e_own * inv, f_other = e_other * inv;
        const uint32_t other_col = la + C::kColO + (b ^ 1) * 128;
        // Four lanes share a row: each loads two of every eight dims, and they trade until each has eight in a row, so
        // that a store writes 128 (or 64) bytes of 8 rows and not 32 (16) of 32 (34.1 -> 33.1 us at 128 heads, 200,000
        // keys of 8 sequences; 51.8 -> 49.6 us at 304 x 1,280).
        const int t4 = lane & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int dim = b * 64 + (q >> 1) * 32, part = (q & 1) * 16;  // 32 dims of 16 of the rows
          uint32_t v[16], w[16];
          tmem_ld_16rows_32cols(o_col + dim + (part << 16), v);
          tmem_ld_16rows_32cols(other_col + dim + (part << 16), w);
          tmem_ld_wait_regs16(v);
          tmem_ld_wait_regs16(w);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int from = part + e * 8 + (lane >> 2);
            const float fo = __shfl_sync(0xFFFFFFFFu, f_own, from), fx = __shfl_sync(0xFFFFFFFFu, f_other, from);
            const int row = (warp & 3) * 32 + from;
            float o[8];  // dims 8 i + 2 t4, + 1
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int at = (j >> 1) * 4 + e * 2 + (j & 1);
              o[j] = (none_own ? 0.0f : __uint_as_float(v[at]) * fo) + (none_other ? 0.0f : __uint_as_float(w[at]) * fx);
            }
            if (whole) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) h[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
              quad_transpose(h, t4);
              if (row < G)  // o is 16-byte aligned
                *reinterpret_cast<uint4*>(p.o + (out_row0 + row) * kHeadDim + dim + 8 * t4) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
              uint32_t x[4], y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[i] = __float_as_uint(o[2 * i]);
                y[i] = __float_as_uint(o[2 * i + 1]);
              }
              quad_transpose(x, t4);
              quad_transpose(y, t4);
              if (row < G)
                st_global_32b(p.part_o + (part_row0 + row) * kHeadDim + dim + 8 * t4, make_uint4(x[0], y[0], x[1], y[1]),
                              make_uint4(x[2], y[2], x[3], y[3]));
            }
          }
        }
      }
      tc_fence_before();
      warp_arrive(&sm.o_free);
      if (b == 0 && r < G) {
        if (whole) {
          p.lse[out_row0 + r] = (m + log2f(l)) * kLn2;
          if (LOGITS) p.norm[out_row0 + r] = row_norm(m, l);
        } else {
          p.part_ml[part_row0 + r] = make_float2(m, l);
        }
      }
      if (sg.first && !sg.last) {
        const long long end = sg.unit + units_of(sg.len, p.unit_shift) - 1;
        crossing = make_int4(sg.seq, g, static_cast<int>(((end + 1) * run.runs - 1) / run.total), 0);
      }
      if (p.by_seq && sg.first && b == 0 && r == 0)
        p.meta[sg.seq * p.hkv + head] = sg.last ? make_int4(-1, 0, 0, 0) : crossing;
    }
    if (!ok && lane == 0) gave_up();
    if (!p.by_seq && b == 0 && r == 0) p.meta[blockIdx.x] = crossing;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) p.flags[blockIdx.x] = sm.err;
}

// ---------------------------------------------------------------- join
// Merges the partials of a sequence that crosses runs.  CTA (entry of meta, KV
// head; 8 / wpr head rows), wpr warps to a row, eight partials in flight each:
// a sequence alone has as many partials as there are runs (and few rows to
// spread them over), the sequences of a large batch have two or three.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) dense_join_kernel(DenseDecodeParams p, int wpr) {
  __shared__ float4 acc[8][32];
  __shared__ float2 ml[8];
  __shared__ uint32_t all_flags;
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 meta = p.meta[blockIdx.x];
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) all_flags = 0;
    __syncthreads();
    uint32_t f = 0;
    for (int i = threadIdx.x; i < p.groups * p.hkv; i += kJoinThreads) f |= p.flags[i];
    if (f) atomicOr(&all_flags, f);
    __syncthreads();
    if (threadIdx.x == 0) p.hdr->status = all_flags;
  }
  if (meta.x < 0) return;
  // A CTA of the split that gave up a wait leaves the entries of its later sequences as the workspace held them: whatever
  // they say, nothing outside the buffers is touched (the call is flagged).
  if (meta.x >= p.num_seqs || meta.y < 0 || meta.y > meta.z || meta.z >= p.groups) return;
  const int head = blockIdx.x % p.hkv, G = p.group;
  const int row = blockIdx.y * (8 / wpr) + warp / wpr, sub = warp % wpr;
  const int n = meta.z - meta.y + 1;
  float m = -INFINITY, l = 0.0f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < G) {
    // run meta.y + i's partial: the first run ends it in slot 1, the others begin with it in slot 0
    const long long first = (static_cast<long long>(meta.y) * p.hkv + head) * 2;
    for (int i0 = sub; i0 < n; i0 += 8 * wpr) {
      float2 x[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * wpr;
        x[u] = make_float2(-INFINITY, 0.0f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
          const long long at = (first + static_cast<long long>(i) * p.hkv * 2 + (i == 0 ? 1 : 0)) * G + row;
          x[u] = p.part_ml[at];
          v[u] = *reinterpret_cast<const float4*>(p.part_o + at * kHeadDim + lane * 4);
        }
      }
      float nm = m;
#pragma unroll
      for (int u = 0; u < 8; ++u) nm = fmaxf(nm, x[u].x);
      const float k = exp2_diff(m, nm);
      a.x *= k; a.y *= k; a.z *= k; a.w *= k;
      l *= k;
      m = nm;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float f = exp2_diff(x[u].x, m);
        l = fmaf(x[u].y, f, l);
        a.x = fmaf(v[u].x, f, a.x);
        a.y = fmaf(v[u].y, f, a.y);
        a.z = fmaf(v[u].z, f, a.z);
        a.w = fmaf(v[u].w, f, a.w);
      }
    }
  }
  if (wpr > 1) {
    acc[warp][lane] = a;
    if (lane == 0) ml[warp] = make_float2(m, l);
    __syncthreads();
    if (sub != 0) return;
    float M = m;
    for (int w = 1; w < wpr; ++w) M = fmaxf(M, ml[warp + w].x);
    float k = exp2_diff(m, M);
    a.x *= k; a.y *= k; a.z *= k; a.w *= k;
    l *= k;
    m = M;
    for (int w = 1; w < wpr; ++w) {
      const float4 v = acc[warp + w][lane];
      k = exp2_diff(ml[warp + w].x, M);
      l = fmaf(ml[warp + w].y, k, l);
      a.x = fmaf(v.x, k, a.x);
      a.y = fmaf(v.y, k, a.y);
      a.z = fmaf(v.z, k, a.z);
      a.w = fmaf(v.w, k, a.w);
    }
  }
  if (row >= G) return;
  const float inv = inverse(l);
  const long long out = (static_cast<long long>(meta.x) * p.hkv + head) * G + row;
  *reinterpret_cast<uint2*>(p.o + out * kHeadDim + lane * 4) =
      make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
  if (lane == 0) {
    p.lse[out] = (m + log2f(l)) * kLn2;
    if (p.norm) p.norm[out] = row_norm(m, l);
  }
}

// ---------------------------------------------------------------- weights
// weight[s, g, j] += sum over the group's heads of 2^(s[h,j] - m_h) / l_h, from
// the logits that the split kernel left (mostly still in L2).  The heads are
// added in order, four keys to a thread: no atomics.
constexpr int kWeightThreads = 512;
__global__ void __launch_bounds__(kWeightThreads, 2) dense_weight_kernel(DenseDecodeParams p) {
  __shared__ RunSmem run_sm;
  __shared__ float2 norm[128];
  griddep_wait();
  if (p.hdr->status & kFlagTimeout) return;  // logits are missing
  const int head = blockIdx.x % p.hkv, g = blockIdx.x / p.hkv, G = p.group;
  Run run;
  if (!find_run(p, g, run_sm, run)) return;
  Walker walk(p, run);
  Segment sg;
  const int tile = 1 << p.unit_shift, per = tile / 4;  // keys and threads of a unit
  const int key = threadIdx.x % per * 4, first = threadIdx.x / per;
  while (walk.next(sg)) {
    __syncthreads();
    const long long row = static_cast<long long>(sg.seq) * p.hkv + head;
    if (threadIdx.x < G) norm[threadIdx.x] = p.norm[row * G + threadIdx.x];
    __syncthreads();
    float* out = p.weight + row * p.weight_stride;
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    for (int i = first; i < sg.count; i += kWeightThreads / per) {
      const int j = ((sg.off + i) << p.unit_shift) + key;
      if (j >= sg.len) continue;
      const float* s = p.logits + ((((sg.unit + i) * p.hkv + head) * G) << p.unit_shift) + key;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int h = 0; h < G; ++h) {
        const float2 n = norm[h];
        const float4 v = *reinterpret_cast<const float4*>(s + (h << p.unit_shift));
        sum.x += exp2_approx(v.x - n.x) * n.y;
        sum.y += exp2_approx(v.y - n.x) * n.y;
        sum.z += exp2_approx(v.z - n.x) * n.y;
        sum.w += exp2_approx(v.w - n.x) * n.y;
      }
      if (vec && j + 4 <= sg.len) {
        float4* at = reinterpret_cast<float4*>(out + j);
        const float4 old = *at;
        *at = make_float4(old.x + sum.x, old.y + sum.y, old.z + sum.z, old.w + sum.w);
      } else {
        out[j] += sum.x;
        if (j + 1 < sg.len) out[j + 1] += sum.y;
        if (j + 2 < sg.len) out[j + 2] += sum.z;
        if (j + 3 < sg.len) out[j + 3] += sum.w;
      }
    }
  }
}

template <bool FP8>
cudaError_t launch_split_tc(const DenseMaps& maps, const DenseDecodeParams& p, cudaStream_t stream) {
  auto* fn = p.logits ? dense_split_tc_kernel<FP8, true> : dense_split_tc_kernel<FP8, false>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kTcSmemBytes));
  if (e != cudaSuccess) return e;
  e = launch_pdl(fn, dim3(p.groups * p.hkv), dim3(TcCfg<FP8>::kThreads), kTcSmemBytes, stream, maps, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

template <int MG, bool FP8>
cudaError_t launch_split(const DenseMaps& maps, const DenseDecodeParams& p, cudaStream_t stream) {
  using C = SplitCfg<MG, FP8>;
  auto* fn = p.logits ? dense_split_kernel<MG, FP8, true> : dense_split_kernel<MG, FP8, false>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  e = launch_pdl(fn, dim3(p.groups * p.hkv), dim3(C::kThreads), C::kSmem, stream, maps, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

template <bool FP8>
cudaError_t launch_split_for(const DenseMaps& maps, const DenseDecodeParams& p, cudaStream_t stream) {
  if (p.group <= 16) return launch_split<1, FP8>(maps, p, stream);
  return launch_split<2, FP8>(maps, p, stream);
}

}  // namespace

int dense_decode_ctas_per_sm(int group) { return group <= 16 ? 2 : 1; }

bool dense_decode_tc(int group) { return group > 32; }

cudaError_t launch_dense_decode(const DenseMaps& maps, const DenseDecodeParams& p, bool fp8, cudaStream_t stream) {
  cudaError_t e = dense_decode_tc(p.group) ? (fp8 ? launch_split_tc<true>(maps, p, stream) : launch_split_tc<false>(maps, p, stream))
                  : fp8                    ? launch_split_for<true>(maps, p, stream)
                                           : launch_split_for<false>(maps, p, stream);
  if (e != cudaSuccess) return e;
  const int entries = p.by_seq ? p.num_seqs : p.groups;
  int wpr = 1;  // warps to a row: one for every four partials that a sequence has on average, up to eight
  while (wpr < 8 && p.groups / entries >= 8 * wpr) wpr *= 2;
  e = launch_pdl(dense_join_kernel, dim3(entries * p.hkv, (p.group * wpr + 7) / 8), dim3(kJoinThreads), 0, stream, p,
                 wpr);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (!p.weight) return cudaSuccess;
  e = launch_pdl(dense_weight_kernel, dim3(p.groups * p.hkv), dim3(kWeightThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaSuccess;
}

}  // namespace msa
