// prompt_attn.cu -- dense attention of many new tokens per sequence: causal prompts and prompt chunks over packed or
// paged keys, and trees of drafted tokens over a paged cache, bf16 or E4M3 pages.
//
// For query head h of group g and new token t of a sequence (the last q_len of its kv_len positions)
//   s[t,h,j] = c q_t,h . k_j,g     lse = ln sum_j e^s     o = sum_j e^(s - lse) v_j,g
// over the keys that t sees: j <= kv_len - q_len + t, or every key before the new ones and those of the new ones whose
// bit is set in t's row of a mask.
//
// A token's G heads share every key, so a tile's 128 rows are floor(128 / G) tokens with their G heads each: any group
// size runs the same kernel, and prompts of few tokens still fill the rows of an MMA.  An item is two such tiles of a
// sequence and KV head.  Per block of 128 keys and tile
//   S = Q K^T   128 x 128 x 128, both operands in shared memory, S in TMEM
//   P = 2^(S c - m)   a row per thread, bf16, written over S in TMEM
//   O += P V    128 x 128 x 128, P from TMEM, O in TMEM
// A warpgroup per tile computes P while the MMAs of the other tile run.  m is a row's reference: the maximum of its first
// block, replaced (and O and l rescaled) only when a block's maximum passes it by more than 2^8.  P is rounded to bf16
// (2^-8 of each weight, as V's type asks: the MMA multiplies two operands of one type); l and lse sum the unrounded
// weights, everything else is fp32.
//
// An item of one tile (a tree of few drafts, the end of a prompt) would leave one warpgroup idle: its blocks go to the
// two warpgroups in turn, each with its own m, l and O, merged at the end.
//
// Items differ in cost.  Where there are enough of them the CTAs take them whole, largest first; where the longest alone
// would hold up the call (few rows over a long cache) all blocks are cut into equal runs, one per CTA, and an item that
// crosses runs leaves (O, m, l) per run, which a join kernel merges.  A plan kernel decides from the lengths.
#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;
// A call is cut into runs when its longest item has this many blocks more than an even share: what a partial's way
// through memory and the join cost.
constexpr int kRunsSlack = 6;

// Exclusive scan over the CTA (kPlanThreads threads); `sh` holds 32 values.
__device__ long long plan_scan(long long v, long long* sh, long long* total) {
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

// Key blocks of the item of a sequence that begins at its token t0.
__device__ __forceinline__ int item_blocks(const PromptParams& p, const SeqInfo& si, int t0) {
  if (p.visible) return (si.kv_len + kBlock - 1) / kBlock;
  const int end = min(si.q_len, t0 + 2 * p.tile_tokens);
  return (si.kv_len - si.q_len + end + kBlock - 1) / kBlock;
}

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(PromptParams p) {
  __shared__ long long sh[32];
  __shared__ int bins[kPlanBins];
  __shared__ int s_bad, s_most;
  griddep_wait();  // the kernel before may still read this workspace
  for (int w = threadIdx.x; w < static_cast<int>(sizeof(WsHeader) / 4); w += kPlanThreads)
    reinterpret_cast<uint32_t*>(p.hdr)[w] = 0u;
  if (threadIdx.x == 0) {
    s_bad = 0;
    s_most = 0;
  }
  for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) bins[i] = 0;
  __syncthreads();
  const int per_item = 2 * p.tile_tokens;
  long long n_items = 0;
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + threadIdx.x;
    int n = 0;
    if (s < p.num_seqs) {
      const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], k0 = p.cu_k[s], k1 = p.cu_k[s + 1];
      const long long ql = static_cast<long long>(q1) - q0, kl = static_cast<long long>(k1) - k0;
      bool bad = ql < 0 || kl < ql || ql > p.max_q || kl > p.max_k || q0 < 0 || k0 < 0 || q1 > p.total_q || k1 > p.total_k;
      if (s == 0 && (q0 != 0 || k0 != 0)) bad = true;
      if (s == p.num_seqs - 1 && (q1 != p.total_q || k1 != p.total_k)) bad = true;
      if (bad) {
        s_bad = 1;
      } else {
        n = static_cast<int>((ql + per_item - 1) / per_item);
      }
      p.seq[s] = SeqInfo{q0, static_cast<int>(ql), k0, static_cast<int>(kl)};
    }
    long long total;
    const long long before = plan_scan(n, sh, &total);
    if (s < p.num_seqs) p.item_base[s] = static_cast<int>(n_items + before);
    n_items += total;
  }
  PromptPlan* plan = p.plan;
  if (s_bad || n_items > p.max_items) {  // the second cannot be when the first is not: a bound for the buffers
    if (threadIdx.x == 0) {
      atomicOr(&p.hdr->status, kFlagBadSeqlens);
      plan->n_items = 0;
      plan->runs = 0;
      plan->total = 0;
    }
    return;
  }
  const int items = static_cast<int>(n_items);
  // costs: their sum, the largest, and how many items there are of each size
  int shift = 0;
  while ((p.max_nb >> shift) >= kPlanBins) ++shift;
  long long sum = 0;
  int most = 0;
  for (int j = threadIdx.x; j < items; j += kPlanThreads) {
    const int s = find_seq(p.item_base, p.num_seqs, j);
    const int n = item_blocks(p, p.seq[s], (j - p.item_base[s]) * per_item);
    sum += n;
    most = max(most, n);
    atomicAdd(&bins[n >> shift], 1);
  }
  atomicMax(&s_most, most);
  long long total;
  plan_scan(sum, sh, &total);  // synchronises
  total *= p.hkv;
  most = s_most;
  const bool split = p.part_o != nullptr && most > total / p.ctas + kRunsSlack;
  if (threadIdx.x == 0) {
    plan->n_items = items;
    plan->runs = split ? static_cast<int>(min(total, static_cast<long long>(p.ctas))) : 0;
    plan->total = total;
  }
  if (split) {
    // the items in order, with the blocks before each (of one KV head)
    long long carry = 0;
    for (int base = 0; base < items; base += kPlanThreads) {
      const int j = base + threadIdx.x;
      int n = 0;
      if (j < items) {
        const int s = find_seq(p.item_base, p.num_seqs, j), t0 = (j - p.item_base[s]) * per_item;
        n = item_blocks(p, p.seq[s], t0);
        p.items[j] = make_int2(s, t0);
      }
      long long t;
      const long long before = plan_scan(n, sh, &t);
      if (j < items) p.block_base[j] = static_cast<int>(carry + before);  // total < ctas * max_nb: fits
      carry += t;
    }
    return;
  }
  // the items by size, largest first (those of a size in any order: each is computed by itself)
  {
    const int c = kPlanBins - 1 - threadIdx.x;
    static_assert(kPlanBins == kPlanThreads, "a bin per thread");
    const int h = bins[c];
    long long t;
    const long long before = plan_scan(h, sh, &t);
    bins[c] = static_cast<int>(before);
  }
  __syncthreads();
  for (int j = threadIdx.x; j < items; j += kPlanThreads) {
    const int s = find_seq(p.item_base, p.num_seqs, j), t0 = (j - p.item_base[s]) * per_item;
    p.items[atomicAdd(&bins[item_blocks(p, p.seq[s], t0) >> shift], 1)] = make_int2(s, t0);
  }
}

// ---------------------------------------------------------------- a CTA's work
// A part of an item: blocks [block, block + count) of its keys, for one KV head.
struct Part {
  int seq, t0, head, block, count;
  int q_start, q_len, k_start, past;
  bool first, last;  // begins / ends the item's blocks
  bool one;          // one tile of rows: its blocks go to the warpgroups in turn
};

// The item (of `items`) that holds unit u of a call that is cut into runs.
__device__ __forceinline__ int item_of(const PromptParams& p, int items, long long u) {
  int lo = 0, hi = items - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(p.block_base[mid]) * p.hkv <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Every warp walks the same parts.
struct PartWalker {
  const PromptParams& p;
  int items, runs, item, round;
  long long at, hi;
  __device__ explicit PartWalker(const PromptParams& params) : p(params) {
    items = p.plan->n_items;
    runs = p.plan->runs;
    round = 0;
    item = 0;
    at = hi = 0;
    if (runs > 0 && static_cast<int>(blockIdx.x) < runs) {
      const long long total = p.plan->total;
      at = total * blockIdx.x / runs;
      hi = total * (blockIdx.x + 1) / runs;
      item = item_of(p, items, at);
    }
  }
  __device__ bool next(Part& g) {
    int j, blk = 0;
    if (runs > 0) {
      if (at >= hi) return false;
      j = item;
    } else {
      // largest first, there and back over the CTAs: what one has more in a round it has less in the next
      const long long n = static_cast<long long>(items) * p.hkv;
      const long long base = static_cast<long long>(round) * gridDim.x;
      const long long i = base + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ++round;
      if (i >= n) return false;  // in a last round that has only the other end, or behind it
      j = static_cast<int>(i / p.hkv);
      g.head = static_cast<int>(i - static_cast<long long>(j) * p.hkv);
    }
    const int2 it = p.items[j];
    const SeqInfo si = p.seq[it.x];
    const int n = item_blocks(p, si, it.y);
    g.seq = it.x;
    g.t0 = it.y;
    g.q_start = si.q_start;
    g.q_len = si.q_len;
    g.k_start = si.k_start;
    g.past = si.kv_len - si.q_len;
    g.one = si.q_len - it.y <= p.tile_tokens;
    if (runs > 0) {
      const long long off = at - static_cast<long long>(p.block_base[j]) * p.hkv;
      g.head = static_cast<int>(off / n);
      blk = static_cast<int>(off - static_cast<long long>(g.head) * n);
      g.count = static_cast<int>(min(static_cast<long long>(n - blk), hi - at));
      at += g.count;
      if (blk + g.count == n && g.head == p.hkv - 1) ++item;
    } else {
      g.count = n;
    }
    g.block = blk;
    g.first = blk == 0;
    g.last = blk + g.count == n;
    return true;
  }
};

// ---------------------------------------------------------------- attention kernel
// Warps 0..3 and 4..7: softmax and output of a tile each; 8 and 10: the MMAs of each; 9: loads; fp8: 12..15 widen codes.
template <bool FP8>
struct PromptCfg {
  static constexpr int kThreads = FP8 ? 512 : 384;
  // a warpgroup's registers per thread; the launch has 65,536 for all
  static constexpr int kSoftmaxRegs = FP8 ? 184 : 208, kOtherRegs = FP8 ? 72 : 88;
  static constexpr int kStages = FP8 ? 3 : 5;      // tiles of 128 keys as the MMAs read them, K and V by turns
  static constexpr int kCodeStages = FP8 ? 4 : 0;  // tiles as they land
  static_assert(!FP8 || kCodeStages == 4, "as the widening warps count them");
  static constexpr int kTile = 32768, kCodes = 16384;
  static constexpr uint32_t kColS = 0, kColO = 256;
};
struct PromptSmem {
  uint64_t full[5], empty[5];            // a stage holds a tile / its MMAs are done
  uint64_t code_full[4], code_empty[4];  // fp8
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_full[2], turn[2];  // by warpgroup
  uint64_t ml_full, o_free, mma_done;
  float2 ml[2][128];
  float scale[8];       // fp8: scales of the last tiles (no more than 3 behind the one that a warpgroup is at)
  float code_scale[4];  // and a code stage's
  uint32_t tmem_base;
  int abort_flag;
  uint32_t err;
};
constexpr size_t kPromptSmemBytes = 7 * 32768 + sizeof(PromptSmem);
static_assert(kPromptSmemBytes <= 227 * 1024, "one CTA's shared memory");

__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// True in one lane of the (converged) warp, the same one each time: MMAs and their commits come from one thread.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Bits of the keys j0 .. j0 + 31 that a new token sees: every key below `past`, and of the `n` new ones behind it those
// whose bit is set in `mask` (`words` words; what is set past n does not count).
__device__ __forceinline__ uint32_t tree_bits(const int32_t* mask, int words, int past, int n, int j0) {
  const int d = j0 - past;  // the first one's place among the new tokens
  if (d <= -32) return 0xFFFFFFFFu;
  if (d >= n) return 0u;
  auto word = [&](int w) { return w < words ? static_cast<uint32_t>(mask[w]) : 0u; };
  uint32_t bits;
  int from = d;  // new tokens from .. from + 31 were looked at, those below 0 are cached keys
  if (d < 0) {
    bits = (word(0) << -d) | ((1u << -d) - 1u);
  } else {
    const int w = d >> 5, sh = d & 31;
    bits = __funnelshift_r(word(w), word(w + 1), sh);
  }
  const int left = n - from;  // columns that are keys at all
  return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

template <bool FP8>
__global__ void __launch_bounds__(PromptCfg<FP8>::kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptMaps maps, PromptParams p) {
  using C = PromptCfg<FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const q_buf = smem;             // two tiles, each two 64-dim halves of 128 rows
  uint8_t* const ring = smem + 2 * 32768;  // stages, as the queries' tiles
  uint8_t* const codes = ring + C::kStages * C::kTile;
  PromptSmem& sm = *reinterpret_cast<PromptSmem*>(smem + 7 * 32768);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, T = p.tile_tokens;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sm.full[i], FP8 ? 4 : 1);
      mbar_init(&sm.empty[i], 2);
    }
    for (int i = 0; i < C::kCodeStages; ++i) {
      mbar_init(&sm.code_full[i], 1);
      mbar_init(&sm.code_empty[i], 4);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.turn[i], 1);
    }
    mbar_init(&sm.ml_full, 8);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.mma_done, 2);
    mbar_arrive(&sm.turn[0]);
    sm.abort_flag = 0;
    sm.err = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  // query rows that no load writes (the group does not divide 128, a second tile that no part had) are zero
  for (int i = threadIdx.x; i < 2 * 32768 / 16; i += C::kThreads) reinterpret_cast<uint4*>(q_buf)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 8) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // set up while the kernel before it ends
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  auto gave_up = [&] {
    *abort_flag = 1;
    atomicOr(&sm.err, kFlagTimeout);
  };
  if (warp >= 8) regs_release<C::kOtherRegs>();

  PartWalker walk(p);
  Part g{};
  if (warp == 9) {
    // ------------------------------------------------------------ loads: Q of a part, its tiles of K and V by turns
    constexpr int kLanding = FP8 ? C::kCodeStages : C::kStages;
    constexpr int kBytes = FP8 ? C::kCodes : C::kTile;
    uint8_t* const to = FP8 ? codes : ring;
    uint64_t* const full = FP8 ? sm.code_full : sm.full;
    uint64_t* const empty = FP8 ? sm.code_empty : sm.empty;
    uint32_t tiles = 0, queries = 0, bad = 0;
    bool ok = true;
    auto load_q = [&] {  // lane 0
      if (queries > 0 && !mbar_wait(&sm.q_empty, (queries - 1) & 1, abort_flag)) return false;
      ++queries;
      const int n = g.one ? 1 : 2;
      mbar_arrive_expect_tx(&sm.q_full, n * T * G * 256);
      for (int b = 0; b < n; ++b)
        for (int half = 0; half < 2; ++half)
          tma_load_3d(q_buf + b * 32768 + half * 16384, &maps.q, &sm.q_full, half * 64, g.head * G,
                      g.q_start + g.t0 + b * T);
      return true;
    };
    while (ok && walk.next(g)) {
      int row = 0;
      float sk = 1.0f, sv = 1.0f;
      for (int i = 0; i < g.count; ++i) {
        if ((i & 31) == 0) {  // the next 32 blocks' rows and scales, one per lane
          const int b = g.block + i + lane;
          row = g.k_start + b * kBlock;
          if (p.block_table && i + lane < g.count) {
            const int e = p.block_table[static_cast<long long>(g.seq) * p.bt_stride + b];
            const bool there = e >= 0 && e < p.n_pages;
            if (!there) bad = 1;
            row = (there ? e : static_cast<int>(p.n_pages)) * kBlock;  // past the cache: TMA reads zeros
            if (FP8) {
              sk = there ? p.k_scale[static_cast<long long>(e) * p.hkv + g.head] : 1.0f;
              sv = there ? p.v_scale[static_cast<long long>(e) * p.hkv + g.head] : 1.0f;
            }
          }
        }
        const int r = __shfl_sync(0xFFFFFFFFu, row, i & 31);
        const float k_sc = FP8 ? __shfl_sync(0xFFFFFFFFu, sk, i & 31) : 1.0f;
        const float v_sc = FP8 ? __shfl_sync(0xFFFFFFFFu, sv, i & 31) : 1.0f;
        if (lane == 0) {
          for (int h = 0; ok && h < 2; ++h, ++tiles) {
            const int st = tiles % kLanding;
            if (tiles >= kLanding && !mbar_wait(&empty[st], (tiles / kLanding - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            if (FP8) sm.code_scale[st] = h ? v_sc : k_sc;
            mbar_arrive_expect_tx(&full[st], kBytes);
            uint8_t* const dst = to + st * kBytes;
            const CUtensorMap* map = h ? &maps.v : &maps.k;
            tma_load_3d(dst, map, &full[st], 0, g.head, r);
            if (!FP8) tma_load_3d(dst + 16384, map, &full[st], 64, g.head, r);
          }
          if (ok && i == 0) ok = load_q();  // behind the first block: it waits for the part before
          if (!ok) gave_up();
        }
        ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
        if (!ok) break;
      }
    }
    if (bad) atomicOr(&sm.err, kFlagBadIndex);
    if (lane == 0) {  // no copy may land after this CTA has left (all have, but after a wait that gave up)
      for (uint32_t f = tiles > kLanding ? tiles - kLanding : 0; f < tiles; ++f)
        mbar_wait(&full[f % kLanding], (f / kLanding) & 1, nullptr);
      if (queries > 0) mbar_wait(&sm.q_full, (queries - 1) & 1, nullptr);
    }
  } else if (warp == 8 || warp == 10) {
    // ------------------------------------------------------------ MMAs
    // A warp for the MMAs of each warpgroup.  They read shared memory at nearly its full rate, under which a look at a
    // barrier takes 160 clocks, and only one or two MMAs (of 64 clocks) wait in the tensor core's queue: one warp that
    // waits and issues leaves it idle for a third of the time.  So one warp waits for its operands while the other issues,
    // and they take turns (without turns their MMAs mix, and both warpgroups wait for both).  The turn is passed on while
    // three MMAs are still to be issued, which covers its way.
    const int b = warp == 8 ? 0 : 1;
    const uint32_t idesc_s = idesc_bf16(128, 128, false), idesc_o = idesc_bf16(128, kHeadDim, true);
    const uint64_t q_desc = sdesc_sw128(smem_u32(q_buf), 16, 1024), k_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(ring), 16384, 1024);
    const uint32_t s_col = tmem + C::kColS + b * 128, o_col = tmem + C::kColO + b * 128;
    uint32_t tiles = 0, parts = 0;  // tiles before the part's, parts before it
    uint32_t p_ph = 0, turn_ph = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      // step i: P V of the warpgroup's block i, S of its block i + 1
      const int every = g.one ? 2 : 1, first = g.one ? b : 0;          // its blocks: first, first + every, ...
      const int steps = g.one ? (g.count + 1) / 2 : g.count;           // of both warps; the second may have one block less
      const int blocks = g.one ? (g.count + 1 - b) / 2 : g.count;
      const uint64_t qa = q_desc + (g.one ? 0 : b * 2048);
      ok = mbar_wait_warp(&sm.q_full, parts & 1, abort_flag);
      for (int i = -1; ok && i < steps; ++i) {
        const bool pv = i >= 0 && i < blocks, s = i + 1 < blocks;
        const uint32_t v_tile = tiles + 2 * (first + i * every) + 1, k_tile = v_tile - 1 + 2 * every;
        const uint32_t v_st = v_tile % C::kStages, k_st = k_tile % C::kStages;
        // With three stages, K of a warpgroup's next block may land only where V of this one has been.
        const bool apart = C::kStages < 5 && g.one && pv;
        if (s && !apart) ok = mbar_wait_warp(&sm.full[k_st], (k_tile / C::kStages) & 1, abort_flag);
        if (pv) {
          ok = ok && mbar_wait_warp(&sm.full[v_st], (v_tile / C::kStages) & 1, abort_flag);
          // O of the part before has been read
          if (i == 0 && parts > 0) ok = ok && mbar_wait_warp(&sm.o_free, (parts - 1) & 1, abort_flag);
          ok = ok && mbar_wait_warp(&sm.p_full[b], p_ph, abort_flag);
          p_ph ^= 1;
        }
        ok = ok && mbar_wait_warp(&sm.turn[b], turn_ph, abort_flag);
        turn_ph ^= 1;
        if (!ok) break;
        tc_fence_after();
        const uint64_t ka = k_desc + k_st * 2048, va = v_desc + v_st * 2048;
        const uint32_t more = i > 0 ? 1u : 0u;
        auto issue_pv = [&](bool pass) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            umma_bf16_ts(o_col, s_col + kk * 8, va + kk * 128, idesc_o, kk ? 1u : more);
            if (kk == 4 && pass) mbar_arrive(&sm.turn[b ^ 1]);
          }
        };
        // S follows P V of the block before: in order on the tensor cores, so S's columns are free
        auto issue_s = [&] {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
            umma_bf16(s_col, qa + off, ka + off, idesc_s, kk ? 1u : 0u);
            if (kk == 4) mbar_arrive(&sm.turn[b ^ 1]);
          }
          umma_commit(&sm.s_full[b]);
        };
        // Every stage and the queries are given back by both warps (by the one that used it, for both, where one did).
        auto give = [&](uint64_t* bar) {
          umma_commit(bar);
          if (g.one) umma_commit(bar);
        };
        if (elect_one()) {
          if (pv) issue_pv(!s);
          if (s && !apart) issue_s();
          if (!pv && !s) mbar_arrive(&sm.turn[b ^ 1]);
          if (pv) {
            if (!s) umma_commit(&sm.o_full[b]);
            give(&sm.empty[v_st]);
          }
          if (s && !apart) give(&sm.empty[k_st]);
        }
        __syncwarp();
        if (s && apart) {
          ok = mbar_wait_warp(&sm.full[k_st], (k_tile / C::kStages) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_s();
            give(&sm.empty[k_st]);
          }
          __syncwarp();
        }
        if (i + 1 == (blocks > 0 ? blocks - 1 : 0)) {  // its last S of the part (or the first step, if it has none)
          if (elect_one()) umma_commit(&sm.q_empty);
          __syncwarp();
        }
      }
      tiles += 2 * g.count;
      ++parts;
    }
    if (!ok && lane == 0) gave_up();
    // every MMA done before the tensor memory is given back
    if (elect_one()) umma_commit(&sm.mma_done);
    __syncwarp();
    mbar_wait_warp(&sm.mma_done, 0, nullptr);
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax and output
    regs_claim<C::kSoftmaxRegs>();
    const int b = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // TMEM lane: row of the tile
    const int my_t = r / G, my_h = r - my_t * G;
    const uint32_t la = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = la + C::kColS + b * 128, o_col = la + C::kColO + b * 128;
    uint32_t tiles = 0, parts = 0, steps = 0, outs = 0, merges = 0;
    bool ok = true;
    auto warp_arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    while (ok && walk.next(g)) {
      const int t_tile = g.t0 + (g.one ? 0 : b * T);  // the tile's first token
      const int tok = t_tile + my_t;
      const bool mine = my_t < T && tok < g.q_len;
      const int sees = p.visible ? g.past : g.past + t_tile + 1;  // keys that every row of the tile sees
      const int32_t* mask = p.visible && mine ? p.visible + static_cast<long long>(g.q_start + tok) * p.mask_words : nullptr;
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      int blk = g.one ? b : 0;
      const int had = blk;
      for (; blk < g.count; blk += g.one ? 2 : 1, ++steps) {
        const int j0 = (g.block + blk) * kBlock;
        const bool edge = j0 + kBlock > sees;  // uniform
        if (!mbar_wait_warp(&sm.s_full[b], steps & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t v_tile = tiles + 2 * blk + 1, v_st = v_tile % C::kStages;
        float c = p.scale_log2, sv = 1.0f;
        if (FP8) {
          // the scales come with their tiles, K's before V's (every earlier fill of the stage is past: its P V came before S of this step)
          if (!mbar_wait_warp(&sm.full[v_st], (v_tile / C::kStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          c = normal_factor(c * sm.scale[(v_tile - 1) & 7]);
          sv = sm.scale[v_tile & 7];
        } else if (edge && j0 + kBlock > g.past + g.q_len && (g.one || b == 0)) {
          // V rows past the sequence's end hold anything, and 0 * NaN is NaN: zero them
          if (!mbar_wait_warp(&sm.full[v_st], (v_tile / C::kStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          uint4* v = reinterpret_cast<uint4*>(ring + v_st * C::kTile);
          for (int i = (g.past + g.q_len - j0) * 8 + r; i < kBlock * 8; i += 128) {
            v[i] = make_uint4(0, 0, 0, 0);
            v[1024 + i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        uint32_t v[4][32];
        float mx[4];
        auto load = [&] {
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld_max_32cols(s_col + 32 * q, v[q], mx[q]);
          tmem_ld_wait_regs_max(v[0], mx[0]);
#pragma unroll
          for (int q = 1; q < 4; ++q) tmem_regs_written(v[q], mx[q]);
          if (edge) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t bits;
              if (p.visible) {
                bits = mask ? tree_bits(mask, p.mask_words, g.past, g.q_len, j0 + 32 * q) : 0u;
              } else {
                const int n = g.past + tok + 1 - j0 - 32 * q;
                bits = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
              }
              float x = -INFINITY;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                if (!(bits >> j & 1)) v[q][j] = 0xFF800000u;
                x = fmaxf(x, __uint_as_float(v[q][j]));
              }
              mx[q] = x;
            }
          }
        };
        load();
        const float x = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c;
        const bool fresh = m == -INFINITY;  // no key counts so far: O and l are 0, or not there yet
        const bool rise = !fresh && x - m > 8.0f;
        if (__any_sync(0xFFFFFFFFu, rise)) {  // O is complete: its P V came before this S
          const float k = rise ? exp2_approx(m - x) : 1.0f;
          l2.x *= k;
          l2.y *= k;
          scale_row(o_col, k);
          load();
        }
        if (fresh || rise) m = x;
        if (__any_sync(0xFFFFFFFFu, fabsf(m) >= kRoundLogits && m != -INFINITY)) {
          // products rounded to fp32 logits before the reference is taken off: see kRoundLogits
          const float k = fabsf(m) >= kRoundLogits ? c : 1.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[q][j] = __float_as_uint(__uint_as_float(v[q][j]) * k);
          if (fabsf(m) >= kRoundLogits) c = 1.0f;
        }
        const float off = m == -INFINITY ? 0.0f : -m;  // -inf - -inf is NaN
        const float2 c2 = make_float2(c, c), nm = make_float2(off, off), s2 = make_float2(sv, sv);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 z = ffma2(make_float2(__uint_as_float(v[q][2 * j]), __uint_as_float(v[q][2 * j + 1])), c2, nm);
            float2 e = make_float2(exp2_approx(z.x), exp2_approx(z.y));
            l2 = fadd2(l2, e);
            if (FP8) e = fmul2(e, s2);
            w[j] = pack_bf16(e.x, e.y);
          }
          tmem_st_16cols(s_col + 16 * q, w);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.p_full[b]);
      }
      if (!ok) break;
      tiles += 2 * g.count;

      // ---- output
      const bool some = had < g.count;
      if (some) {
        if (!mbar_wait_warp(&sm.o_full[b], outs & 1, abort_flag)) {
          ok = false;
          break;
        }
        ++outs;
        tc_fence_after();
      }
      float l = l2.x + l2.y;
      const bool whole = g.first && g.last;
      const long long out_row = (static_cast<long long>(g.q_start) + tok) * p.hq + g.head * G + my_h;
      const long long part_row =
          (static_cast<long long>(blockIdx.x) * 2 + (g.first ? 1 : 0)) * 256 + (g.one ? 0 : b * 128) + r;
      if (g.one) {
        // both warpgroups' sums of a row, each writes half of the dims
        if (parts > 0 && !mbar_wait_warp(&sm.o_free, (parts - 1) & 1, abort_flag)) {  // the part before's are read
          ok = false;
          break;
        }
        sm.ml[b][r] = make_float2(m, l);
        warp_arrive(&sm.ml_full);
        if (!mbar_wait_warp(&sm.ml_full, merges & 1, abort_flag)) {
          ok = false;
          break;
        }
        ++merges;
        tc_fence_after();
        const float2 other = sm.ml[b ^ 1][r];
        const float top = fmaxf(m, other.x);
        const float k_own = exp2_diff(m, top), k_other = exp2_diff(other.x, top);
        l = b == 0 ? fmaf(l, k_own, other.y * k_other) : fmaf(other.y, k_other, l * k_own);  // the same in both
        m = top;
        const bool both = g.count > 1;  // else O of warpgroup 1 holds an older part's
        const float inv = whole ? inverse(l) : 1.0f;
        const float f0 = (b == 0 ? k_own : k_other) * inv, f1 = (b == 0 ? k_other : k_own) * inv;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int dim = b * 64 + q * 32;
          uint32_t x[32], y[32];
          tmem_ld_32cols(la + C::kColO + dim, x);
          tmem_ld_32cols(la + C::kColO + 128 + dim, y);
          tmem_ld_wait_regs(x);
          float unused = 0.0f;
          tmem_regs_written(y, unused);
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = (l > 0.0f || !(l == 0.0f))
                       ? (f0 == 0.0f ? 0.0f : __uint_as_float(x[j]) * f0) + (both && f1 != 0.0f ? __uint_as_float(y[j]) * f1 : 0.0f)
                       : 0.0f;
          if (mine) {
            if (whole) {
              __nv_bfloat16* to = p.o + out_row * kHeadDim + dim;
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = pack_bf16(o[j + 2 * i], o[j + 2 * i + 1]);
                *reinterpret_cast<uint4*>(to + j) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(to + j + 8) = make_uint4(h[4], h[5], h[6], h[7]);
              }
            } else {
              float* to = p.part_o + part_row * kHeadDim + dim;
#pragma unroll
              for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
          }
        }
      } else {
        const float inv = whole ? inverse(l) : 1.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t x[32];
          tmem_ld_32cols(o_col + 32 * q, x);
          tmem_ld_wait_regs(x);
          if (mine) {
            if (whole) {
              __nv_bfloat16* to = p.o + out_row * kHeadDim + 32 * q;
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  h[i] = pack_bf16(__uint_as_float(x[j + 2 * i]) * inv, __uint_as_float(x[j + 2 * i + 1]) * inv);
                *reinterpret_cast<uint4*>(to + j) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(to + j + 8) = make_uint4(h[4], h[5], h[6], h[7]);
              }
            } else {
              float* to = p.part_o + part_row * kHeadDim + 32 * q;
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<uint4*>(to + j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            }
          }
        }
      }
      if (mine && (!g.one || b == 0)) {
        if (whole) p.lse[out_row] = (m + log2f(l)) * kLn2;
        else p.part_ml[part_row] = make_float2(m, l);
      }
      tc_fence_before();
      warp_arrive(&sm.o_free);
      ++parts;
    }
    if (!ok && lane == 0) gave_up();
  } else if (FP8 && warp >= 12) {
    // ------------------------------------------------------------ codes to bf16
    const int thread = threadIdx.x - 384;
    uint32_t tile = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      for (int i = 0; i < 2 * g.count; ++i, ++tile) {
        const int cs = FP8 ? tile % 4 : 0, st = tile % C::kStages;
        if (!mbar_wait_warp(&sm.code_full[cs], (tile / 4) & 1, abort_flag) ||
            (tile >= C::kStages && !mbar_wait_warp(&sm.empty[st], (tile / C::kStages - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (thread == 0) sm.scale[tile & 7] = sm.code_scale[cs];
        // rows past the sequence's end: zeros, as 0 * NaN is NaN (V)
        const int valid = g.past + g.q_len - (g.block + (i >> 1)) * kBlock;
        widen<true>(codes + cs * C::kCodes, ring + st * C::kTile, thread, valid);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.code_empty[cs]);
          mbar_arrive(&sm.full[st]);
        }
      }
    }
    if (!ok && lane == 0) gave_up();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sm.err) atomicOr(&p.hdr->status, sm.err);
}

// ---------------------------------------------------------------- join
// Merges the partials of an item that crosses runs: CTA (x, y) the item, if any, that begins in run x and goes on; a warp
// to a row, four dims to a lane, eight partials in flight.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(PromptParams p) {
  griddep_wait();
  const int runs = p.plan->runs;
  const int run = blockIdx.x;
  if (run + 1 >= runs) return;
  const long long total = p.plan->total;
  const long long edge = total * (run + 1) / runs;  // the first unit of the next run
  const int j = item_of(p, p.plan->n_items, edge);
  const int2 it = p.items[j];
  const SeqInfo si = p.seq[it.x];
  const int n = item_blocks(p, si, it.y);
  const long long base = static_cast<long long>(p.block_base[j]) * p.hkv;
  const int head = static_cast<int>((edge - base) / n);
  const long long start = base + static_cast<long long>(head) * n;
  if (start == edge || start < total * run / runs) return;  // no item goes on here, or it began in an earlier run
  const int last = static_cast<int>(((start + n) * runs - 1) / total);
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int b = row >> 7, t = (row & 127) / p.group, h = (row & 127) - t * p.group;
  const int tok = it.y + b * p.tile_tokens + t;
  if (t >= p.tile_tokens || tok >= si.q_len) return;
  float m = -INFINITY, l = 0.0f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = run; i0 <= last; i0 += 8) {
    float2 x[8];
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u;
      x[u] = make_float2(-INFINITY, 0.0f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i <= last) {
        const long long at = (static_cast<long long>(i) * 2 + (i == run ? 1 : 0)) * 256 + row;
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
  const float inv = inverse(l);
  const long long out = (static_cast<long long>(si.q_start) + tok) * p.hq + head * p.group + h;
  *reinterpret_cast<uint2*>(p.o + out * kHeadDim + lane * 4) =
      make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
  if (lane == 0) p.lse[out] = (m + log2f(l)) * kLn2;
}

template <bool FP8>
cudaError_t launch_attn(const PromptMaps& maps, const PromptParams& p, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(prompt_attn_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kPromptSmemBytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_attn_kernel<FP8>, dim3(p.ctas), dim3(PromptCfg<FP8>::kThreads), kPromptSmemBytes, stream, maps, p);
}

}  // namespace

bool prompt_may_split(int max_nb) { return max_nb > kRunsSlack; }

cudaError_t launch_prompt_attn(const PromptMaps& maps, const PromptParams& p, bool fp8, cudaStream_t stream) {
  cudaError_t e = launch_pdl(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (p.total_q == 0) return cudaSuccess;  // the lengths have been checked; there is no row to compute
  e = fp8 ? launch_attn<true>(maps, p, stream) : launch_attn<false>(maps, p, stream);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (!p.part_o || p.ctas < 2) return cudaSuccess;
  e = launch_pdl(prompt_join_kernel, dim3(p.ctas - 1, 256 / kJoinWarps), dim3(kJoinWarps * 32), 0, stream, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace msa
