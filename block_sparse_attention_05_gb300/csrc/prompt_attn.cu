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
//   P = 2^(S c - m)   a row per thread, 16 bits, written over S in TMEM
//   O += P V    128 x 128 x 128, P from TMEM, O in TMEM
// A warpgroup per tile computes P while the MMAs of the other tile run.  m is a row's reference: the maximum of its first
// block, replaced (and O and l rescaled) only when a block's maximum passes it by more than 2^8.  P is rounded to
// bf16 (2^-8 of each weight), as V's type asks: the MMA multiplies two operands of one type, and a second product with the
// rest would take half as much time again; l and lse sum the unrounded weights, everything else is fp32.
//
// E4M3 pages: K's codes are multiplied as they are (kind::f8f6f4), by queries that are two codes each; V's are widened to fp16
// by four warps of their own, and P is fp16 (2^-11).  Widening K as well had those warps bound the kernel: 6.2 ms for a
// 20,000-token prompt of 64/4 heads, which now takes 4.2.
//
// What bounds it.  A block takes a pair of tiles 2,048 clocks of MMAs, which also read shared memory at its full rate (128 bytes
// a clock: S alone 64 KB per tile).  Measured 2,900: a warpgroup's chain of S, its way to the softmax (390), the softmax
// (1,200), P's way back (180) and P V is longer than the other's MMAs.  A 20,000-token prompt of 64/4 heads: 3.84 ms in a
// burst (1,707 TFLOP/s); back to back for seconds 4.16 (1,577, at the 1,815 MHz that the power limit leaves it), where the library's
// matrix product holds 1,748 (at 1,477 MHz, its pipe fuller).  P V begun at half of P shortens the chain and changes nothing there.
//
// What is rare (a reference that rises, logits above 2^10, V's scales far apart) is found by one vote a block: with two a 20,000-token
// prompt over E4M3 pages took 4.9 ms instead of 4.5.
//
// An item of one tile (a tree of few drafts, the end of a prompt) would leave one warpgroup idle: its blocks go to the
// two warpgroups in turn, each with its own m, l and O, merged at the end.
//
// Items differ in cost.  Where there are enough of them the CTAs take them whole, largest first; where the longest alone
// would hold up the call (few rows over a long cache) all blocks are cut into runs of equal cost, one per CTA, and an item that
// crosses runs leaves (O, m, l) per run, which a join kernel merges.  A plan kernel decides from the lengths.
#include <cuda_fp8.h>

#include <atomic>

#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 1024;
// What the CTAs' shares of a call are measured in: a block of a pair of tiles takes 1.55 us, one of a single tile (most of its
// time is the memory's) 1.2, and an item beside its blocks 4.5: its queries' way in, the first block's through the pipeline,
// the output.  E4M3 pages: 1.9, 1.0, 4.5.  With runs of equally many blocks the CTAs of 16 trees of 2 to 31 drafts end
// after 75 to 113 us.
struct PromptCosts {
  int pair, one, item, slack;
};
constexpr int kPairCost = 4;  // the largest
__device__ __forceinline__ PromptCosts costs(const PromptParams& p) {
  return p.k_scale ? PromptCosts{kPairCost, 2, 9, 20} : PromptCosts{kPairCost, 3, 12, 30};
}
// A call is cut into runs when its longest item costs `slack` more than an even share, which is about what a partial's way
// through memory and the join take (6 drafts over 1,500 E4M3 keys: 27.1 us whole, 19.7 in runs; over 880 bf16 keys 19.2 and 16.4).
// Never where no item has more than so many blocks: such calls have no join launch either (8 drafts over 760 keys: bf16 16.2 us, with
// runs and join 17.9, E4M3 18.4 and 18.9; over 640 keys 15.5 and 17.3, 18.2 and 20.4; over 890, seven blocks, 16.6 either way).
constexpr int kWholeBlocks = 6;

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

// Cost of a block of the item that begins at token t0 of q_len, and of the item.
__device__ __forceinline__ int block_cost(const PromptParams& p, int q_len, int t0) {
  return q_len - t0 <= p.tile_tokens ? costs(p).one : costs(p).pair;
}
__device__ __forceinline__ int item_cost(const PromptParams& p, const PromptItem& it) {
  return it.blocks * block_cost(p, it.q_len, it.t0) + costs(p).item;
}
// The block that lies `off` behind an item's beginning: its first one for what the item costs beside them, too.
__device__ __forceinline__ int block_at(const PromptParams& p, long long off, int cost) {
  return static_cast<int>(max(off - costs(p).item, 0LL)) / cost;
}

// One CTA plans the call.  Everything here waits for something before it, so what it makes of up to kPlanThreads sequences
// and items stays in shared memory: with the lists in global memory 16 sequences took 4.7 us.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(PromptParams p) {
  __shared__ long long sh[32];
  __shared__ SeqInfo s_seq[kPlanThreads];
  __shared__ int s_base[kPlanThreads], s_item[kPlanThreads];
  __shared__ long long s_at[kPlanThreads];
  __shared__ int bins[kPlanBins];
  __shared__ int s_bad, s_most, s_cost;
  griddep_wait();  // the kernel before may still read this workspace
  for (int w = threadIdx.x; w < static_cast<int>(sizeof(WsHeader) / 4); w += kPlanThreads)
    reinterpret_cast<uint32_t*>(p.hdr)[w] = 0u;
  if (threadIdx.x == 0) {
    s_bad = 0;
    s_most = 0;
    s_cost = costs(p).one;
  }
  for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) bins[i] = 0;
  __syncthreads();
  const int per_item = 2 * p.tile_tokens;
  const bool few = p.num_seqs <= kPlanThreads;
  SeqInfo* const seq = few ? s_seq : p.seq;
  int* const item_base = few ? s_base : p.item_base;
  long long n_items = 0;
  for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
    const int s = base + threadIdx.x;
    int n = 0;
    if (s < p.num_seqs) {
      const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], k0 = p.cu_k[s], k1 = p.cu_k[s + 1];
      const long long ql = static_cast<long long>(q1) - q0, kl = static_cast<long long>(k1) - k0;
      bool bad = ql < 0 || kl < ql || ql > p.max_q || kl > p.max_k || q0 < 0 || k0 < 0 || q1 > p.total_q || k1 > p.total_k;
      if (s == 0 && (q0 != 0 || k0 != 0)) bad = true;
      // (paged: total_k is a bound, so that a captured call can follow a cache that grows)
      if (s == p.num_seqs - 1 && (q1 != p.total_q || (!p.block_table && k1 != p.total_k))) bad = true;
      if (bad) {
        s_bad = 1;
      } else {
        n = static_cast<int>((ql + per_item - 1) / per_item);
      }
      seq[s] = SeqInfo{q0, static_cast<int>(ql), k0, static_cast<int>(kl)};
    }
    long long total;
    const long long before = plan_scan(n, sh, &total);
    if (s < p.num_seqs) item_base[s] = static_cast<int>(n_items + before);
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
  __syncthreads();  // item_base is there
  const int items = static_cast<int>(n_items);
  // costs: their sum, the largest, and how many items there are of each size
  int shift = 0;
  while ((static_cast<long long>(p.max_nb) * kPairCost + costs(p).item >> shift) >= kPlanBins) ++shift;
  long long sum = 0;
  int most = 0;
  for (int j = threadIdx.x; j < items; j += kPlanThreads) {
    const int s = find_seq(item_base, p.num_seqs, j);
    const int t0 = (j - item_base[s]) * per_item, cost = block_cost(p, seq[s].q_len, t0);
    const int n = item_blocks(p, seq[s], t0) * cost + costs(p).item;
    if (cost == kPairCost) s_cost = kPairCost;
    sum += n;
    most = max(most, n);
    atomicAdd(&bins[n >> shift], 1);
  }
  atomicMax(&s_most, most);
  long long total;
  plan_scan(sum, sh, &total);  // synchronises
  total *= p.hkv;
  most = s_most;
  const bool split = p.part_o != nullptr && most > total / p.ctas + costs(p).slack;
  // A block's cost each at least.  Where an item's own cost passes a run's share several runs are cut back to the item's beginning
  // below; all of them but the last are empty then.
  const int runs = split ? static_cast<int>(min(total / s_cost, static_cast<long long>(p.ctas))) : 0;
  if (threadIdx.x == 0) {
    plan->n_items = items;
    plan->runs = runs;
    plan->total = total;
  }
  auto item = [&](int j) {
    const int s = find_seq(item_base, p.num_seqs, j), t0 = (j - item_base[s]) * per_item;
    const SeqInfo si = seq[s];
    return PromptItem{s, t0, si.q_start, si.q_len, si.k_start, si.kv_len - si.q_len, item_blocks(p, si, t0), 0};
  };
  if (split) {
    // the items in order, with the cost of those before each (for one KV head), and the item that each run begins in
    long long carry = 0;
    for (int base = 0; base < items; base += kPlanThreads) {
      const int j = base + threadIdx.x;
      PromptItem it{};
      if (j < items) it = item(j);
      long long t;
      const long long before = carry + plan_scan(j < items ? item_cost(p, it) : 0, sh, &t);
      if (j < items) {
        it.base = before;
        p.items[j] = it;
        if (base == 0) {
          s_at[j] = before;
          s_item[j] = it.blocks << 1 | (block_cost(p, it.q_len, it.t0) == kPairCost ? 1 : 0);
        }
      }
      carry += t;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < runs) {
      const long long at = total * threadIdx.x / runs;
      const bool near = items <= kPlanThreads;
      int lo = 0, hi = items - 1;  // the last item that begins at or before it
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((near ? s_at[mid] : p.items[mid].base) * p.hkv <= at) lo = mid;
        else hi = mid - 1;
      }
      long long begin;
      int blocks, cost;
      if (near) {
        begin = s_at[lo];
        blocks = s_item[lo] >> 1;
        cost = s_item[lo] & 1 ? kPairCost : costs(p).one;
      } else {
        const PromptItem it = p.items[lo];
        begin = it.base;
        blocks = it.blocks;
        cost = block_cost(p, it.q_len, it.t0);
      }
      p.run_item[threadIdx.x] = lo;
      // back to where its block begins
      const long long off = (at - begin * p.hkv) % (blocks * cost + costs(p).item);
      const int blk = block_at(p, off, cost);
      p.run_at[threadIdx.x] = at - off + (blk > 0 ? costs(p).item + static_cast<long long>(blk) * cost : 0);
    }
    if (threadIdx.x == 0) p.run_at[runs] = total;
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
    const PromptItem it = item(j);
    p.items[atomicAdd(&bins[item_cost(p, it) >> shift], 1)] = it;
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

// Every warp walks the same parts.
template <bool FP8>
struct PartWalker {
  const PromptParams& p;
  int items, runs, item, round;
  long long at, hi;  // where the run is and ends, in units of cost
  __device__ explicit PartWalker(const PromptParams& params) : p(params) {
    // (without runs: not values, and not used)
    const int start = p.run_item[blockIdx.x];
    const long long first = p.run_at[blockIdx.x], behind = p.run_at[blockIdx.x + 1];
    items = p.plan->n_items;
    runs = p.plan->runs;
    round = 0;
    item = 0;
    at = hi = 0;
    if (static_cast<int>(blockIdx.x) < runs) {
      at = first;
      hi = behind;
      item = start;
    }
  }
  __device__ bool next(Part& g) {
    int j, blk = 0;
    if (runs > 0) {
      if (at >= hi) return false;
      j = item;
    } else {
      // largest first, there and back over the CTAs: what one has more in a round it has less in the next.  (A 32-bit division
      // for E4M3 alone: bf16 prompts are 1 % slower with it.)
      const long long n = static_cast<long long>(items) * p.hkv;
      const long long base = static_cast<long long>(round) * gridDim.x;
      const long long i = base + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      ++round;
      if (i >= n) return false;  // in a last round that has only the other end, or behind it
      j = FP8 && n >> 31 == 0 ? static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.hkv)) : static_cast<int>(i / p.hkv);
      g.head = static_cast<int>(i - static_cast<long long>(j) * p.hkv);
    }
    const PromptItem it = p.items[j];
    g.seq = it.seq;
    g.t0 = it.t0;
    g.q_start = it.q_start;
    g.q_len = it.q_len;
    g.k_start = it.k_start;
    g.past = it.past;
    g.one = it.q_len - it.t0 <= p.tile_tokens;
    if (runs > 0) {
      const int cost = block_cost(p, it.q_len, it.t0), n = item_cost(p, it);
      const long long base = it.base * p.hkv;
      g.head = static_cast<int>((at - base) / n);
      const long long begin = base + static_cast<long long>(g.head) * n;
      blk = block_at(p, at - begin, cost);
      g.count = (hi - begin >= n ? it.blocks : block_at(p, hi - begin, cost)) - blk;
      at = min(begin + n, hi);
      if (blk + g.count == it.blocks && g.head == p.hkv - 1) ++item;
    } else {
      g.count = it.blocks;
    }
    g.block = blk;
    g.first = blk == 0;
    g.last = blk + g.count == it.blocks;
    return true;
  }
};

// ---------------------------------------------------------------- attention kernel
// Warps 0..3 and 4..7: softmax and output of a tile each; 8 and 10: the MMAs of each; 9: loads; fp8: 12..15 widen codes.
template <bool FP8>
struct PromptCfg {
  static constexpr int kThreads = FP8 ? 512 : 384;
  // A warpgroup's registers per thread; their sum is the launch's.  What the compiler keeps out of the softmax loop hangs on them and
  // on the unrolling of the output: a 20,000-token prompt over E4M3 pages takes 4.25 ms as it is, 4.80 with 176 and 80.
  static constexpr int kSoftmaxRegs = FP8 ? 184 : 216, kOtherRegs = 72;
  static constexpr int kRegsNeeded = 256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs;
  // bf16: stages of tiles of 128 keys.  A part of one tile of rows has the second tile's room as one more.
  static constexpr int kStages = 5;
  static constexpr int kOutStage = kStages - 2;  // bf16: a part's output passes through this and the next one
  // fp8: stages of K's codes, of V's as they land, of V's values (the output passes through these)
  static constexpr int kK8 = 4, kV8 = 2, kV16 = 2;
  static constexpr int kTile = 32768, kCodes = 16384;
  static constexpr uint32_t kColS = 0, kColO = 256;
};
struct PromptSmem {
  uint64_t full[6], empty[6];            // a stage holds a tile / its MMAs are done
  uint64_t code_full[2], code_empty[2];  // fp8: V's codes
  uint64_t q_full, q_empty, q_ready;     // fp8: ready when they are codes
  uint64_t s_full[2], p_full[2], o_full[2], turn[2];  // by warpgroup
  uint64_t ml_full, o_free, out_free, mma_done;
  float2 ml[2][128];
  float k_scale[8], v_scale[8];  // fp8: scales of the last blocks, V's as log2 (loaded at most 5 ahead of the one that a warpgroup is at)
  int8_t q_up[2][256];  // fp8: exponents of the queries' scales, by the part's parity
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

// Waits for two barriers as mbar_wait_warp does for one.
__device__ __forceinline__ bool mbar_wait_both_warp(uint64_t* x, uint32_t x_parity, uint64_t* y, uint32_t y_parity,
                                                    volatile int* abort_flag) {
  uint64_t t0 = 0;
  bool ok = true;
  for (uint32_t n = 0;; ++n) {
    const bool xs = mbar_try_wait(x, x_parity), ys = mbar_try_wait(y, y_parity);
    if (__all_sync(0xFFFFFFFFu, xs && ys)) return true;
    if ((n & 63) == 63) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) ok = false;
      if (*abort_flag) ok = false;
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    }
  }
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

// The tiles of a part in the order in which they are loaded.  Two tiles of rows: K and V of a block by turns.  One: K of two
// blocks (one per warpgroup), then their V, so that stages come free in the order in which they are wanted.
struct Fill {
  int st;           // stage
  uint32_t parity;  // of its barrier's phase
};
template <bool FP8>
struct Tiles {
  static constexpr int STAGES = PromptCfg<false>::kStages;
  int total;     // tiles of the part
  bool one;      // one tile of rows: a stage more
  uint32_t ph;   // a bit per stage: parity of its next fill
  __device__ __forceinline__ void part(const Part& g) {
    one = g.one;
    total = 2 * g.count;
  }
  __device__ __forceinline__ int k_tile(int block) const {
    return one ? 4 * (block >> 1) + (block & 1) : 2 * block;
  }
  __device__ __forceinline__ int v_tile(int block) const {
    // the last of an odd number has no other's K before its V
    return one ? 4 * (block >> 1) + ((block | 1) < total / 2 ? 2 + (block & 1) : 1) : 2 * block + 1;
  }
  __device__ __forceinline__ int block(int tile, bool& v) const {
    if (!one) {
      v = tile & 1;
      return tile >> 1;
    }
    const int first = tile >> 2 << 1, w = tile & 3;
    const bool pair = first + 1 < total / 2;
    v = pair ? w >= 2 : w == 1;
    return first + (pair ? w & 1 : 0);
  }
  // Every part begins with stage 0.
  __device__ __forceinline__ int stage(int tile) const {
    const uint32_t t = tile;
    return one ? t % (STAGES + 1) : t % STAGES;
  }
  __device__ __forceinline__ uint32_t parity(int tile) const {
    const uint32_t t = tile;
    return (ph >> stage(tile) ^ (one ? t / (STAGES + 1) : t / STAGES)) & 1u;
  }
  __device__ __forceinline__ Fill k(int block) const { return {stage(k_tile(block)), parity(k_tile(block))}; }
  __device__ __forceinline__ Fill v(int block) const { return {stage(v_tile(block)), parity(v_tile(block))}; }
  // The last fill of the stage that a warpgroup's output passes through.
  __device__ __forceinline__ Fill out(int b) const {
    const int st = PromptCfg<false>::kOutStage + (one ? 1 : b);
    return {st, (ph >> st & 1) ^ 1};
  }
  __device__ __forceinline__ void done() {
    const int n = STAGES + (one ? 1 : 0);
    const int q = total / n, r = total - q * n;
    ph ^= ((q & 1) ? (1u << n) - 1u : 0u) ^ ((1u << r) - 1u);
  }
};
// fp8: K and V have stages of their own, 0 .. 3 and 4 .. 5, taken by the blocks of all parts in turn.
template <>
struct Tiles<true> {
  uint32_t base;  // blocks before the part's
  int count;
  bool one;
  __device__ __forceinline__ void part(const Part& g) {
    count = g.count;
    one = g.one;
  }
  __device__ __forceinline__ Fill k(int block) const {
    const uint32_t n = base + block;
    return {static_cast<int>(n & 3), n >> 2 & 1};
  }
  __device__ __forceinline__ Fill v(int block) const {
    const uint32_t n = base + block;
    return {static_cast<int>(4 + (n & 1)), n >> 1 & 1};
  }
  __device__ __forceinline__ Fill out(int b) const {
    const int st = one ? 0 : b;
    return {4 + st, ((base + 1 - st >> 1) - 1) & 1};
  }
  __device__ __forceinline__ void done() { base += count; }
};

// E4M3 codes of a tile (rows of 128 bytes, TMA's 128-byte swizzle) to fp16 in the layout in which TMA lands 16-bit rows;
// exact.  128 threads, 16 codes at a time, four pieces in flight: shared memory answers in 150 clocks beside the MMAs.  Eight
// lanes read a row, and those of its second half write their pieces in the other order, so that eight lanes' stores
// meet all banks.  Rows from `valid` on become zeros (0 * NaN is NaN).  (The decode kernel's widens one piece at a time: it
// measured more in flight 2 to 8 % slower.)
__device__ __forceinline__ void widen_tile(const uint8_t* codes, uint8_t* to, int thread, int valid) {
  const int chunk = thread & 7, half = chunk >> 2, x = (thread >> 3) & 7;  // x: the row mod 8, the same in every pass
  const uint32_t flip = half;
  const uint4* from = reinterpret_cast<const uint4*>(codes + (thread >> 3) * 128 + ((chunk ^ x) << 4));
  uint4* dst = reinterpret_cast<uint4*>(to + half * 16384 + (thread >> 3) * 128);
  const uint32_t at = 2 * (chunk & 3);
#pragma unroll 1
  for (int pass = 0; pass < 8; pass += 4) {
    uint4 in[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      in[k] = from[(pass + k) * 128];
      if ((thread >> 3) + (pass + k) * 16 >= valid) in[k] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
      uint32_t out[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = e4m3x2_to_f16x2(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
      const uint4 a = make_uint4(out[0], out[1], out[2], out[3]), b = make_uint4(out[4], out[5], out[6], out[7]);
      uint4* d = dst + (pass + k) * 128;
      d[(at + flip) ^ x] = flip ? b : a;
      d[(at + 1 - flip) ^ x] = flip ? a : b;
    }
  }
}

// K's codes are multiplied as they are, so the queries are codes too, two per value: the first its E4M3 rounding, the second
// that of the rest.  Four and four significant bits hold bf16's eight exactly, down to 2^-10 of the row's largest value
// (below that the second is off by 2^-18 of the largest).  A row's scale is a power of two that brings its largest value to
// 224 .. 448.  Both take a value's 16 bits: row `row` of a tile, as TMA landed it (two halves of 64 dims), becomes 128 first and
// 128 second codes in its place.  A thread per row; returns the scale's exponent, or -128 where the row has an inf or NaN
// (its logits are NaN).  The warps that widen codes do it while the softmax warps are at the output of the part before: 20 ragged
// prompts of 40 heads take 627 us; with the softmax warps doing it 669, as a pass of its own over memory 720.
__device__ __forceinline__ int query_codes(uint8_t* tile, int row) {
  uint8_t* const at = tile + row * 128;
  const int x = row & 7;
  auto piece = [&](int half, int c) { return reinterpret_cast<uint4*>(at + half * 16384 + ((c ^ x) << 4)); };
  uint32_t m = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int c0 = 0; c0 < 8; c0 += 4) {
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = *piece(half, c0 + c);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        m = __vmaxu2(__vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu), __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu)), m);
    }
  }
  m = max(m & 0xFFFFu, m >> 16);
  // 448 = 1.75 * 2^8; a row without an inf or NaN has an exponent below 255
  const int e = static_cast<int>(m >> 7) - 127, up = m == 0 ? 0 : min(8 - e - ((m & 127) > 96 ? 1 : 0), 120);
  const float lift = __int_as_float((127 + max(up, -126)) << 23);  // up >= -120
  auto codes = [&](const uint4& v, uint2& first, uint2& second) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = fmul2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), make_float2(lift, lift));
      hi[j] = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
      const uint32_t h = e4m3x2_to_f16x2(hi[j]);
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
      lo[j] = __nv_cvt_float2_to_fp8x2(make_float2(a.x - back.x, a.y - back.y), __NV_SATFINITE, __NV_E4M3);
    }
    first = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    second = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  };
  // In an order in which a code goes where every value has been read: the upper half's second codes from behind, its first
  // codes at the end.
  auto sixteen = [&](int half, int k, uint4& first, uint4& second) {
    uint2 a, b, c, d;
    codes(*piece(half, 2 * k), a, b);
    codes(*piece(half, 2 * k + 1), c, d);
    first = make_uint4(a.x, a.y, c.x, c.y);
    second = make_uint4(b.x, b.y, d.x, d.y);
  };
  uint4 upper[4];
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    uint4 second;
    sixteen(1, k, upper[k], second);
    *piece(1, 4 + k) = second;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4 first, second;
    sixteen(0, k, first, second);
    *piece(0, k) = first;
    *piece(1, k) = second;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) *piece(0, 4 + k) = upper[k];
  return m < 0x7F80u ? up : -128;
}

template <bool FP8>
__global__ void __launch_bounds__(PromptCfg<FP8>::kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptMaps maps, PromptParams p) {
  using C = PromptCfg<FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // Two tiles of queries, each two 64-dim halves of 128 rows (fp8: which become two tiles of codes); the stages.  bf16: as the queries'
  // tiles, the last one is the second tile of queries.  fp8: K's codes, V's codes, V's values.
  uint8_t* const q_buf = smem;
  uint8_t* const ring = smem + 2 * 32768;
  uint8_t* const v_codes = ring + C::kK8 * C::kCodes;
  uint8_t* const v_ring = v_codes + C::kV8 * C::kCodes;
  PromptSmem& sm = *reinterpret_cast<PromptSmem*>(smem + 7 * 32768);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, T = p.tile_tokens;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&sm.full[i], FP8 && i >= C::kK8 ? 4 : 1);
      mbar_init(&sm.empty[i], 2);
    }
    for (int i = 0; i < C::kV8; ++i) {
      mbar_init(&sm.code_full[i], 1);
      mbar_init(&sm.code_empty[i], 4);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    mbar_init(&sm.q_ready, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.turn[i], 1);
    }
    mbar_init(&sm.ml_full, 8);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.out_free, 8);
    mbar_init(&sm.mma_done, 2);
    mbar_arrive(&sm.turn[0]);
    sm.abort_flag = 0;
    sm.err = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
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

  // stages of values: bf16 all of them, fp8 those of V
  auto stage_at = [&](int st) {
    if (FP8) return v_ring + (st - C::kK8) * C::kTile;
    return st < C::kStages ? ring + st * C::kTile : q_buf + 32768;
  };
  PartWalker<FP8> walk(p);
  Part g{};
  Tiles<FP8> tl{};
  if (warp == 9) {
    // ------------------------------------------------------------ loads: Q of a part, its tiles
    uint32_t parts = 0, queries = 0, bad = 0, blocks = 0;
    uint32_t used = 0, filled = 0;  // bf16: a bit per stage that has been filled; its last fill's parity
    bool ok = true, lent = false;   // bf16: the second tile of queries has been a stage since it was loaded last
    uint32_t lent_parity = 0;
    // Rows of a part's blocks, 32 at a time, one per lane, and their scales; the next 32 are on their way while these load.
    struct Rows {
      int row;
      float sk, sv;
    };
    auto look_up = [&](int from) {
      Rows x{0, 1.0f, 0.0f};
      const int b = g.block + from + lane;
      x.row = g.k_start + b * kBlock;
      if (p.block_table && from + lane < g.count) {
        const int e = p.block_table[static_cast<long long>(g.seq) * p.bt_stride + b];
        const bool there = e >= 0 && e < p.n_pages;
        if (!there) bad = 1;
        x.row = (there ? e : static_cast<int>(p.n_pages)) * kBlock;  // past the cache: TMA reads zeros
        if (FP8) {
          x.sk = there ? p.k_scale[static_cast<long long>(e) * p.hkv + g.head] : 1.0f;
          const float sv = there ? p.v_scale[static_cast<long long>(e) * p.hkv + g.head] : 1.0f;
          x.sv = sv == 0.0f ? -149.0f : log2f(sv);  // (a scale of 0: below the smallest)
        }
      }
      return x;
    };
    // Q: behind the first block where it waits for the part before
    auto load_q = [&] {
      if (!((parts == 0 || mbar_wait_warp(&sm.q_empty, (parts - 1) & 1, abort_flag)) &&
            (g.one || !lent || mbar_wait_warp(&sm.empty[C::kStages], lent_parity, abort_flag))))
        return false;
      if (!g.one) lent = false;
      if (lane == 0) {
        const int n = g.one ? 1 : 2;
        mbar_arrive_expect_tx(&sm.q_full, n * T * G * 256);
        for (int b = 0; b < n; ++b)
          for (int half = 0; half < 2; ++half)
            tma_load_3d(q_buf + b * 32768 + half * 16384, &maps.q, &sm.q_full, half * 64, g.head * G,
                        g.q_start + g.t0 + b * T);
      }
      __syncwarp();
      ++queries;
      return true;
    };
    // Every wait and shuffle takes 150 clocks beside the MMAs, and a tile has 1,000: the whole warp waits, and a tile's row
    // is fetched from its lane while the tile before it is waited for.
    while (ok && walk.next(g)) {
      tl.part(g);
      Rows now = look_up(0), then = look_up(32);
      int row = __shfl_sync(0xFFFFFFFFu, now.row, 0);
      if (parts == 0) ok = load_q();
      if constexpr (FP8) {
        float sk = __shfl_sync(0xFFFFFFFFu, now.sk, 0), sv = __shfl_sync(0xFFFFFFFFu, now.sv, 0);
        for (int i = 0; ok && i < g.count; ++i, ++blocks) {
          if (((i + 1) & 31) == 0) {
            now = then;
            then = look_up(i + 1 + 32);
          }
          const int next = (i + 1) & 31;
          const int next_row = __shfl_sync(0xFFFFFFFFu, now.row, next);
          const float next_sk = __shfl_sync(0xFFFFFFFFu, now.sk, next), next_sv = __shfl_sync(0xFFFFFFFFu, now.sv, next);
          const Fill k = tl.k(i);
          ok = blocks < C::kK8 || mbar_wait_warp(&sm.empty[k.st], k.parity ^ 1, abort_flag);
          if (!ok) break;
          if (lane == 0) {
            sm.k_scale[blocks & 7] = sk;
            sm.v_scale[blocks & 7] = sv;
            mbar_arrive_expect_tx(&sm.full[k.st], C::kCodes);
            tma_load_3d(ring + k.st * C::kCodes, &maps.k, &sm.full[k.st], 0, g.head, row);
          }
          __syncwarp();
          const int st = blocks & 1;
          ok = blocks < C::kV8 || mbar_wait_warp(&sm.code_empty[st], (blocks / 2 - 1) & 1, abort_flag);
          if (!ok) {
            ++blocks;  // K's tile is on its way
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.code_full[st], C::kCodes);
            tma_load_3d(v_codes + st * C::kCodes, &maps.v, &sm.code_full[st], 0, g.head, row);
          }
          __syncwarp();
          row = next_row;
          sk = next_sk;
          sv = next_sv;
          if (i == 0 && parts > 0) {
            ok = load_q();
            if (!ok) {
              ++blocks;
              break;
            }
          }
        }
      } else {
        bool v = false, next_v;
        bool out_read = parts == 0;  // the part before has read its output's stages
        for (int t = 0; ok && t < tl.total; ++t, v = next_v) {
          if (((t + 1) & 63) == 0) {  // 32 blocks in either order
            now = then;
            then = look_up(((t + 1) >> 1) + 32);
          }
          const int next = tl.block(t + 1, next_v) & 31;
          const int next_row = __shfl_sync(0xFFFFFFFFu, now.row, next);
          const CUtensorMap* map = v ? &maps.v : &maps.k;
          const int st = tl.stage(t);
          // Q of a part of one block comes before its V, which waits for the output of the part before: a look behind V could
          // come after that of this part too, and take its phase for one that is still to come.
          const bool last = t == tl.total - 1;
          if (last && t == 1 && parts > 0) {
            ok = load_q();
            if (!ok) break;
          }
          if ((st >= C::kOutStage || last) && !out_read) {
            ok = mbar_wait_warp(&sm.out_free, (parts - 1) & 1, abort_flag);
            if (!ok) break;
            out_read = true;
          }
          // its last fill, if any, has been given back
          ok = !(used >> st & 1) || mbar_wait_warp(&sm.empty[st], tl.parity(t) ^ 1, abort_flag);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.full[st], C::kTile);
            uint8_t* const dst = stage_at(st);
            tma_load_3d(dst, map, &sm.full[st], 0, g.head, row);
            tma_load_3d(dst + 16384, map, &sm.full[st], 64, g.head, row);
          }
          __syncwarp();
          used |= 1u << st;
          filled = (filled & ~(1u << st)) | tl.parity(t) << st;
          row = next_row;
          if (t == 1 && !last && parts > 0) {
            ok = load_q();
            if (!ok) break;
          }
        }
        if (g.one && tl.total > C::kStages) {  // the lent stage's last fill in this part
          const int n = C::kStages + 1;
          lent = true;
          lent_parity = tl.parity(C::kStages + (tl.total - n) / n * n);
        }
      }
      tl.done();
      ++parts;
    }
    if (!ok && lane == 0) gave_up();
    if (bad) atomicOr(&sm.err, kFlagBadIndex);
    if (lane == 0) {  // no copy may land after this CTA has left (all have, but after a wait that gave up)
      if (FP8) {
        for (uint32_t f = blocks > 4 ? blocks - 4 : 0; f < blocks; ++f) mbar_wait(&sm.full[f & 3], (f / 4) & 1, nullptr);
        for (uint32_t f = blocks > 2 ? blocks - 2 : 0; f < blocks; ++f) mbar_wait(&sm.code_full[f & 1], (f / 2) & 1, nullptr);
      } else {
        for (int st = 0; st <= C::kStages; ++st)
          if (used >> st & 1) mbar_wait(&sm.full[st], filled >> st & 1, nullptr);
      }
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
    const uint32_t idesc_s = FP8 ? idesc_e4m3(128, 128) : idesc_bf16(128, 128, false), idesc_o = FP8 ? idesc_f16(128, kHeadDim, true) : idesc_bf16(128, kHeadDim, true);
    const uint64_t q_desc = sdesc_sw128(smem_u32(q_buf), 16, 1024), k_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(FP8 ? v_ring : ring), 16384, 1024);
    const uint32_t s_col = tmem + C::kColS + b * 128, o_col = tmem + C::kColO + b * 128;
    uint32_t parts = 0;  // parts before this one
    uint32_t p_ph = 0, turn_ph = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      // step i: P V of the warpgroup's block i, S of its block i + 1
      const int every = g.one ? 2 : 1, first = g.one ? b : 0;          // its blocks: first, first + every, ...
      const int steps = g.one ? (g.count + 1) / 2 : g.count;           // of both warps; the second may have one block less
      const int blocks = g.one ? (g.count + 1 - b) / 2 : g.count;
      const uint64_t qa = q_desc + (g.one ? 0 : b * 2048);
      tl.part(g);
      ok = mbar_wait_warp(FP8 ? &sm.q_ready : &sm.q_full, parts & 1, abort_flag);
      for (int i = -1; ok && i < steps; ++i) {
        const bool pv = i >= 0 && i < blocks, s = i + 1 < blocks;
        const Fill v = tl.v(pv ? first + i * every : 0), k = tl.k(s ? first + (i + 1) * every : 0);
        if (s) ok = mbar_wait_warp(&sm.full[k.st], k.parity, abort_flag);
        if (pv) {
          ok = ok && mbar_wait_warp(&sm.full[v.st], v.parity, abort_flag);
          // O of the part before has been read
          if (i == 0 && parts > 0) ok = ok && mbar_wait_warp(&sm.o_free, (parts - 1) & 1, abort_flag);
        }
        // two looks at once take no longer than one
        ok = ok && mbar_wait_both_warp(&sm.turn[b], turn_ph, pv ? &sm.p_full[b] : &sm.turn[b], pv ? p_ph : turn_ph, abort_flag);
        if (pv) p_ph ^= 1;
        turn_ph ^= 1;
        if (!ok) break;
        tc_fence_after();
        // (bf16: the lent stage lies one tile before the first)
        const uint64_t ka = k_desc + (FP8 ? k.st * 1024 : (k.st < C::kStages ? k.st : -1) * 2048);
        const uint64_t va = v_desc + (FP8 ? v.st - C::kK8 : v.st < C::kStages ? v.st : -1) * 2048;
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
            // 64 dims (fp8: the queries' first or second codes) and 32 bytes of them
            const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
            if (FP8) umma_e4m3(s_col, qa + off, ka + (kk & 3) * 2, idesc_s, kk ? 1u : 0u);
            else umma_bf16(s_col, qa + off, ka + off, idesc_s, kk ? 1u : 0u);
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
          if (s) issue_s();
          if (!pv && !s) mbar_arrive(&sm.turn[b ^ 1]);
          if (pv) {
            if (!s) umma_commit(&sm.o_full[b]);
            give(&sm.empty[v.st]);
          }
          if (s) give(&sm.empty[k.st]);
        }
        __syncwarp();
        if (i + 1 == (blocks > 0 ? blocks - 1 : 0)) {  // its last S of the part (or the first step, if it has none)
          if (elect_one()) umma_commit(&sm.q_empty);
          __syncwarp();
        }
      }
      tl.done();
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
    const uint32_t group_inv = 65536u / G + 1;  // row * group_inv >> 16 = row / G for rows below 128
    const uint32_t la = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = la + C::kColS + b * 128, o_col = la + C::kColO + b * 128;
    constexpr float kLift = FP8 ? 7.0f : 0.0f;  // O is 2^kLift times larger than m says
    uint32_t parts = 0, steps = 0, outs = 0, merges = 0;
    bool ok = true;
    auto warp_arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool there = walk.next(g);
    // fp8: V of a part is widened when every warp has seen that its queries are codes (and has read the output's stages of the part
    // before).  Without that the next part's q_ready could come before a late warp has looked at this one's: it would wait
    // for a phase that is past.
    if (FP8 && there) {
      ok = mbar_wait_warp(&sm.q_ready, 0, abort_flag);
      if (ok) warp_arrive(&sm.out_free);
    }
    while (ok && there) {
      const int t_tile = g.t0 + (g.one ? 0 : b * T);  // the tile's first token
      const int tok = t_tile + my_t;
      const bool mine = my_t < T && tok < g.q_len;
      const int sees = p.visible ? g.past : g.past + t_tile + 1;  // keys that every row of the tile sees
      tl.part(g);
      float qc = 1.0f;  // fp8: the row's queries are codes of a scale of their own
      if constexpr (FP8) {
        const int up = sm.q_up[parts & 1][(g.one ? 0 : b * 128) + r];
        if (mine) qc = normal_factor(p.scale_log2 * __int_as_float(up == -128 ? 0x7FC00000 : (127 - up) << 23));
      }
      float m = -INFINITY;
      float d = 0.0f;  // fp8: l is that of 2^(logit - (m - d)), O that of 2^(logit + log2(V's scale) - m)
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
        const Fill vf = tl.v(blk);
        float c = p.scale_log2, lv = 0.0f;
        if constexpr (FP8) {
          // the scales come before V's codes (every earlier fill of the stage is past: its P V came before S of this step)
          if (!mbar_wait_warp(&sm.full[vf.st], vf.parity, abort_flag)) {
            ok = false;
            break;
          }
          c = normal_factor(qc * sm.k_scale[tl.base + blk & 7]);
          lv = sm.v_scale[tl.base + blk & 7];
        } else if (edge && j0 + kBlock > g.past + g.q_len && (g.one || b == 0)) {
          // V rows past the sequence's end hold anything, and 0 * NaN is NaN: zero them
          if (!mbar_wait_warp(&sm.full[vf.st], vf.parity, abort_flag)) {
            ok = false;
            break;
          }
          uint4* v = reinterpret_cast<uint4*>(stage_at(vf.st));
          for (int i = (g.past + g.q_len - j0) * 8 + r; i < kBlock * 8; i += 128) {
            v[i] = make_uint4(0, 0, 0, 0);
            v[1024 + i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        // Hides what the row does not see of 32 columns, and gives the maximum of the others.
        auto hide = [&](uint32_t (&v)[32], int q) {
          uint32_t bits;
          if (p.visible) {
            bits = mine ? tree_bits(p.visible + static_cast<long long>(g.q_start + tok) * p.mask_words, p.mask_words, g.past, g.q_len, j0 + 32 * q) : 0u;
          } else {
            const int n = g.past + tok + 1 - j0 - 32 * q;
            bits = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
          }
          float x = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (!(bits >> j & 1)) v[j] = 0xFF800000u;
            x = fmaxf(x, __uint_as_float(v[j]));
          }
          return x;
        };
        // The row of S stays in registers from its maximum to its weights.
        uint32_t v[4][32];
        auto row_max = [&] {
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld_max_32cols(s_col + 32 * q, v[q], mx[q]);
          tmem_ld_wait_regs_max(v[0], mx[0]);
#pragma unroll
          for (int q = 1; q < 4; ++q) tmem_regs_written(v[q], mx[q]);
          if (edge) {
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = hide(v[q], q);
          }
          return fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        };
        // fp8: V's scale goes to the weights as a summand of their exponents, and they are 2^7 times larger: one fp16 value each,
        // at most 2^15 whatever the pages' scales, with its 11 significant bits down to 2^-21 of the row's largest (four
        // more, with references replaced from 2^4 on, made ragged prompts 20 % slower).  The sum of weights knows no scale: its
        // reference is m less log2 of the scale that m was taken with (d), replaced for itself where a page of a smaller scale
        // has larger logits.
        const float x = fmaf(row_max(), c, lv);
        if (m == -INFINITY) {  // no key counts so far: O and l are 0, or not there yet
          m = x;
          d = lv;
        }
        float up = x - m, t = d - lv;
        auto is_large = [&] { return fabsf(m) >= kRoundLogits && m != -INFINITY; };
        // (rows of nobody hold what the stages held before: they neither rescale nor round)
        if (__any_sync(0xFFFFFFFFu, mine && (FP8 ? up + fmaxf(t, 0.0f) > 8.0f || t > 60.0f || is_large() : up > 8.0f || is_large()))) {
          const bool rise = mine && up > 8.0f, grow = FP8 ? rise || (mine && up + t > 8.0f) : rise;
          if (__any_sync(0xFFFFFFFFu, grow)) {  // O is complete: its P V came before this S
            const float gap = up + t, k = grow && gap > 0.0f ? exp2_approx(-gap) : 1.0f;
            l2.x *= k;
            if (!FP8) l2.y *= k;
            if (FP8 && grow) d = rise ? (gap > 0.0f ? lv : d + up) : d - gap;
            scale_row(o_col, rise ? exp2_approx(-up) : 1.0f);
            row_max();  // the row again
            if (rise) m = x;
            t = d - lv;
          }
          const bool large = is_large(), far = t > 60.0f;
          const float add = FP8 && large ? lv : 0.0f, less = FP8 && large ? m : 0.0f;
          if (FP8 && __any_sync(0xFFFFFFFFu, mine && far)) {
            // a page of a scale so much smaller: weights that still count in the sum are too small for fp32
            const float off = large ? t : d - m;
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < 32; ++j) sum += exp2_approx(fmaf(__uint_as_float(v[q][j]), c, add) - less + off);
            if (far) {
              l2.x += sum;
              t = -INFINITY;
            }
          }
          if (__any_sync(0xFFFFFFFFu, mine && large)) {
            // Products rounded to fp32 logits before the reference is taken off: see kRoundLogits.  fp8: with V's scale in the same
            // rounding, which is the reference's, and the lift behind the difference: from logits of 2^23 on either would be
            // rounded away by itself, and the largest weights pass fp16.
            const float k = large ? c : 1.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float s = __uint_as_float(v[q][j]);
                v[q][j] = __float_as_uint(FP8 ? fmaf(s, k, add) - less : s * k);
              }
            if (large) c = 1.0f;
            if (FP8 && large) lv = m;
          }
        }
        const float off = m == -INFINITY ? 0.0f : lv - m + kLift;  // -inf - -inf is NaN
        const float2 c2 = make_float2(c, c), nm = make_float2(off, off);
        float2 sum = FP8 ? make_float2(0.0f, 0.0f) : l2;
        auto weights = [&](uint32_t (&v)[32], int q) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 z = ffma2(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), c2, nm);
            const float2 e = make_float2(exp2_approx(z.x), exp2_approx(z.y));
            sum = fadd2(sum, e);
            w[j] = FP8 ? pack_f16(e.x, e.y) : pack_bf16(e.x, e.y);
          }
          tmem_st_16cols(s_col + 16 * q, w);
        };
#pragma unroll
        for (int q = 0; q < 4; ++q) weights(v[q], q);
        if (FP8) {
          const float back = exp2_approx(t - kLift);
          l2.x = fmaf(sum.x + sum.y, back, l2.x);
        } else {
          l2 = sum;
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.p_full[b]);
      }
      if (!ok) break;
      tl.done();

      // ---- output
      Part then{};
      there = walk.next(then);  // looked up while P V runs
      const bool some = had < g.count;
      if (some) {
        if (!mbar_wait_warp(&sm.o_full[b], outs & 1, abort_flag)) {
          ok = false;
          break;
        }
        ++outs;
        tc_fence_after();
      }
      float l = FP8 ? l2.x : l2.x + l2.y;
      if constexpr (FP8) {
        // O, m and l with one reference; an excess of d goes to O and m, so that l is within 2^40 of a sum of weights in every part
        // and the merge's factors do not lose one beside another
        const float less = d - fminf(fmaxf(d, -40.0f), 40.0f);
        if (__any_sync(0xFFFFFFFFu, mine && less != 0.0f)) {
          scale_row(o_col, exp2_approx(less));
          tc_fence_before();
          m -= less;
        }
        l *= exp2_approx(less - d);
      }
      if (l != l) m = INFINITY;  // a NaN among the logits, of which the maximum may know nothing: it passes every merge
      const bool whole = g.first && g.last;
      const long long part_at = static_cast<long long>(blockIdx.x) * 4 + (g.first ? 2 : 0) + (g.one ? 0 : b);  // a tile's
      float f_own = 1.0f, f_other = 0.0f;  // what this warpgroup's and the other's O count with
      if (g.one) {  // both warpgroups' sums of a row; each writes half of the dims
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
        f_own = exp2_diff(m, top);
        f_other = exp2_diff(other.x, top);
        l = b == 0 ? fmaf(l, f_own, other.y * f_other) : fmaf(other.y, f_other, l * f_own);  // the same in both
        m = top;
      }
      // A row without a key that counts has O = 0.
      const float inv = l == 0.0f ? 0.0f : (whole ? 1.0f / l : 1.0f) * (FP8 ? 0x1p-7f : 1.0f);
      f_own *= inv;
      f_other *= inv;
      // Where a warpgroup had no block of the part its O holds an older one's (uniform: by the part alone).
      const bool own_there = some, other_there = g.one && (b == 0 ? g.count > 1 : true);
      const uint32_t other_col = la + C::kColO + (b ^ 1) * 128;
      const int dim0 = g.one ? b * 64 : 0, chunks = g.one ? 2 : 4;
      // The output goes through a stage of the ring (whose last tile has been multiplied), each warp's rows by the warp
      // itself, so that a store writes whole rows: with 16 bytes of 32 rows to a store the output took 7,200 clocks of every
      // part, through shuffles (150 clocks each beside the MMAs) more.
      const Fill of = tl.out(b);
      uint8_t* const stage = stage_at(of.st);
      if (whole && !mbar_wait_warp(&sm.empty[of.st], of.parity, abort_flag)) {
        ok = false;
        break;
      }
#pragma unroll 1
      for (int q = 0; q < chunks; ++q) {
        const int dim = dim0 + q * 32;
        uint32_t x[32];
        tmem_ld_32cols(o_col + dim, x);
        tmem_ld_wait_regs(x);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = own_there && f_own != 0.0f ? __float_as_uint(__uint_as_float(x[j]) * f_own) : 0u;
        if (other_there) {
          uint32_t y[32];
          tmem_ld_32cols(other_col + dim, y);
          tmem_ld_wait_regs(y);
          if (f_other != 0.0f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(fmaf(__uint_as_float(y[j]), f_other, __uint_as_float(x[j])));
          }
        }
        if (whole) {
          uint8_t* const to = stage + (dim >> 6) * 16384 + r * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = pack_bf16(__uint_as_float(x[8 * k + 2 * i]), __uint_as_float(x[8 * k + 2 * i + 1]));
            const int chunk = (dim >> 3 & 4) + k;
            *reinterpret_cast<uint4*>(to + ((chunk ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
          // partials: four dims of 128 rows after four dims of 128 rows
          float* const to = p.part_o + ((part_at * 32 + dim / 4) * 128 + r) * 4;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(to + k * 512) = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
      }
      tc_fence_before();
      warp_arrive(&sm.o_free);  // (synchronises the warp)
      if (mine && (!g.one || b == 0)) {
        if (whole) p.lse[(static_cast<long long>(g.q_start) + tok) * p.hq + g.head * G + my_h] = (m + log2f(l)) * kLn2;
        else p.part_ml[part_at * 128 + r] = make_float2(m, l);
      }
      if (whole) {
        __nv_bfloat16* const out = p.o + ((static_cast<long long>(g.q_start) + t_tile) * p.hq + g.head * G) * kHeadDim;
        const int left = min(T, g.q_len - t_tile);
        const int per = g.one ? 8 : 16;                  // lanes to a row
        const int c = lane & (per - 1), half = g.one ? b : c >> 3;
#pragma unroll(FP8 ? 4 : 2)
        for (int i = lane / per; i < 32; i += 32 / per) {
          const int row = (warp & 3) * 32 + i;
          const int t = static_cast<int>(static_cast<uint32_t>(row) * group_inv >> 16), h = row - t * G;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + half * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
          if (t < left)
            *reinterpret_cast<uint4*>(out + (static_cast<long long>(t) * p.hq + h) * kHeadDim + half * 64 + (c & 7) * 8) = w;
        }
        fence_proxy_async_smem();  // before the stage is loaded again
      }
      ++parts;
      if (FP8 && there && !mbar_wait_warp(&sm.q_ready, parts & 1, abort_flag)) {
        ok = false;
        break;
      }
      warp_arrive(&sm.out_free);
      g = then;
    }
    if (!ok && lane == 0) gave_up();
  } else if (FP8 && warp >= 12) {
    // ------------------------------------------------------------ V's codes to fp16
    const int thread = threadIdx.x - 384;
    uint32_t blocks = 0, parts = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
      if constexpr (FP8) {
        tl.part(g);
        // the queries, while the part before ends
        ok = mbar_wait_warp(&sm.q_full, parts & 1, abort_flag);
        if (!ok) break;
#pragma unroll 1
        for (int b = 0; b < (g.one ? 1 : 2); ++b) sm.q_up[parts & 1][b * 128 + thread] = static_cast<int8_t>(query_codes(q_buf + b * 32768, thread));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready);
        // the part before has read its output's stages, and these queries have been seen
        ok = mbar_wait_warp(&sm.out_free, parts & 1, abort_flag);
        for (int i = 0; ok && i < g.count; ++i, ++blocks) {
          const int cs = blocks & 1;
          const Fill v = tl.v(i);
          ok = mbar_wait_warp(&sm.code_full[cs], blocks >> 1 & 1, abort_flag) &&
               (blocks < C::kV16 || mbar_wait_warp(&sm.empty[v.st], v.parity ^ 1, abort_flag));
          if (!ok) break;
          // rows past the sequence's end: zeros, as 0 * NaN is NaN
          widen_tile(v_codes + cs * C::kCodes, stage_at(v.st), thread, g.past + g.q_len - (g.block + i) * kBlock);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.code_empty[cs]);
            mbar_arrive(&sm.full[v.st]);
          }
        }
        tl.done();
        ++parts;
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
// Merges the partials of the items that cross runs.  Every CTA lists them (one thread per pair of runs) and takes its share of
// the tasks: 32 of an item's 256 rows and 32 of the dims.  A row to a lane, so that what a warp reads (four dims of 32
// rows) lies together; 16 dims to a warp and every fourth partial (a sequence alone has one per run, and few rows),
// four of them in flight.
constexpr int kJoinWarps = 8;
constexpr int kJoinCtas = 304;
static_assert(kPromptMaxCtas <= kJoinWarps * 32, "a thread per run");
constexpr int kJoinFew = 4;  // an item of so many partials: its rows' dims go to the warps, not its partials
struct JoinSmem {
  union {
    struct {
      float4 sums[kJoinWarps][4][32];
      float2 ml[kJoinWarps][32];
      uint2 turned[32][9];
    };
    uint2 rows_turned[32][34];
  };
  int4 item[kPromptMaxCtas];  // first run, last run, first query row, head
  int2 rows[kPromptMaxCtas];  // first token, new tokens of the sequence
  int2 in_warp[kJoinWarps];  // items of many and of few partials
};
// Rows task / 4 and dims task % 4 of an item.
__device__ __forceinline__ void join_rows(const PromptParams& p, JoinSmem& sm, int4 item, int2 rows, int task) {
  const int run = item.x, last = item.y, q_start = item.z, head = item.w, t0 = rows.x, q_len = rows.y;
  const int b = task >> 4, row0 = (task >> 2 & 3) * 32;  // tile and first row
  if (t0 + b * p.tile_tokens >= q_len || row0 >= p.tile_tokens * p.group) return;  // nobody's rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = row0 + lane, sub = warp >> 1;
  const int quad0 = (task & 3) * 8 + (warp & 1) * 4;  // first of the warp's four quadruples of dims
  float m = -INFINITY, l = 0.0f;
  float4 a[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = run + sub; i0 <= last; i0 += 16) {
    float2 x[4];
    float4 v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 4 * u;
      const long long at = static_cast<long long>(i) * 4 + (i == run ? 2 : 0) + b;
      x[u] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i > last) continue;
      x[u] = p.part_ml[at * 128 + row];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[u][c] = *reinterpret_cast<const float4*>(p.part_o + ((at * 32 + quad0 + c) * 128 + row) * 4);
    }
    const float nm = fmaxf(fmax3(m, x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
    const float k = exp2_diff(m, nm);
    l *= k;
    m = nm;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      a[c].x *= k; a[c].y *= k; a[c].z *= k; a[c].w *= k;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = exp2_diff(x[u].x, m);
      if (f == 0.0f) continue;  // what a part without a key that counts left does not
      l = fmaf(x[u].y, f, l);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        a[c].x = fmaf(v[u][c].x, f, a[c].x);
        a[c].y = fmaf(v[u][c].y, f, a[c].y);
        a[c].z = fmaf(v[u][c].z, f, a[c].z);
        a[c].w = fmaf(v[u][c].w, f, a[c].w);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) sm.sums[warp][c][lane] = a[c];
  sm.ml[warp][lane] = make_float2(m, l);
  __syncthreads();
  {
    // the four warps of the same dims, in order; each takes one of the four quadruples
    const int c = sub, w0 = warp & 1;
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, sm.ml[w0 + 2 * u][lane].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 x = sm.ml[w0 + 2 * u][lane];
      const float4 v = sm.sums[w0 + 2 * u][c][lane];
      const float f = exp2_diff(x.x, top);
      l = fmaf(x.y, f, l);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    m = top;
    const float inv = inverse(l);
    sm.turned[lane][w0 * 4 + c] = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
  auto out_row = [&](int r) {  // of the output, or -1: a row of nobody
    const int t = r / p.group, h = r - t * p.group, tok = t0 + b * p.tile_tokens + t;
    if (t >= p.tile_tokens || tok >= q_len) return -1LL;
    return (static_cast<long long>(q_start) + tok) * p.hq + head * p.group + h;
  };
  __syncthreads();
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7;  // 8 lanes write 64 bytes of a row
  const long long out = out_row(row0 + r);
  if (out >= 0) *reinterpret_cast<uint2*>(p.o + out * kHeadDim + (task & 3) * 32 + c * 4) = sm.turned[r][c];
  const long long lse_at = out_row(row);
  if (threadIdx.x < 32 && (task & 3) == 0 && lse_at >= 0) p.lse[lse_at] = (m + log2f(l)) * kLn2;
  __syncthreads();  // the next task's sums
}

// The same for few partials: 32 rows (task) and every dim, 16 of them a warp's, all partials in flight at once.  With the
// tasks above 50 items of two or three partials took 11 us (now 7), and most warps had nothing to read.
__device__ __forceinline__ void join_few(const PromptParams& p, JoinSmem& sm, int4 item, int2 rows, int task) {
  const int run = item.x, last = item.y, q_start = item.z, head = item.w, t0 = rows.x, q_len = rows.y;
  const int b = task >> 2, row0 = (task & 3) * 32;  // tile and first row
  if (t0 + b * p.tile_tokens >= q_len || row0 >= p.tile_tokens * p.group) return;  // nobody's rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = row0 + lane;
  float2 x[kJoinFew];
  float4 v[kJoinFew][4];
#pragma unroll
  for (int u = 0; u < kJoinFew; ++u) {
    const long long at = static_cast<long long>(run + u) * 4 + (u == 0 ? 2 : 0) + b;
    x[u] = make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (run + u > last) continue;
    x[u] = p.part_ml[at * 128 + row];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      v[u][c] = *reinterpret_cast<const float4*>(p.part_o + ((at * 32 + warp * 4 + c) * 128 + row) * 4);
  }
  static_assert(kJoinFew == 4, "the maximum of four");
  const float m = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
  float l = 0.0f;
  float4 a[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kJoinFew; ++u) {
    const float f = exp2_diff(x[u].x, m);
    if (f == 0.0f) continue;  // what a part without a key that counts left does not
    l = fmaf(x[u].y, f, l);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      a[c].x = fmaf(v[u][c].x, f, a[c].x);
      a[c].y = fmaf(v[u][c].y, f, a[c].y);
      a[c].z = fmaf(v[u][c].z, f, a[c].z);
      a[c].w = fmaf(v[u][c].w, f, a[c].w);
    }
  }
  const float inv = inverse(l);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    sm.rows_turned[lane][warp * 4 + c] = make_uint2(pack_bf16(a[c].x * inv, a[c].y * inv), pack_bf16(a[c].z * inv, a[c].w * inv));
  auto out_row = [&](int r) {  // of the output, or -1: a row of nobody
    const int t = r / p.group, h = r - t * p.group, tok = t0 + b * p.tile_tokens + t;
    if (t >= p.tile_tokens || tok >= q_len) return -1LL;
    return (static_cast<long long>(q_start) + tok) * p.hq + head * p.group + h;
  };
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // 16 lanes write a row
    const int r = (threadIdx.x >> 4) + 16 * i, c = threadIdx.x & 15;
    const long long out = out_row(row0 + r);
    if (out >= 0) *reinterpret_cast<uint4*>(p.o + out * kHeadDim + c * 8) = *reinterpret_cast<const uint4*>(&sm.rows_turned[r][2 * c]);
  }
  const long long lse_at = out_row(row);
  if (threadIdx.x < 32 && lse_at >= 0) p.lse[lse_at] = (m + log2f(l)) * kLn2;
  __syncthreads();  // the next task's rows
}

__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(PromptParams p) {
  __shared__ JoinSmem sm;
  griddep_wait();
  const int run = threadIdx.x;
  int4 item = make_int4(-1, 0, 0, 0);
  int2 rows = make_int2(0, 0);
  if (run + 1 < kPromptMaxCtas) {
    // the item that goes on behind run `run`, if one does: that of the next run's first block (past the last run
    // neither is a value, and not used)
    const int runs = p.plan->runs, j = p.run_item[run + 1];
    const long long total = p.plan->total, lo = p.run_at[run], edge = p.run_at[run + 1];  // where the two begin
    if (run + 1 < runs) {
      const PromptItem it = p.items[j];
      const long long base = it.base * p.hkv, n = item_cost(p, it);
      const int head = static_cast<int>((edge - base) / n);
      const long long start = base + head * n;
      if (start != edge && start >= lo) {  // it began in this run; the last run that begins before its end has its end
        item = make_int4(run, static_cast<int>(((start + n) * runs - 1) / total), it.q_start, head);
        rows = make_int2(it.t0, it.q_len);
      }
    }
  }
  // the lists have one order in all CTAs: items of many partials from the front, those of few from behind
  const bool is = item.x >= 0, few = is && item.y - item.x < kJoinFew;
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, is), some_few = __ballot_sync(0xFFFFFFFFu, few), some_many = some & ~some_few;
  const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
  if ((threadIdx.x & 31) == 0) sm.in_warp[threadIdx.x >> 5] = make_int2(__popc(some_many), __popc(some_few));
  __syncthreads();
  int n_many = 0, n_few = 0, at = __popc((few ? some_few : some_many) & below);
  for (int w = 0; w < kJoinWarps; ++w) {
    const int2 n = sm.in_warp[w];
    if (w < static_cast<int>(threadIdx.x >> 5)) at += few ? n.y : n.x;
    n_many += n.x;
    n_few += n.y;
  }
  if (is) {
    if (few) at = kPromptMaxCtas - 1 - at;
    sm.item[at] = item;
    sm.rows[at] = rows;
  }
  __syncthreads();
  for (int task = blockIdx.x; task < n_many * 32 + n_few * 8; task += gridDim.x) {
    if (task < n_many * 32) {
      join_rows(p, sm, sm.item[task >> 5], sm.rows[task >> 5], task & 31);
    } else {
      const int t = task - n_many * 32, i = kPromptMaxCtas - 1 - (t >> 3);
      join_few(p, sm, sm.item[i], sm.rows[i], t & 7);
    }
  }
}

template <bool FP8>
cudaError_t launch_attn(const PromptMaps& maps, const PromptParams& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(prompt_attn_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kPromptSmemBytes));
  if (e != cudaSuccess) return e;
  // the register reallocation's increases must fit in the launch allocation, or they would never complete
  static std::atomic<int> built{0};  // registers of the kernel, once they have been read
  int regs = built.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, prompt_attn_kernel<FP8>);
    if (e != cudaSuccess) return e;
    built.store(regs = fa.numRegs, std::memory_order_relaxed);
  }
  if (regs < PromptCfg<FP8>::kOtherRegs || regs * PromptCfg<FP8>::kThreads < PromptCfg<FP8>::kRegsNeeded) return cudaErrorInvalidConfiguration;
  return launch_pdl(prompt_attn_kernel<FP8>, dim3(p.ctas), dim3(PromptCfg<FP8>::kThreads), kPromptSmemBytes, stream, maps, p);
}

}  // namespace

bool prompt_may_split(int max_nb) { return max_nb > kWholeBlocks; }

cudaError_t launch_prompt_attn(const PromptMaps& maps, const PromptParams& p, bool fp8, cudaStream_t stream) {
  cudaError_t e = launch_pdl(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (p.total_q == 0) return cudaSuccess;  // the lengths have been checked; there is no row to compute
  e = fp8 ? launch_attn<true>(maps, p, stream) : launch_attn<false>(maps, p, stream);
  if (e != cudaSuccess) return e;
  note_launches(1);
  if (!p.part_o) return cudaSuccess;
  e = launch_pdl(prompt_join_kernel, dim3(kJoinCtas), dim3(kJoinWarps * 32), 0, stream, p);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace msa
