// kernels.h -- internal launch interface between the C ABI (api.cu) and the
// kernels.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace msa {

struct WsHeader;
struct SeqInfo;

// Adds n to the library's count of enqueued kernels (msa_kernel_launch_count).
void note_launches(int n);

// Launches `kernel` with programmatic dependent launch allowed (see griddep_wait in common.cuh): the kernel
// must call griddep_wait() before it touches memory of the kernel before it on the stream.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------- planning
struct PlanParams {
  int num_seqs;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int total_q, total_k, max_q, max_k;
  int qt;               // queries per index-scoring tile (0: build no tile list)
  int max_nb;           // ceil(max_k / 128)
  SeqInfo* seq;         // [num_seqs]
  int32_t* blk_off;     // [num_seqs + 1] exclusive prefix of key blocks
  int32_t* tile_base;   // [num_seqs + 1] scratch
  int32_t* hist;        // [max_nb + 2] scratch
  int32_t* cursor;      // [max_nb + 2] scratch
  int2* tiles;          // [max_tiles] (seq, first query) sorted by descending cost
  WsHeader* hdr;
};
cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream);

// Device-wide exclusive scan of n int32 values; out has n + 1 entries (the
// last is the total).  If total_dst != nullptr the total is also stored there.
// tmp needs scan_tmp_ints(n) int32 elements.
int scan_tmp_ints(int n);
cudaError_t launch_exclusive_scan(const int32_t* in, int32_t* out, int n, int32_t* tmp, uint32_t* total_dst,
                                  const WsHeader* hdr, cudaStream_t stream);

// ---------------------------------------------------------------- index branch
struct IndexParams {
  const SeqInfo* seq;
  const int2* tiles;
  WsHeader* hdr;
  int hkv, d_idx, topk, qt;
  float* pooled;
  int64_t pooled_stride;
  int32_t* idx;
  // fp8 index (launch with fp8 = true; tq / tk then map E4M3 codes, d_idx 128): Q_idx scales [total_q * hkv],
  // K_idx scales [n_key_blocks], first key block of each sequence
  const float* q_scale;
  const float* k_scale;
  const int32_t* blk_off;
};
size_t index_score_smem_bytes(bool fp8);
cudaError_t launch_index_score(const CUtensorMap& tq, const CUtensorMap& tk, const IndexParams& p, bool fused,
                               bool fp8, int grid, cudaStream_t stream);

// Top-k over pooled rows r = i * hkv + g (rows of queries, or of decode
// sequences when every q_len is 1).
struct TopkParams {
  int num_seqs, total_q, hkv, topk, max_nb;
  bool one_query_per_seq;  // every sequence has exactly one query (a decode batch): query i is sequence i
  const int32_t* cu_q;
  const SeqInfo* seq;
  const float* pooled;
  int64_t pooled_stride;
  int32_t* idx;
  WsHeader* hdr;
};
cudaError_t launch_topk_pooled(const TopkParams& p, int max_nb, cudaStream_t stream);

// Decode index scan: pooled scores of the single query of each sequence.
struct DecodeScanParams {
  int num_seqs, hkv, d_idx;
  const SeqInfo* seq;
  const __nv_bfloat16* q_idx;   // [num_seqs, hkv, d_idx]
  // fp8 index (launch with fp8 = true; tk then maps E4M3 codes, d_idx 128): Q_idx codes and scales
  // [num_seqs * hkv], K_idx scales per key block (packed: first block of each sequence in blk_off) or per page
  const uint8_t* q_idx8;
  const float* q_scale;
  const float* k_scale;
  const int32_t* blk_off;
  float* pooled;                // [num_seqs * hkv, pooled_stride]
  int64_t pooled_stride;
  int units_per_seq;            // work units per sequence
  int blocks_per_unit;
  long long total_k;            // rows of K_idx (for checked builds)
  WsHeader* hdr;
  // Paged cache (optional): key block b of sequence s is page block_table[s * bt_stride + b] of 128 rows;
  // null: packed rows starting at the sequence's k_start.
  const int32_t* block_table;
  int bt_stride;
  long long n_pages;
};
size_t decode_scan_smem_bytes();
cudaError_t launch_decode_scan(const CUtensorMap& tk, const DecodeScanParams& p, bool fp8, int grid,
                               cudaStream_t stream);

// ---------------------------------------------------------------- main branch
// Partial results of one (query, group, slot): G rows of 128 16-bit values + G
// lse + G log weights.  The true partial output (normalised within the block)
// is o * exp(ow - lse): the decode kernel stores it as is in bf16 (ow = lse),
// the prefill kernel in fp16 over V scaled by 2^-e, whose magnitude stays below
// 2^14 (ow = lse + e ln 2; for fp8 V, ow = lse + ln of the V scale): fp16's 11
// significant bits keep the partial's rounding well under the output's own
// bf16 rounding.
struct PartialBuffers {
  uint16_t* o;        // [total_q, hkv, topk, G, 128]: fp16 (prefill) or bf16 (decode)
  float* lse;         // [total_q, hkv, topk, G]
  float* ow;          // [total_q, hkv, topk, G]
};

// fp16 copy of V for the prefill Main Branch: V * 2^-v_scale_shift(max |V|).
// Two launches: max |V| into hdr->vmax_bits (zeroed by the caller), then the copy.
cudaError_t launch_v_prep(const __nv_bfloat16* v, __half* v16, long long n_elems, WsHeader* hdr, int sms,
                          cudaStream_t stream);

// Main Branch work item: at most this many tiles (of qpt <= 16 queries each).
constexpr int kTilesPerChunk = 16;

// A schedule entry packs one incidence as (query << kSlotBits) | slot (slot < topk <= 64).
constexpr int kSlotBits = 6;
constexpr int kSlotMask = (1 << kSlotBits) - 1;

struct ScheduleParams {
  int num_seqs, total_q, hkv, topk, window, total_blocks, n_windows, qpc;
  const int32_t* cu_q;
  const SeqInfo* seq;
  const int32_t* blk_off;
  const int32_t* idx;
  int32_t* count;         // [n_buckets]
  int32_t* bucket_start;  // [n_buckets + 1]
  int32_t* cursor;        // [n_buckets]
  int32_t* nchunk;        // [n_buckets]
  int32_t* chunk_start;   // [n_buckets + 1]
  int32_t* entries;       // [total_q * hkv * topk]: (query << kSlotBits) | slot
  int4* chunks;           // [max_chunks] (begin, count, g | block << 8, seq)
  int32_t* scan_tmp;
  WsHeader* hdr;
  long long n_buckets;
};
cudaError_t launch_schedule(const ScheduleParams& p, cudaStream_t stream);

struct AttnParams {
  const __nv_bfloat16* q;  // [total_q, hq, 128] (also behind tm_q; read directly for L2 prefetches)
  const SeqInfo* seq;
  const int4* chunks;
  const int32_t* entries;
  PartialBuffers part;
  WsHeader* hdr;
  int hkv, group, topk, qpt;
  float scale_log2;       // softmax scale * log2(e)
  // fp8 K/V (tk / tv then map the 16-bit copies of the codes): scales [n_key_blocks, hkv], first key block of
  // each sequence; null for bf16 K/V
  const float* k_scale;
  const float* v_scale;
  const int32_t* blk_off;
};
size_t sparse_attn_smem_bytes();
cudaError_t launch_sparse_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const AttnParams& p, int grid, cudaStream_t stream);

struct DecodeAttnParams {
  int num_seqs, hkv, group, topk;
  int sms;                 // persistent grid size
  const SeqInfo* seq;
  const int32_t* idx;      // [num_seqs, hkv, topk]
  PartialBuffers part;     // Q [num_seqs, hq, 128] comes through a tensor map (min(G, 16) heads x 64 dims boxes)
  float scale_log2;
  WsHeader* hdr;
  const int32_t* block_table;  // as in DecodeScanParams
  int bt_stride;
  long long n_pages;
  // fp8 K/V (launch with fp8 = true; tk / tv then map E4M3 codes): scales [n_key_blocks, hkv] and the first key
  // block of each sequence
  const float* k_scale;
  const float* v_scale;
  const int32_t* blk_off;
};
size_t decode_attn_smem_bytes();
cudaError_t launch_decode_attn(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const DecodeAttnParams& p, bool fp8, cudaStream_t stream);

// ---------------------------------------------------------------- index prologue
// Hidden states -> Q_idx and the new tokens' K_idx rows (projection, RMSNorm, RoPE on dims 0..63).
struct PrologueParams {
  int num_seqs, total_q, hkv, d_model;
  const int32_t* cu_q;
  const SeqInfo* seq;
  const __nv_bfloat16* gamma_q;  // [128]
  const __nv_bfloat16* gamma_k;  // [128]
  __nv_bfloat16* q_idx;          // [total_q, hkv, 128]
  __nv_bfloat16* k_idx;          // [total_k, 128]: row k_start + pos(i) of token i
  float rope_turns_hi[32];       // theta_j / (2 pi) = hi + lo, theta_j = 10000^(-j/32)
  float rope_turns_lo[32];
  WsHeader* hdr;
};
size_t index_prologue_smem_bytes();
cudaError_t launch_index_prologue(const CUtensorMap& tx, const CUtensorMap& twq, const CUtensorMap& twk,
                                  const PrologueParams& p, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- fp8 K/V
// Quantization of bf16 K and V to E4M3 codes with one scale per (key block, KV head).
struct QuantParams {
  int num_seqs, hkv;
  const SeqInfo* seq;
  const int32_t* blk_off;       // [num_seqs + 1] first key block of each sequence (plan)
  const __nv_bfloat16* k;       // [total_k, hkv, 128]
  const __nv_bfloat16* v;
  uint8_t* k8;                  // [total_k, hkv, 128] E4M3 codes
  uint8_t* v8;
  float* k_scale;               // [n_key_blocks, hkv]
  float* v_scale;
  WsHeader* hdr;
};
cudaError_t launch_quantize_kv_fp8(const QuantParams& p, long long max_blocks, cudaStream_t stream);
// Quantization of the index inputs to E4M3 codes: K_idx with one scale per key block of a sequence, Q_idx with
// one per (query row, group); either side may be skipped (null input).  d_idx 128.
struct IndexQuantParams {
  int num_seqs, hkv, total_q;
  const SeqInfo* seq;
  const int32_t* blk_off;
  const __nv_bfloat16* q_idx;   // [total_q, hkv, 128] or null
  const __nv_bfloat16* k_idx;   // [total_k, 128] or null
  uint8_t* q8;
  float* q_scale;               // [total_q * hkv]
  uint8_t* k8;
  float* k_scale;               // [n_key_blocks]
  long long key_ctas;           // CTAs of the grid that take key blocks (the rest take query rows)
  WsHeader* hdr;
};
cudaError_t launch_quantize_index_fp8(const IndexQuantParams& p, cudaStream_t stream);
// 16-bit copies of fp8 K (bf16) and V (fp16) for the prefill Main Branch; exact.
cudaError_t launch_kv8_widen(const uint8_t* k8, const uint8_t* v8, __nv_bfloat16* k16, __half* v16,
                             long long n_elems, const WsHeader* hdr, int sms, cudaStream_t stream);

struct CombineParams {
  int total_q, hq, hkv, group, topk, num_seqs;
  bool one_query_per_seq;  // as in TopkParams
  int sms;  // grid: two CTAs per SM, grid-stride over the (query, head pair) items
  const int32_t* cu_q;
  const SeqInfo* seq;
  const int32_t* idx;
  PartialBuffers part;
  __nv_bfloat16* o;
  float* lse;
  WsHeader* hdr;
};
// f16_partials: the partial outputs are fp16 (prefill) rather than bf16 (decode).
cudaError_t launch_combine(const CombineParams& p, bool f16_partials, cudaStream_t stream);

// ---------------------------------------------------------------- dense decode attention
// One new token per sequence over every key of a paged cache.
constexpr int kDenseTile = 64;      // keys of a work unit (128 where the split runs on tcgen05)
constexpr int kDenseMaxCtas = 320;  // CTAs of the split at most (two per SM), or num_kv_heads where that is more
struct DenseDecodeParams {
  int num_seqs, hkv, group, max_k, total_k;
  int groups;                   // runs the batch is cut into; groups * hkv CTAs
  int unit_shift;               // a work unit has 1 << unit_shift keys
  const int32_t* cu_k;
  const __nv_bfloat16* q;       // [num_seqs, hkv * group, 128]
  const int32_t* block_table;   // [num_seqs, bt_stride]
  int bt_stride;
  long long n_pages;
  const float* k_scale;         // fp8: [n_pages, hkv]
  const float* v_scale;
  __nv_bfloat16* o;             // [num_seqs, hkv * group, 128]
  float* lse;                   // [num_seqs, hkv * group]
  float* weight;                // [num_seqs, hkv, weight_stride] or null
  long long weight_stride;
  float scale_log2;             // softmax scale * log2(e)
  // workspace
  WsHeader* hdr;                // only the status is written
  float* part_o;                // [groups, hkv, 2, group, 128]: slot 1 the sequence that goes on behind the run
  float2* part_ml;              // [groups, hkv, 2, group] (maximum in log2 units, sum)
  // [entries, hkv] the sequences that cross runs: (sequence or -1, first run, last run), an entry per sequence (by_seq,
  // num_seqs <= groups) or per run (the sequence that begins there and goes on)
  int4* meta;
  bool by_seq;
  uint32_t* flags;              // [groups, hkv] device error flags
  float* logits;                // with weight: [units, hkv, group, unit's keys] in log2 units; else null
  float2* norm;                 // with weight: [num_seqs, hkv * group] (maximum, 1 / sum); else null
};
int dense_decode_ctas_per_sm(int group);
// Whether the split runs on tcgen05 (units of 128 keys).  Its time hardly depends on the group (47 to 49 us for 160 MB of
// bf16 pages at 64 to 128 heads, 42 to 44 us for 80 MB of E4M3); the other kernel, which repeats its work for every 16
// heads, takes 36 us for either at 17 to 32 and 51 us for the E4M3 pages at 33 to 64.
bool dense_decode_tc(int group);
constexpr int kDenseTail = 16;  // rows of the boxes that a sequence's last unit is loaded by
struct DenseMaps {
  CUtensorMap k, v;            // boxes of a unit's rows of one head (64 dims in bf16, 128 codes in fp8)
  CUtensorMap k_tail, v_tail;  // boxes of kDenseTail rows (not on tcgen05)
  CUtensorMap q;               // on tcgen05: boxes of 64 dims of a group's heads
};
cudaError_t launch_dense_decode(const DenseMaps& maps, const DenseDecodeParams& p, bool fp8, cudaStream_t stream);

// ---------------------------------------------------------------- dense attention of prompts and drafted trees
constexpr int kPromptMaxCtas = 160;  // CTAs of the attention kernel at most (one per SM)
// What the plan kernel leaves for the others.
struct PromptPlan {
  long long total;  // cost of all items and KV heads
  int n_items;
  int runs;         // > 0: all blocks are cut into so many runs; 0: items are taken whole
};
// Up to two tiles of new tokens of a sequence, for every KV head.
struct PromptItem {
  int seq, t0;                     // its first token
  int q_start, q_len, k_start, past;  // the sequence: first query row, new tokens, first key row, cached keys
  int blocks;                      // key blocks of the item
  long long base;                  // with runs: cost of the items before it, for one KV head
};
struct PromptParams {
  int num_seqs, hq, hkv, group, total_q, total_k, max_q, max_k, max_nb;
  int tile_tokens;              // 128 / group: tokens of a tile; an item has two tiles
  int ctas;                     // grid of the attention kernel
  long long max_items;          // bound of the item buffers
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* block_table;   // [num_seqs, bt_stride], or null: packed keys
  int bt_stride;
  long long n_pages;
  const float* k_scale;         // fp8: [n_pages, hkv]
  const float* v_scale;
  const int32_t* visible;       // [total_q, mask_words] bits of the new tokens that a new token sees, or null: causal
  int mask_words;
  __nv_bfloat16* o;             // [total_q, hq, 128]
  float* lse;                   // [total_q, hq]
  float scale_log2;             // softmax scale * log2(e)
  // workspace
  WsHeader* hdr;
  PromptPlan* plan;
  SeqInfo* seq;                 // [num_seqs]
  int32_t* item_base;           // [num_seqs] items before a sequence's
  PromptItem* items;            // [max_items]
  int32_t* run_item;            // [kPromptMaxCtas] with runs: the item that each begins in
  long long* run_at;            // [kPromptMaxCtas + 1] and where, in units of cost; behind the last one the total
  // [ctas, 2, 2 tiles, 32, 128, 4] four dims of 128 rows each: slot 1 the item that goes on behind the run; null: never runs
  float* part_o;
  float2* part_ml;              // [ctas, 2, 2, 128] (reference, sum)
};
bool prompt_may_split(int max_nb);  // whether a call with so many key blocks can be cut into runs
struct PromptMaps {
  CUtensorMap q;     // boxes of a group's heads of tile_tokens tokens (64 dims in bf16, 128 codes in fp8)
  CUtensorMap k, v;  // boxes of 128 rows of a head (64 dims in bf16, 128 codes in fp8)
};
cudaError_t launch_prompt_attn(const PromptMaps& maps, const PromptParams& p, bool fp8, cudaStream_t stream);

// ---------------------------------------------------------------- filling a paged cache
struct ExtendParams {
  int num_seqs;
  const int32_t* lengths;       // [num_seqs] cached tokens
  const int32_t* new_tokens;    // [num_seqs]
  long long capacity;           // entries of slots and positions
  long long max_len;            // tokens that a row of the table can hold
  const int32_t* free_pages;    // [num_free]
  int num_free;
  long long n_pages;
  const int32_t* taken;         // free pages handed out before, or null: none
  int32_t* taken_out;
  int32_t* block_table;         // [num_seqs, bt_stride]
  int bt_stride;
  int32_t* new_lengths;         // [num_seqs] or null
  int32_t* cu_q;                // [num_seqs + 1]
  int32_t* cu_k;                // [num_seqs + 1]
  long long* slots;             // [capacity]
  int32_t* positions;           // [capacity]
  WsHeader* hdr;
  int32_t* page_base;           // [num_seqs] workspace: place in the free list of a sequence's first new page
};
cudaError_t launch_extend(const ExtendParams& p, int sms, cudaStream_t stream);

// One tensor of new rows and its cache.
struct AppendPlane {
  const __nv_bfloat16* x;  // [tokens] rows of `width`, `stride` elements apart
  long long stride;
  int width;
  void* cache;             // [n_pages * 128, width] bf16, or E4M3 codes with
  float* scale;            // [n_pages, width / 128]
};
struct AppendParams {
  AppendPlane plane[3];
  int planes;
  const long long* slots;  // [tokens], -1: no row
  long long tokens;
  long long n_pages;
  WsHeader* hdr;           // null (bf16): no flags
  uint32_t* marks;         // fp8: [n_pages] behind the header
};
cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream);
cudaError_t launch_append_fp8(const AppendParams& p, size_t clear_bytes, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- eviction
struct EvictParams {
  int num_seqs, hkv, max_k, total_k, budget, recent;
  int new_blocks;               // pages of the longest new sequence (bound)
  const int32_t* cu_k;
  void* k;                      // [n_pages * 128, hkv, 128] bf16, or E4M3 codes
  void* v;
  float* k_scale;               // fp8: [n_pages, hkv]
  float* v_scale;
  const int32_t* block_table;
  int bt_stride;
  const int32_t* new_table;
  int new_stride;
  long long n_pages;
  const float* weight;          // [num_seqs, hkv, weight_stride]
  long long weight_stride;
  float* new_weight;            // [num_seqs, hkv, new_weight_stride]
  long long new_weight_stride;
  int32_t* kept;                // [num_seqs, hkv, budget]
  int32_t* new_cu_k;            // [num_seqs + 1]
  WsHeader* hdr;
  uint32_t* marks;              // [n_pages] behind the header
  size_t clear_bytes;           // header and marks
};
cudaError_t launch_evict(const EvictParams& p, bool fp8, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- residual sum and norm
struct NormParams {
  long long rows;
  int width;
  float eps;
  const __nv_bfloat16* x;         // [rows, width]
  const __nv_bfloat16* residual;  // [rows, width] or null
  const __nv_bfloat16* gamma;     // [width]
  __nv_bfloat16* sum;             // [rows, width] or null
  __nv_bfloat16* y;               // [rows, width], or
  uint8_t* y8;                    // E4M3 codes with
  float* scale;                   // one scale per row
};
cudaError_t launch_add_rms_norm(const NormParams& p, int sms, cudaStream_t stream);

}  // namespace msa
