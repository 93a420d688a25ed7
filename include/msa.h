/*
 * msa.h -- C ABI of the MiniMax Sparse Attention (MSA) forward pass on GB300
 * (sm_103a).  Plain pointers and sizes only: no C++ or framework types cross
 * this boundary.
 *
 * The method ("MiniMax Sparse Attention: let each query pick its own blocks",
 * section "The mechanism, precisely", and the same page's Figure 1):
 *   Index Branch: per GQA group g, one index-query head; one index-key head
 *     shared by all groups.  For query i at key position pos(i):
 *       s[g,i,j] = Q_idx[i,g,:] . K_idx[j,:]             (fp32, j <= pos(i))
 *       P[g,i,b] = max over keys j of block b, j <= pos(i), of s[g,i,j]
 *       sel(i,g) = {local block pos(i)/B} U top-(k-1) of the other causal
 *                  blocks by (P descending, block index ascending)
 *   Main Branch: every query head h of group g attends, with exact softmax,
 *     to the tokens j <= pos(i) of the blocks in sel(i,g) only.
 * Deployed values: block B = 128, k = 16 (a 2,048-token budget per query);
 * 64 query heads over 4 KV heads, head dim 128 (the atlas record of the
 * report, summary paragraph).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Batches are packed variable-length sequences.  Sequence s owns query rows
 * [cu_seqlens_q[s], cu_seqlens_q[s+1]) and key rows [cu_seqlens_k[s],
 * cu_seqlens_k[s+1]).  Its queries are the LAST q_len positions of the
 * sequence: query t sits at key position pos = kv_len - q_len + t
 * (bottom-right causal alignment; a decode step is q_len = 1).  Query head h
 * belongs to group h / (num_q_heads / num_kv_heads).
 *
 * Tensors (all row-major and contiguous, all DEVICE memory of the current
 * CUDA device, owned by the caller):
 *   q      [total_q, num_q_heads,  head_dim]   bf16
 *   k, v   [total_k, num_kv_heads, head_dim]   bf16
 *   q_idx  [total_q, num_kv_heads, index_dim]  bf16
 *   k_idx  [total_k, index_dim]                bf16
 *   idx    [total_q, num_kv_heads, topk]       int32  selected blocks, ascending,
 *                                                     -1 padding at the tail
 *   o      [total_q, num_q_heads,  head_dim]   bf16
 *   lse    [total_q, num_q_heads]              fp32   natural-log sum of exp of the
 *                                                     scaled logits
 * Every tensor pointer must be 16-byte aligned; the workspace 256-byte aligned.
 *
 * Supported shapes: head_dim = 128, block_size = 128, index_dim in {64, 128},
 * 1 <= topk <= 64, num_kv_heads dividing 128, group size num_q_heads /
 * num_kv_heads a power of two in [8, 128], total_q < 2^25; decode batches
 * also need num_kv_heads <= 8.  Other values return MSA_ERR_UNSUPPORTED.
 *
 * Size of a prefill call: the workspace holds one partial output per (query,
 * group, selected block) until the combine, so it grows with total_q * topk:
 * about total_q * num_q_heads * topk * 264 bytes, plus total_k * num_kv_heads
 * * 256 bytes (an fp16 copy of V) and the schedule (msa_workspace_size gives
 * the exact figure).  At 64 query / 4 KV heads and topk 16 that is about 270 KB
 * per query row: 35 GB for a 131,072-query prefill, so one call on a 288 GB
 * GB300 takes up to roughly 1M query rows with nothing else resident.  Longer
 * prefills go in chunks of queries (each call's sequences with q_len <
 * kv_len: the queries are the last q_len positions), which select and attend
 * exactly as one call would.
 *
 * Execution: every call validates its arguments on the host, then enqueues
 * kernels on `stream` and returns without synchronising.  Nothing is
 * allocated or freed: the caller provides a workspace of at least
 * msa_workspace_size() bytes, which the call overwrites.  Two calls that run
 * at the same time must not share a workspace.  On any non-OK status nothing
 * has been enqueued, except MSA_ERR_CUDA, which reports a launch failure.
 * Errors that only the device can see (cu_seqlens that contradict the host
 * sizes, a kernel wait that timed out) make the kernels skip their work and
 * set flags that msa_read_device_status() returns.
 *
 * CUDA graphs: since a call neither allocates nor synchronises, it may be
 * enqueued on a stream that is being captured.  The graph keeps the pointers
 * and sizes of the captured call (its workspace and outputs included) and
 * reads the inputs' contents at each replay; the decode chain's dependent
 * launches become programmatic edges.  Make one call of each entry point
 * before the first capture (one-time driver look-ups happen on that call).
 * msa_read_device_status() synchronises and is not capturable.
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (NULL = the legacy default stream). */
typedef struct CUstream_st *msa_stream_t;

typedef enum msa_status {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = -1,  /* null pointer, negative size, inconsistent sizes */
  MSA_ERR_UNSUPPORTED = -2,  /* valid but outside the supported shapes above */
  MSA_ERR_ALIGNMENT = -3,    /* a pointer is not aligned as required */
  MSA_ERR_WORKSPACE = -4,    /* workspace missing or smaller than required */
  MSA_ERR_CUDA = -5,         /* a CUDA call or kernel launch failed */
  MSA_ERR_DEVICE = -6        /* no usable sm_103 device is current */
} msa_status_t;

/* Device-side error flags (msa_read_device_status). */
#define MSA_DEVICE_TIMEOUT 1u        /* a kernel wait exceeded its time limit */
#define MSA_DEVICE_BAD_SEQLENS 2u    /* cu_seqlens disagree with the host sizes */
#define MSA_DEVICE_BAD_INDEX 4u      /* a computed index failed its check (checked builds), or a block-table
                                        entry of a paged call named a page outside the cache (or, for
                                        msa_evict_paged, a page that it may not write) */

typedef struct msa_problem {
  int32_t num_seqs;              /* >= 1 */
  const int32_t *cu_seqlens_q;   /* device [num_seqs + 1], cu[0] = 0, nondecreasing */
  const int32_t *cu_seqlens_k;   /* device [num_seqs + 1], kv_len >= q_len per sequence */
  int32_t total_q;               /* = cu_seqlens_q[num_seqs] */
  int32_t total_k;               /* = cu_seqlens_k[num_seqs] */
  int32_t max_seqlen_q;          /* >= every q_len (host bound used for sizing) */
  int32_t max_seqlen_k;          /* >= every kv_len */
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;              /* 128 */
  int32_t index_dim;             /* 64 or 128 */
  int32_t block_size;            /* 128 */
  int32_t topk;                  /* 1..64, counts the local block */
  float softmax_scale;           /* <= 0 selects 1/sqrt(head_dim) */
} msa_problem_t;

typedef enum msa_op {
  MSA_OP_INDEX_POOL = 1,         /* msa_index_pool */
  MSA_OP_INDEX_TOPK = 2,         /* msa_index_topk */
  MSA_OP_SPARSE_ATTN_PREFILL = 3,/* msa_sparse_attn_prefill */
  MSA_OP_SPARSE_ATTN_DECODE = 4, /* msa_sparse_attn_decode */
  MSA_OP_FORWARD = 5,            /* msa_forward */
  MSA_OP_TOPK_POOLED = 6,        /* msa_topk_pooled */
  MSA_OP_QUANTIZE_KV_FP8 = 7,    /* msa_quantize_kv_fp8 */
  MSA_OP_SPARSE_ATTN_PREFILL_FP8 = 8, /* msa_sparse_attn_prefill_fp8 */
  MSA_OP_SPARSE_ATTN_DECODE_FP8 = 9,  /* msa_sparse_attn_decode_fp8 */
  MSA_OP_FORWARD_FP8 = 10,       /* msa_forward_fp8 */
  MSA_OP_INDEX_PROLOGUE = 11,    /* msa_index_prologue */
  MSA_OP_QUANTIZE_INDEX_FP8 = 12,/* msa_quantize_index_fp8 */
  MSA_OP_DENSE_ATTN_DECODE = 13, /* msa_dense_attn_decode_paged(_fp8), weight = NULL */
  MSA_OP_DENSE_ATTN_DECODE_WEIGHT = 14, /* the same with a weight */
  /* 15 is no operation */
  MSA_OP_DENSE_ATTN_PREFILL = 16, /* msa_dense_attn_prefill, msa_dense_attn_prefill_paged(_fp8) */
  MSA_OP_TREE_ATTN = 17          /* msa_tree_attn_paged(_fp8) */
} msa_op_t;

/* Workspace bytes that `op` needs for `problem` (host-only; no CUDA call).
 * Returns MSA_ERR_INVALID_ARG / MSA_ERR_UNSUPPORTED as the op itself would. */
msa_status_t msa_workspace_size(const msa_problem_t *problem, msa_op_t op, size_t *bytes);

/* Index Branch, scoring and pooling only ("The mechanism, precisely": scores
 * Q_idx . K_idx^T max-pooled to blocks).  Writes pooled[r * pooled_stride + b]
 * for query/group row r = i * num_kv_heads + g and causal block
 * b <= pos(i) / block_size (the local block pools only keys j <= pos(i));
 * entries past the causal end are left untouched.  pooled_stride >= the
 * largest number of causal blocks, ceil(max_seqlen_k / block_size). */
msa_status_t msa_index_pool(const msa_problem_t *problem, const void *q_idx, const void *k_idx,
                            float *pooled, int64_t pooled_stride, void *workspace,
                            size_t workspace_bytes, msa_stream_t stream);

/* Top-k over precomputed pooled rows (same layout as msa_index_pool), local
 * block forced in: idx[r][0..topk) = ascending set, -1 padded.  Ranking:
 * pooled score descending, equal scores to the lower block index, +0 == -0. */
msa_status_t msa_topk_pooled(const msa_problem_t *problem, const float *pooled,
                             int64_t pooled_stride, int32_t *idx, void *workspace,
                             size_t workspace_bytes, msa_stream_t stream);

/* Index Branch: scores, block max-pool and top-k with the local block forced
 * ("The mechanism, precisely", first bullet).  Writes idx.  Prefill batches
 * (max_seqlen_q > 1) use the tensor-core scoring kernel with the top-k fused
 * into its epilogue; decode batches (max_seqlen_q == 1) a streaming scan. */
msa_status_t msa_index_topk(const msa_problem_t *problem, const void *q_idx, const void *k_idx,
                            int32_t *idx, void *workspace, size_t workspace_bytes,
                            msa_stream_t stream);

/* Main Branch for prefill ("The mechanism, precisely", second bullet): exact
 * softmax attention over the blocks in idx (any ascending, -1 padded set that
 * contains only causal blocks; every row must contain at least one block).
 * Writes o and lse. */
msa_status_t msa_sparse_attn_prefill(const msa_problem_t *problem, const void *q, const void *k,
                                     const void *v, const int32_t *idx, void *o, float *lse,
                                     void *workspace, size_t workspace_bytes,
                                     msa_stream_t stream);

/* Main Branch for decode batches (every q_len == 1): "MiniMax Sparse
 * Attention: let each query pick its own blocks", section "The mechanism,
 * precisely", second bullet -- exact attention of the one new query of each
 * sequence (at pos = kv_len - 1) over the blocks in idx; the groundtruth.day
 * article on the llama.cpp merge ("Key facts") gives the effect: about 2,048
 * KV tokens read per decode step whatever the context length.  Split over the
 * selected blocks (one partial result per (sequence, group, block)), then a
 * log-sum-exp combine.  Same arguments and results as the prefill call. */
msa_status_t msa_sparse_attn_decode(const msa_problem_t *problem, const void *q, const void *k,
                                    const void *v, const int32_t *idx, void *o, float *lse,
                                    void *workspace, size_t workspace_bytes,
                                    msa_stream_t stream);

/* Size of the device array behind msa_sparse_attn_decode_static (32 MiB). */
#define MSA_STATIC_SCRATCH_BYTES (32u << 20)

/* msa_sparse_attn_decode for callers that cannot allocate device memory: no
 * workspace argument; the scratch lives in a fixed device array of
 * MSA_STATIC_SCRATCH_BYTES that this library declares (every GPU that loads
 * the library holds it until the process exits).  The method's pages have no
 * counterpart to this call; it exists for code that runs where cudaMalloc is
 * not available or not allowed -- a host framework that hands out only its
 * own pre-allocated tensors, an allocator-free serving loop, a process whose
 * memory pool is already fully reserved -- and that would otherwise have no
 * way to provide the workspace.
 * Arguments, layouts and results are those of msa_sparse_attn_decode.  The
 * call allocates and frees nothing.  Batches whose scratch would exceed the
 * array (about 120 decode sequences at 64 query / 4 KV heads and topk 16)
 * return MSA_ERR_WORKSPACE, and msa_last_error_detail() states the bytes
 * needed and available.  The first call on a device looks up the array's
 * device address (cudaGetSymbolAddress, with that device current) and caches
 * it; make that first call before any stream capture.  The cached address
 * belongs to the context it was looked up in: after a device reset (a new
 * primary context) the next call looks it up again.  Every call uses the
 * same array and leaves its contents behind (each call clears what must start
 * at zero), so calls whose kernels may overlap on the GPU -- on different
 * streams, or from several host threads -- race and must be serialised by the
 * caller.  Device-side errors of a call (MSA_DEVICE_* flags) are kept in the
 * array's header: read them with msa_read_device_status(NULL, ...). */
msa_status_t msa_sparse_attn_decode_static(const msa_problem_t *problem, const void *q,
                                           const void *k, const void *v, const int32_t *idx,
                                           void *o, float *lse, msa_stream_t stream);

/* The whole MSA layer forward ("MiniMax Sparse Attention: let each query pick
 * its own blocks", section "The mechanism, precisely", both bullets, and
 * Figure 1: Index Branch -> top-k block indices -> Main Branch):
 * msa_index_topk, then msa_sparse_attn_prefill, or msa_sparse_attn_decode when
 * every q_len is 1, on one workspace (size: op MSA_OP_FORWARD).  Writes idx
 * (the selection), o and lse. */
msa_status_t msa_forward(const msa_problem_t *problem, const void *q, const void *k,
                         const void *v, const void *q_idx, const void *k_idx, int32_t *idx,
                         void *o, float *lse, void *workspace, size_t workspace_bytes,
                         msa_stream_t stream);

/* msa_forward for a decode batch whose cache is paged: the same operation
 * ("MiniMax Sparse Attention: let each query pick its own blocks", section
 * "The mechanism, precisely": index scores over the cached keys, block
 * max-pool, top-k with the local block forced, exact attention over the
 * selected blocks), with K, V and K_idx read from pages of 128 tokens -- one
 * key block each -- instead of packed rows.  The pages describe no paged
 * layout; this is the decode call in the form a serving cache keeps it.
 *   problem     as for msa_forward, every sequence with q_len = 1;
 *               cu_seqlens_k gives the cached lengths (its offsets are not
 *               used as row positions here).
 *   k_cache, v_cache  [num_pages * 128, Hkv, 128] bf16; k_idx_cache
 *               [num_pages * 128, d_idx] bf16.  Row 128 * p + t of a cache is
 *               token t of page p.
 *   block_table int32 [num_seqs, max_blocks_per_seq], device: key block b of
 *               sequence s (tokens 128 b .. 128 b + 127) is page
 *               block_table[s * max_blocks_per_seq + b]; entries past a
 *               sequence's last block are not read.  4-byte aligned.
 *   max_blocks_per_seq  row stride of block_table; at least
 *               ceil(max_seqlen_k / 128).
 *   num_pages   pages in each cache; num_pages * 128 < 2^31.
 *   idx, o, lse, workspace, stream  as for msa_forward (workspace size: op
 *               MSA_OP_FORWARD of the same problem).
 * A block-table entry outside [0, num_pages) is not dereferenced: its block
 * reads as zeros and the workspace status gets MSA_DEVICE_BAD_INDEX (read it
 * with msa_read_device_status).  Host-side argument errors return before any
 * launch, as for msa_forward. */
msa_status_t msa_forward_decode_paged(const msa_problem_t *problem, const void *q, const void *k_cache,
                                      const void *v_cache, const void *q_idx, const void *k_idx_cache,
                                      const int32_t *block_table, int32_t max_blocks_per_seq,
                                      int64_t num_pages, int32_t *idx, void *o, float *lse,
                                      void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* Index prologue: hidden states -> index heads ("MiniMax Sparse Attention:
 * let each query pick its own blocks", Figure 1: the Index Branch takes the
 * hidden states through a linear projection, a norm and RoPE to the index
 * query and key heads; the atlas record gives d_model 3072 and a RoPE
 * dimension of 64 on 128-dim heads, and names no norm).  For every new token
 * (query row i at key position pos(i)):
 *   y_h = W_q[h] x_i (h < num_kv_heads), y_k = W_k x_i      (fp32 accumulation)
 *   z = y / sqrt(mean(y^2) + 1e-6) * gamma   per head (gamma_q for the index
 *       query heads, gamma_k for the key head)
 *   RoPE on dims 0..63: pairs (j, j + 32) rotated by pos(i) * 10000^(-j/32)
 *   Q_idx[i, h, :] = z_h;  K_idx[k_start + pos(i), :] = z_k   (bf16)
 * so a prefill writes its tokens' rows of the index-key cache and a decode
 * step appends one row per sequence.
 *   x        [total_q, d_model] bf16; d_model a multiple of 64 (at most 65536)
 *   w_q      [num_kv_heads * 128, d_model] bf16 (a linear layer's weight)
 *   w_k      [128, d_model] bf16
 *   gamma_q, gamma_k  [128] bf16
 *   q_idx    [total_q, num_kv_heads, 128] bf16 (written)
 *   k_idx    [total_k, 128] bf16 (the new tokens' rows written, others kept)
 * Needs index_dim = 128 (else MSA_ERR_UNSUPPORTED); workspace: op
 * MSA_OP_INDEX_PROLOGUE.  Pointers 16-byte aligned (gamma 2-byte). */
msa_status_t msa_index_prologue(const msa_problem_t *problem, const void *x, int32_t d_model, const void *w_q,
                                const void *w_k, const void *gamma_q, const void *gamma_k, void *q_idx,
                                void *k_idx, void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * fp8 K and V.  The atlas record of the report (provenance of section 4.2)
 * says the kernels handle fp8 as well and gives no format; this library reads
 * it as OCP E4M3 codes ("E4M3FN": bias 7, 3 mantissa bits, largest finite
 * 448, no infinities) with one fp32 scale per (key block of 128 tokens of a
 * sequence, KV head), for K and for V separately:
 *   scale = max |x| over the block's rows of that head / 448 (1 when 0),
 *   code  = round-to-nearest-even(x / scale) in fp32, saturated to +-448,
 *   value = code * scale.
 *   k8, v8            [total_k, num_kv_heads, 128] uint8 codes, 16-byte aligned
 *   k_scale, v_scale  [n_key_blocks, num_kv_heads] fp32, 4-byte aligned, where
 *                     n_key_blocks = sum over sequences of ceil(kv_len / 128)
 *                     (at most total_k / 128 + num_seqs); key block b of
 *                     sequence s is row (key blocks of sequences 0..s-1) + b.
 * The Index Branch reads bf16 Q_idx / K_idx here (a quantized index selects
 * other blocks; the fp8 index below is a separate option).  The fp8 Main
 * Branch computes exactly the bf16 one over the dequantized values
 * (value = code * scale); results differ from bf16 K/V by the quantization.
 * Decode reads the codes directly (half the K/V bytes); prefill widens them
 * once per call into exact 16-bit copies in the workspace.  A paged decode
 * cache (msa_forward_decode_paged_fp8) has one scale row per page instead:
 * k_scale / v_scale [num_pages, num_kv_heads]; msa_quantize_kv_fp8 produces
 * exactly that layout when given the page pool as one sequence of
 * num_pages * 128 keys (each page is then one key block).
 * ------------------------------------------------------------------------ */

/* bf16 K and V -> E4M3 codes and scales as above (msa_workspace_size op
 * MSA_OP_QUANTIZE_KV_FP8).  Only the rows of the sequences' key blocks are
 * written. */
msa_status_t msa_quantize_kv_fp8(const msa_problem_t *problem, const void *k, const void *v, void *k8, void *v8,
                                 float *k_scale, float *v_scale, void *workspace, size_t workspace_bytes,
                                 msa_stream_t stream);

/* msa_sparse_attn_prefill over fp8 K and V (op MSA_OP_SPARSE_ATTN_PREFILL_FP8). */
msa_status_t msa_sparse_attn_prefill_fp8(const msa_problem_t *problem, const void *q, const void *k8,
                                         const void *v8, const float *k_scale, const float *v_scale,
                                         const int32_t *idx, void *o, float *lse, void *workspace,
                                         size_t workspace_bytes, msa_stream_t stream);

/* msa_sparse_attn_decode over fp8 K and V (op MSA_OP_SPARSE_ATTN_DECODE_FP8). */
msa_status_t msa_sparse_attn_decode_fp8(const msa_problem_t *problem, const void *q, const void *k8,
                                        const void *v8, const float *k_scale, const float *v_scale,
                                        const int32_t *idx, void *o, float *lse, void *workspace,
                                        size_t workspace_bytes, msa_stream_t stream);

/* msa_forward with fp8 K and V for the Main Branch and bf16 Q_idx / K_idx for
 * the Index Branch (op MSA_OP_FORWARD_FP8). */
msa_status_t msa_forward_fp8(const msa_problem_t *problem, const void *q, const void *k8, const void *v8,
                             const float *k_scale, const float *v_scale, const void *q_idx, const void *k_idx,
                             int32_t *idx, void *o, float *lse, void *workspace, size_t workspace_bytes,
                             msa_stream_t stream);

/* msa_forward_decode_paged with fp8 K and V caches (op MSA_OP_FORWARD_FP8):
 * k8_cache, v8_cache [num_pages * 128, num_kv_heads, 128] E4M3 codes, and
 * k_scale, v_scale [num_pages, num_kv_heads] fp32, one row per page (see
 * above); the Index Branch reads the bf16 k_idx_cache as in
 * msa_forward_decode_paged.  Arguments, block table, errors and the device
 * flag for a page outside the cache as for msa_forward_decode_paged. */
msa_status_t msa_forward_decode_paged_fp8(const msa_problem_t *problem, const void *q, const void *k8_cache,
                                          const void *v8_cache, const float *k_scale, const float *v_scale,
                                          const void *q_idx, const void *k_idx_cache, const int32_t *block_table,
                                          int32_t max_blocks_per_seq, int64_t num_pages, int32_t *idx, void *o,
                                          float *lse, void *workspace, size_t workspace_bytes,
                                          msa_stream_t stream);

/* ------------------------------------------------------------------------
 * fp8 index (the same provenance as fp8 K/V above; the report also warns that
 * quantizing the index changes which blocks are selected, so this is an
 * option beside the bf16 Index Branch, and its selections are those of the
 * method applied to the dequantized index inputs, not to the bf16 ones).
 * Q_idx and K_idx as E4M3 codes (index_dim 128 only) with the rounding of
 * msa_quantize_kv_fp8 (scale = max |x| / 448, 1 when 0; code = RNE(x / scale)
 * in fp32, saturated):
 *   q_idx8       [total_q, num_kv_heads, 128] uint8, 16-byte aligned
 *   q_idx_scale  [total_q, num_kv_heads] fp32: one scale per (query row, group)
 *   k_idx8       [total_k, 128] uint8, 16-byte aligned
 *   k_idx_scale  [n_key_blocks] fp32: one scale per key block of 128 tokens of
 *                a sequence, block b of sequence s at row (key blocks of
 *                sequences 0..s-1) + b, as for k_scale above.
 * A token score is the fp32 dot product of the two code rows (the tensor
 * cores multiply E4M3 codes exactly and sum in fp32) and a block's pooled
 * score is the block's maximum times q_idx_scale * k_idx_scale: scales must be
 * positive and finite (msa_quantize_index_fp8 gives such), so the maximum of
 * the scaled scores is the scaled maximum.  Half the index bytes of bf16: the
 * decode index scan, which streams every cached key, reads half as much.
 * ------------------------------------------------------------------------ */

/* bf16 Q_idx and/or K_idx -> E4M3 codes and scales as above (workspace op
 * MSA_OP_QUANTIZE_INDEX_FP8).  Either input may be NULL to skip that side (for
 * example a decode step that quantizes only its new queries); the outputs of
 * a given side are then not touched.  Only the rows of the sequences' key
 * blocks are written. */
msa_status_t msa_quantize_index_fp8(const msa_problem_t *problem, const void *q_idx, const void *k_idx,
                                    void *q_idx8, float *q_idx_scale, void *k_idx8, float *k_idx_scale,
                                    void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* msa_index_pool over fp8 index inputs (workspace op MSA_OP_INDEX_POOL). */
msa_status_t msa_index_pool_fp8(const msa_problem_t *problem, const void *q_idx8, const float *q_idx_scale,
                                const void *k_idx8, const float *k_idx_scale, float *pooled,
                                int64_t pooled_stride, void *workspace, size_t workspace_bytes,
                                msa_stream_t stream);

/* msa_index_topk over fp8 index inputs (workspace op MSA_OP_INDEX_TOPK):
 * prefill and decode batches, the same selection rule. */
msa_status_t msa_index_topk_fp8(const msa_problem_t *problem, const void *q_idx8, const float *q_idx_scale,
                                const void *k_idx8, const float *k_idx_scale, int32_t *idx, void *workspace,
                                size_t workspace_bytes, msa_stream_t stream);

/* msa_forward_fp8 with the Index Branch on fp8 inputs as well (workspace op
 * MSA_OP_FORWARD_FP8): every K, V, Q_idx and K_idx read is an E4M3 code. */
msa_status_t msa_forward_fp8_index(const msa_problem_t *problem, const void *q, const void *k8, const void *v8,
                                   const float *k_scale, const float *v_scale, const void *q_idx8,
                                   const float *q_idx_scale, const void *k_idx8, const float *k_idx_scale,
                                   int32_t *idx, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                   msa_stream_t stream);

/* msa_forward_decode_paged_fp8 with the index-key cache in fp8 as well
 * (workspace op MSA_OP_FORWARD_FP8): k_idx8_cache [num_pages * 128, 128] E4M3
 * codes with k_idx_scale [num_pages], one scale per page (msa_quantize_index_fp8
 * gives that layout for the page pool taken as one sequence of num_pages * 128
 * keys), and q_idx8 / q_idx_scale for the batch's queries.  Block table,
 * errors and the device flag for a page outside the cache as for
 * msa_forward_decode_paged. */
msa_status_t msa_forward_decode_paged_fp8_index(const msa_problem_t *problem, const void *q, const void *k8_cache,
                                                const void *v8_cache, const float *k_scale, const float *v_scale,
                                                const void *q_idx8, const float *q_idx_scale,
                                                const void *k_idx8_cache, const float *k_idx_scale,
                                                const int32_t *block_table, int32_t max_blocks_per_seq,
                                                int64_t num_pages, int32_t *idx, void *o, float *lse,
                                                void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * The full-attention layers beside the sparse ones, over the same pages: the
 * dense attention of a decode step, eviction from a cache by the attention
 * weight its keys have received, and the residual sum and norm in front of a
 * layer's projections.
 *
 * msa_dense_attn_decode_paged: exact softmax attention of the one new query of
 * each sequence over ALL its cached keys.  For query head h of group g
 *   s[h,j] = softmax_scale * q_h . k_j,   lse_h = ln sum_j exp(s[h,j]),
 *   o_h = sum_j exp(s[h,j] - lse_h) v_j,
 * and, with a weight array, for every cached key j (in place)
 *   weight[g,j] += sum over the heads h of group g of exp(s[h,j] - lse_h).
 *   problem     a decode batch (max_seqlen_q = 1, total_q = num_seqs; query i
 *               is sequence i, cu_seqlens_q is not read).  cu_seqlens_k gives
 *               the cached lengths; a length of 0 is allowed (o = 0, lse =
 *               -inf).  index_dim and topk are not looked at.  head_dim =
 *               block_size = 128; any group size num_q_heads / num_kv_heads
 *               from 1 to 128, num_kv_heads <= 1024, num_seqs <= 2^20,
 *               max_seqlen_k <= 2^30, softmax_scale < 1e30.
 *   k_cache, v_cache, block_table, max_blocks_per_seq, num_pages
 *               as for msa_forward_decode_paged; what the rows past a
 *               sequence's last key hold does not matter.  Sequences may share
 *               pages.
 *   weight      fp32 [num_seqs, num_kv_heads, weight_stride], weight_stride >=
 *               max_seqlen_k, 4-byte aligned, or NULL.  Entries past a
 *               sequence's length are left as they were.  One thread adds the
 *               group's heads in order: the sums do not depend on timing.
 *   o, lse      written for every sequence.
 * Workspace: op MSA_OP_DENSE_ATTN_DECODE, or MSA_OP_DENSE_ATTN_DECODE_WEIGHT
 * with a weight (it then holds the logits: 4 bytes per query head and key).
 * Numbers.  A logit is an fp32 sum of the 128 products, times the factor; any
 * finite logit gives finite results (rows with logits of 710 and more round them
 * to fp32 before the maximum is taken off, and with a weight every row does).  A
 * logit of +inf gives NaN; keys of -inf do not count, and a head with no key that
 * counts has o = 0, lse = -inf.  What one head's query holds does not change
 * another head's results.  Exponentials are the hardware's 2^x (2^-22 of the
 * value).  Maximum, sum, O, lse and weight are fp32; a weight that meets V has 16
 * significant bits (bf16 V) or 11 (E4M3 V: fp16, full down to 2^-25 of the largest
 * weight times page scale).  E4M3 pages, groups of up to 32 heads: the query goes
 * to fp16 with a power of two per head, exact but for values 2^-24 below its
 * largest.  An inf or NaN in a key's row shows in the heads that meet the key.
 * Lengths that contradict the host sizes make the kernels skip the call
 * (MSA_DEVICE_BAD_SEQLENS); a page outside the cache reads as zeros
 * (MSA_DEVICE_BAD_INDEX).
 * ------------------------------------------------------------------------ */
msa_status_t msa_dense_attn_decode_paged(const msa_problem_t *problem, const void *q, const void *k_cache,
                                         const void *v_cache, const int32_t *block_table,
                                         int32_t max_blocks_per_seq, int64_t num_pages, float *weight,
                                         int64_t weight_stride, void *o, float *lse, void *workspace,
                                         size_t workspace_bytes, msa_stream_t stream);

/* The same over E4M3 pages with one scale per (page, KV head), positive and
 * finite, as for msa_forward_decode_paged_fp8: the attention over the
 * dequantized values. */
msa_status_t msa_dense_attn_decode_paged_fp8(const msa_problem_t *problem, const void *q, const void *k8_cache,
                                             const void *v8_cache, const float *k_scale, const float *v_scale,
                                             const int32_t *block_table, int32_t max_blocks_per_seq,
                                             int64_t num_pages, float *weight, int64_t weight_stride, void *o,
                                             float *lse, void *workspace, size_t workspace_bytes,
                                             msa_stream_t stream);

/* Workspace bytes of msa_evict_paged and msa_evict_paged_fp8 (host-only). */
msa_status_t msa_evict_workspace_size(const msa_problem_t *problem, int32_t budget, int64_t num_pages,
                                      size_t *bytes);

/* Eviction by accumulated weight.  Per sequence (n cached keys) and KV head: when
 * n <= budget every slot is kept; else the last `recent` slots (0 <= recent <=
 * budget, budget >= 1) and, of the others, the budget - recent with the
 * largest weight -- equal weights (-0 = +0) to the lower slot, NaN below every
 * number.  The kept slots of a head, in ascending order, become slots 0 ..
 * min(n, budget) - 1 of the sequence's pages in new_block_table: every sequence
 * of the call moves to its new pages (leave out of the batch what is to stay
 * where it is), and its old pages are the caller's to reuse.  The heads of a
 * page then hold different tokens at one slot, so a cache that is evicted from
 * serves dense attention, not the block selection of the sparse layers.
 *   problem, caches, block_table, num_pages   as above; the caches are read
 *               through block_table and written through new_block_table.
 *   weight      fp32 [num_seqs, num_kv_heads, weight_stride >= max_seqlen_k]
 *   new_block_table  int32 [num_seqs, new_max_blocks_per_seq], at least
 *               ceil(min(max_seqlen_k, budget) / 128) wide.  Its pages must be
 *               apart from those of block_table and named once: a page that is
 *               not, or that is outside the cache, is not written and raises
 *               MSA_DEVICE_BAD_INDEX (a page outside the cache in block_table
 *               reads as zeros and raises it too).
 *   kept        int32 [num_seqs, num_kv_heads, budget] (written): the kept slots,
 *               ascending, -1 at the tail.
 *   new_weight  fp32 [num_seqs, num_kv_heads, new_weight_stride >=
 *               min(max_seqlen_k, budget)] (written): the kept slots' weights;
 *               entries past the new length are left as they were.  Not `weight`.
 *   new_cu_seqlens_k  int32 [num_seqs + 1] (written): prefix sums of
 *               min(n, budget).  Not the problem's.
 * Rows of a new page past the new length are left as they were. */
msa_status_t msa_evict_paged(const msa_problem_t *problem, void *k_cache, void *v_cache, const int32_t *block_table,
                             int32_t max_blocks_per_seq, int64_t num_pages, const float *weight,
                             int64_t weight_stride, int32_t budget, int32_t recent, const int32_t *new_block_table,
                             int32_t new_max_blocks_per_seq, int32_t *kept, float *new_weight,
                             int64_t new_weight_stride, int32_t *new_cu_seqlens_k, void *workspace,
                             size_t workspace_bytes, msa_stream_t stream);

/* The same over E4M3 pages.  A page has one scale per KV head, so a new page's
 * rows are rounded again: value = code * scale of the page it came from, scale
 * = fp32(max |value| / 448) over the new page's rows (1, and codes 0, when the
 * largest is below 2^-118), code =
 * round-to-nearest-even of the exact value * 448 / max |value| (so a page that
 * keeps its largest value keeps its codes when that one's code is 448). */
msa_status_t msa_evict_paged_fp8(const msa_problem_t *problem, void *k8_cache, void *v8_cache, float *k_scale,
                                 float *v_scale, const int32_t *block_table, int32_t max_blocks_per_seq,
                                 int64_t num_pages, const float *weight, int64_t weight_stride, int32_t budget,
                                 int32_t recent, const int32_t *new_block_table, int32_t new_max_blocks_per_seq,
                                 int32_t *kept, float *new_weight, int64_t new_weight_stride,
                                 int32_t *new_cu_seqlens_k, void *workspace, size_t workspace_bytes,
                                 msa_stream_t stream);

/* Residual sum and root-mean-square norm, for each of `rows` rows of d_model
 * elements (1 .. 65536):
 *   h = x + residual   (fp32; residual = NULL: h = x),   sum = bf16(h),
 *   y = h / sqrt(mean(h^2) + eps) * gamma   (from h before its rounding, bf16)
 *   x, residual, sum, y  [rows, d_model] bf16, gamma [d_model] bf16, 16-byte
 *   aligned; sum may be NULL.  sum may be x or residual (in place), and y the
 *   other one; outputs must not overlap otherwise, nor in part.
 *   mean(h^2) is an fp32 sum: it passes fp32 where a row has values of about
 *   1e19 and more (y is then 0).
 * No workspace; rows = 0 is no work. */
msa_status_t msa_add_rms_norm(const void *x, const void *residual, const void *gamma, int64_t rows, int32_t d_model,
                              float eps, void *sum, void *y, msa_stream_t stream);

/* The same with y as E4M3 codes y8 [rows, d_model] (16-byte aligned) and one
 * scale per row y_scale [rows] (4-byte aligned): scale = max |y| / 448 (1 when
 * that is below 2^-120), code = round-to-nearest-even(y / scale) in fp32,
 * saturated. */
msa_status_t msa_add_rms_norm_fp8(const void *x, const void *residual, const void *gamma, int64_t rows,
                                  int32_t d_model, float eps, void *sum, void *y8, float *y_scale,
                                  msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Many new tokens at once, in the full-attention layers: prompts and chunks of
 * prompts, and trees of drafted tokens.
 *
 * msa_dense_attn_prefill: exact causal softmax attention.  For new token t of a
 * sequence (query row t, at position kv_len - q_len + t) and query head h of
 * group g, over the keys j <= kv_len - q_len + t:
 *   s[t,h,j] = softmax_scale * q_t,h . k_j,g,   lse = ln sum_j exp(s),
 *   o = sum_j exp(s - lse) v_j,g.
 *   problem     any packed batch: q_len <= kv_len per sequence, either may be 0;
 *               index_dim and topk are not looked at.  head_dim = block_size =
 *               128; any group size num_q_heads / num_kv_heads from 1 to 128,
 *               num_kv_heads <= 1024, num_seqs <= 2^20, total_q < 2^25,
 *               max_seqlen_k <= 2^30, softmax_scale < 1e30.
 *   q, k, v     packed, as in the conventions above.
 *   o, lse      written for every query row; o must not overlap q.
 * Workspace: op MSA_OP_DENSE_ATTN_PREFILL (42 MB and 40 bytes per pair of tiles of
 * 128 / group tokens).
 * Numbers.  Logits, references, sums, O and lse are fp32; a weight that meets V is
 * rounded to bf16 (2^-8 of the weight; E4M3 pages: fp16, 2^-11, down to 2^-21 of the
 * row's largest weight times page scale), the sum takes it unrounded.  Over E4M3
 * pages a query's values are two E4M3 codes each: exact down to 2^-10 of the row's
 * largest, 2^-18 of the largest below that.  Exponentials are the hardware's 2^x
 * (2^-22 of the value).  Any finite logit gives finite results; a logit of +inf gives
 * NaN, keys of -inf do not count.  A key that a query does not see does not count
 * whatever its K holds; an inf or NaN in V shows in the queries that see it, and can
 * show in those of the 2 floor(128 / group) + 126 places before it (382 for groups of
 * one head; in a tree: of the whole sequence).  What
 * one query row or sequence holds does not change another's results, and what lies
 * past a sequence's last key does not matter.  The same inputs give the same bits.
 * Lengths that contradict the host sizes make the kernels skip the call
 * (MSA_DEVICE_BAD_SEQLENS).
 * ------------------------------------------------------------------------ */
msa_status_t msa_dense_attn_prefill(const msa_problem_t *problem, const void *q, const void *k, const void *v,
                                    void *o, float *lse, void *workspace, size_t workspace_bytes,
                                    msa_stream_t stream);

/* The same over paged keys (the new tokens' rows are in the cache already, see
 * msa_append_paged): k_cache, v_cache, block_table, max_blocks_per_seq and
 * num_pages as for msa_dense_attn_decode_paged; a page outside the cache reads as
 * zeros (MSA_DEVICE_BAD_INDEX).  total_k may be more than cu_seqlens_k[num_seqs]:
 * a captured call whose total_k and max_seqlen_k are what the table has room for
 * follows a cache that grows from replay to replay (total_q is what it is). */
msa_status_t msa_dense_attn_prefill_paged(const msa_problem_t *problem, const void *q, const void *k_cache,
                                          const void *v_cache, const int32_t *block_table,
                                          int32_t max_blocks_per_seq, int64_t num_pages, void *o, float *lse,
                                          void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* The same over E4M3 pages with one scale per (page, KV head): the attention over
 * the dequantized values.  Scales of any size from 0 on, in any mixture.  A page of zeros
 * has a scale too (1, as msa_append_paged_fp8 writes it): beside much smaller scales of V
 * it can be the largest weight times page scale that the weights' 2^-21 is taken of. */
msa_status_t msa_dense_attn_prefill_paged_fp8(const msa_problem_t *problem, const void *q, const void *k8_cache,
                                              const void *v8_cache, const float *k_scale, const float *v_scale,
                                              const int32_t *block_table, int32_t max_blocks_per_seq,
                                              int64_t num_pages, void *o, float *lse, void *workspace,
                                              size_t workspace_bytes, msa_stream_t stream);

/* Attention of a tree of drafted tokens: the q_len new tokens of a sequence (the
 * drafts, in the cache's last q_len slots) see every cached key before them and,
 * of one another, what a mask says.
 *   visible     int32 [total_q, mask_words], mask_words >= ceil(max_seqlen_q /
 *               32), 4-byte aligned: bit d % 32 of word d / 32 of draft t's row is
 *               set when draft t sees draft d of its sequence (its ancestors and
 *               itself).  Bits from q_len on do not count.  A draft that sees no
 *               key at all has o = 0, lse = -inf.
 * Everything else as for msa_dense_attn_prefill_paged; workspace: op
 * MSA_OP_TREE_ATTN. */
msa_status_t msa_tree_attn_paged(const msa_problem_t *problem, const void *q, const void *k_cache,
                                 const void *v_cache, const int32_t *block_table, int32_t max_blocks_per_seq,
                                 int64_t num_pages, const int32_t *visible, int32_t mask_words, void *o, float *lse,
                                 void *workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_tree_attn_paged_fp8(const msa_problem_t *problem, const void *q, const void *k8_cache,
                                     const void *v8_cache, const float *k_scale, const float *v_scale,
                                     const int32_t *block_table, int32_t max_blocks_per_seq, int64_t num_pages,
                                     const int32_t *visible, int32_t mask_words, void *o, float *lse,
                                     void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* ------------------------------------------------------------------------
 * Filling a paged cache: tables from lengths, and the new tokens' rows.
 *
 * msa_extend_block_table: sequence s, of lengths[s] cached tokens, gets
 * new_tokens[s] more.  Its ceil((lengths + new) / 128) - ceil(lengths / 128) new
 * blocks take the next free pages, sequence by sequence:
 *   free_pages   int32 [num_free], the first *taken of which are gone (taken =
 *                NULL: none); *taken_out (may be taken) is what is gone behind the
 *                call.
 *   block_table  int32 [num_seqs, max_blocks_per_seq]: the new blocks' entries are
 *                written, the others left as they were.
 *   new_lengths  int32 [num_seqs] (may be lengths, or NULL): lengths + new.
 *   cu_seqlens_q, cu_seqlens_k  int32 [num_seqs + 1]: prefix sums of new_tokens and
 *                of lengths + new_tokens, as a problem of the grown cache has them.
 *   slots        int64 [capacity], 8-byte aligned: the cache row of each new token,
 *                sequence by sequence; -1 past the last one.
 *   positions    int32 [capacity]: its place in its sequence; 0 past the last one.
 *   num_pages    pages of the cache.  Tokens whose page is outside it (in the
 *                table's last old block or the free list), or for whose block the
 *                list has no page, get slots of -1, and such a new block's entry
 *                is -1 (MSA_DEVICE_BAD_INDEX).
 * Negative lengths, sequences that the table has no room for, *taken past the list
 * and more new tokens than `capacity` (or 2^31 keys) make the call do nothing but
 * fill slots with -1 and positions and prefix sums with 0
 * (MSA_DEVICE_BAD_SEQLENS).  num_seqs <= 2^20.  Workspace:
 * msa_extend_workspace_size.
 *
 * Taking tokens back (rejected drafts): lengths is the caller's to shorten, and a
 * block counts as held as long as ceil(lengths / 128) reaches it.  The pages of the
 * blocks behind that are then in no list; before the next call the caller puts the
 * n pages back (entries of -1 are none), in any order, where handed-out ones stood,
 * free_pages[*taken - n] to free_pages[*taken - 1], and lowers *taken by n.  Accepted drafts that do not lie
 * together (a path through a tree) are written again with msa_append_paged(_fp8):
 * their rows of k and v, at the step's first slots.  (A page's E4M3 scale that
 * rejected drafts have raised stays.) */
msa_status_t msa_extend_workspace_size(int32_t num_seqs, size_t *bytes);
msa_status_t msa_extend_block_table(int32_t num_seqs, const int32_t *lengths, const int32_t *new_tokens,
                                    int64_t capacity, const int32_t *free_pages, int32_t num_free,
                                    const int32_t *taken, int64_t num_pages, int32_t *block_table,
                                    int32_t max_blocks_per_seq, int32_t *new_lengths, int32_t *cu_seqlens_q,
                                    int32_t *cu_seqlens_k, int64_t *slots, int32_t *positions, int32_t *taken_out,
                                    void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* New tokens' rows into their slots: k_cache[slots[i]] = k[i] and so on.
 *   k, v       bf16 [tokens, num_kv_heads, 128], tokens k_stride (v_stride)
 *              elements apart: slices of a wider projection's output, say.
 *   k_idx      bf16 [tokens, index_dim] (k_idx_stride apart) with k_idx_cache, or
 *              NULL for both.  index_dim 64 or 128.  k, v and their caches may all be
 *              NULL: K_idx alone (bf16 index pages beside K and V in E4M3 pages, as
 *              msa_forward_decode_paged_fp8 reads them; num_kv_heads is not looked at).
 *   slots      int64 [tokens], 8-byte aligned, distinct; -1: the token has no row.
 *              Others outside the cache are skipped (MSA_DEVICE_BAD_INDEX).
 * Strides are multiples of 8 and at least a row; pointers 16-byte aligned.  workspace
 * may be NULL (no device flags) or has 256 bytes.  num_kv_heads <= 1024. */
msa_status_t msa_append_paged(const void *k, int64_t k_stride, const void *v, int64_t v_stride, const void *k_idx,
                              int64_t k_idx_stride, const int64_t *slots, int64_t tokens, int32_t num_kv_heads,
                              int32_t index_dim, void *k_cache, void *v_cache, void *k_idx_cache, int64_t num_pages,
                              void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* The same into E4M3 pages with one scale per (page, head) (k_idx8_cache with
 * k_idx_scale [num_pages], index_dim 128).  The tokens that follow one another into
 * one page -- a page's tokens have to, 128 at most -- are taken together: with L the
 * smallest row among them, the page's rows below L hold values already;
 *   scale' = max(scale if L > 0, fp32(max |new| / 448))   (1 when that is 0; a max
 *            |new| below 2^-118 counts as 0, inf and NaN do not count)
 *   code   = round-to-nearest-even, saturated, of the exact x * 448 / max |new| where
 *            the new rows set the scale, else of fp32(x / scale),
 * and where scale' > scale the codes of the rows below L become those of code * scale *
 * 448 / max |new| (two fp32 roundings).  Other rows are left as they
 * were.  A page that comes twice raises MSA_DEVICE_BAD_INDEX and its contents are
 * undefined.  tokens * num_kv_heads below 2^37.  Workspace:
 * msa_append_workspace_size. */
msa_status_t msa_append_workspace_size(int64_t num_pages, size_t *bytes);
msa_status_t msa_append_paged_fp8(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                  const void *k_idx, int64_t k_idx_stride, const int64_t *slots, int64_t tokens,
                                  int32_t num_kv_heads, void *k8_cache, void *v8_cache, float *k_scale,
                                  float *v_scale, void *k_idx8_cache, float *k_idx_scale, int64_t num_pages,
                                  void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* Waits for `stream`, then returns in *flags the MSA_DEVICE_* bits that the
 * last call on this workspace raised (0 = none).  workspace = NULL reads the
 * flags of the last msa_sparse_attn_decode_static call on the current device.
 * The only synchronising call. */
msa_status_t msa_read_device_status(const void *workspace, uint32_t *flags, msa_stream_t stream);

/* Stages of a call, for msa_set_stage_events. */
#define MSA_STAGE_PLAN 0      /* cu_seqlens validation, per-sequence facts, work lists */
#define MSA_STAGE_INDEX 1     /* index scores + block max-pool (+ fused top-k in prefill) */
#define MSA_STAGE_TOPK 2      /* top-k over pooled rows (decode, msa_topk_pooled) */
#define MSA_STAGE_SCHEDULE 3  /* inversion of the selection into per-block work items */
#define MSA_STAGE_ATTN 4      /* Main Branch partial attention */
#define MSA_STAGE_COMBINE 5   /* log-sum-exp merge of the partials into o and lse */
#define MSA_NUM_STAGES 6

/* Optional per-stage timing for the calling host thread.  `events` holds
 * 2 * MSA_NUM_STAGES cudaEvent_t handles created by the caller; while set,
 * every call records events[2*s] on its stream just before stage s and
 * events[2*s + 1] just after it (stages a call does not run are not
 * recorded).  Pass NULL to stop.  Recording adds no synchronisation. */
msa_status_t msa_set_stage_events(void *const *events);

/* Number of kernels this library has enqueued since the process started
 * (all host threads; memsets included).  A diagnostic for launch accounting. */
int64_t msa_kernel_launch_count(void);

/* For the calling host thread: a description of the CUDA failure behind the
 * last MSA_ERR_CUDA (stage and CUDA error name) -- or of the scratch shortfall
 * behind an MSA_ERR_WORKSPACE from msa_sparse_attn_decode_static -- or "". */
const char *msa_last_error_detail(void);

/* Static description of a status code. */
const char *msa_status_string(msa_status_t status);

/* ABI version of this header (bumped on incompatible changes). */
int32_t msa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
