/*
 * msa.h -- C ABI of a single-GPU (sm_103a) library for two-stage GQA
 * block-sparse attention, the "MiniMax Sparse Attention" block.
 *
 * Source of the method: the Atlas Cloud guide "MiniMax goes sparse: decoding
 * M3's attention from a single diagram" (Portuguese, Spanish and French
 * editions), section 1:
 *   Step 1 (index branch): each GQA group has one index query; block-level
 *     scores are formed from token keys pooled per fixed-size block; a top-k
 *     keeps a short list of KV blocks per layer and per group.
 *   Step 2 (sparse branch): every query head of a group attends, with ordinary
 *     softmax attention, over the real (uncompressed) K/V of the blocks its
 *     group selected.
 * Where the guide leaves a step open, this library fixes it as a parameter:
 *   - block size 64 tokens;
 *   - block summary key = mean of the block's 64 keys of the KV head itself
 *     (scoring it equals the block mean of the token scores);
 *   - group index query = sum of the group's query heads (decode) or of the
 *     tile's 64 tokens x group heads (prefill);
 *   - the block holding the newest token (decode) or the tile's diagonal block
 *     (prefill) is always kept and never scored;
 *   - top-k ties go to the lower block index.
 *
 * Conventions for every call:
 *   - Every pointer argument is a DEVICE pointer unless marked "host".
 *   - The caller owns and allocates every buffer (inputs, outputs, workspace);
 *     the library never allocates device memory and never synchronises the
 *     stream, except msa_read_device_status.
 *   - Calls are asynchronous on `stream`. Calls that share a workspace must be
 *     ordered on one stream; distinct workspaces make calls independent.
 *   - Argument errors are found on the host before any launch and return
 *     MSA_ERR_INVALID_ARG / MSA_ERR_UNSUPPORTED / MSA_ERR_WORKSPACE with no
 *     work queued. A failed launch returns MSA_ERR_CUDA.
 *   - Data-dependent errors (a page id outside [0, num_pages), a sequence
 *     length above the cache capacity) never fault: the kernel skips the access
 *     and sets a sticky status word in the workspace, read with
 *     msa_read_device_status.
 *   - Head dimension D = 128 and block size 64 are the only supported values.
 *   - Rows of k and v past a sequence's length (in a prefill: past its chunk's end) may
 *     hold anything, NaN and infinities among it.
 *   - q, out, k, v, their scales and the pooled keys are moved in 16-byte pieces (vector
 *     loads and stores, asynchronous and tensor-memory-access copies): their
 *     base addresses must be 16-byte aligned (MSA_ERR_INVALID_ARG otherwise).
 *
 * Layouts (row-major, innermost last):
 *   q (decode)   [batch, num_q_heads, 128]         KV dtype (bf16 for an e4m3 cache)
 *   q (prefill)  [n_q_tokens, num_q_heads, 128]    KV dtype
 *   KV contiguous  k, v: [batch, num_kv_heads, max_tokens, 128]
 *   KV paged       k, v: [num_pages, num_kv_heads, 64, 128], page_table
 *                  [batch, max_pages_per_seq] int32 (logical block -> page)
 *   pooled keys (same dtype as q), per (sequence, KV head) in logical block
 *   order for both cache layouts, so a unit's candidates are one run of rows:
 *     contiguous   [batch, num_kv_heads, max_tokens/64, 128]
 *     paged        [batch, num_kv_heads, max_pages_per_seq, 128]
 *   Query head j belongs to KV head j / G, G = num_q_heads / num_kv_heads.
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* msa_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum msa_status {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, inconsistent shapes */
  MSA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. head_dim != 128) */
  MSA_ERR_WORKSPACE = 3,     /* workspace null or smaller than msa_workspace_size */
  MSA_ERR_CUDA = 4,          /* a CUDA launch or API call failed */
  MSA_ERR_DEVICE_BOUNDS = 5, /* (device status) a page id or length was out of range */
  MSA_ERR_TIMEOUT = 6,       /* (device status) a bounded wait gave up */
  MSA_ERR_OUT_OF_PAGES = 7   /* (device status) too few free pages for the new tokens */
} msa_status;

/* MSA_DTYPE_E4M3: k and v hold 8-bit e4m3 codes (1 sign, 4 exponent, 3 mantissa
 * bits, largest value 448, no infinities) and every row of 128 (one head of one
 * token) has an fp32 scale >= 0 in k_scale / v_scale: element = code * scale.
 * q, out and the pooled keys of such a cache are bf16. Read by pooling,
 * selection, sparse and dense decode, the decode step and the prefill attention.
 * Scales past a sequence's length may hold anything, as rows may. */
typedef enum msa_dtype { MSA_DTYPE_F32 = 0, MSA_DTYPE_BF16 = 1, MSA_DTYPE_E4M3 = 2 } msa_dtype;
typedef enum msa_kv_layout { MSA_KV_CONTIGUOUS = 0, MSA_KV_PAGED = 1 } msa_kv_layout;

/* The block-scoring operator of Step 1.
 * MEAN_POOLED_KEYS: q_idx . pooled[b], the summary key being the mean of the
 *   block's keys of the KV head itself -- by linearity the block mean of the
 *   token scores q_idx . k_t.
 * TOKEN_MAX: the guide's Step 1 as drawn (§1, Step 1: token-level scores
 *   against a single index-key head shared by all groups, then a block max
 *   pool): max over the block's 64 tokens of q_idx . K_idx[t], with K_idx a
 *   caller-provided index-key cache passed in place of the summaries. */
typedef enum msa_score_mode { MSA_SCORE_MEAN_POOLED_KEYS = 0, MSA_SCORE_TOKEN_MAX = 1 } msa_score_mode;

/* Description of a KV cache. All pointers are device pointers. */
typedef struct msa_kv_desc {
  int32_t layout;            /* msa_kv_layout */
  int32_t dtype;             /* msa_dtype of k and v; q, pooled keys and outputs: the same, bf16 for e4m3 */
  int32_t batch;             /* number of sequences */
  int32_t num_kv_heads;      /* Hkv */
  int32_t head_dim;          /* must be 128 */
  int32_t block_size;        /* must be 64 */
  const void* k;             /* keys, layout above */
  const void* v;             /* values, same layout as k */
  int64_t max_tokens;        /* contiguous: token capacity per sequence, a multiple of 64 */
  const int32_t* page_table; /* paged: [batch, max_pages_per_seq] */
  int32_t max_pages_per_seq; /* paged */
  int32_t num_pages;         /* paged: number of pages in k and v */
  const int32_t* seq_lens;   /* [batch] tokens present per sequence (device) */
  const float* k_scale;      /* e4m3 only (not read otherwise): the scale of every row of k, ... */
  const float* v_scale;      /* ... and of v: contiguous [batch, Hkv, max_tokens], paged [num_pages, Hkv, 64] */
} msa_kv_desc;

/* Rows of 128 elements for every (token, head): element d of head h of token t
 * is data[t * token_stride + h * head_stride + d] (strides in elements). data
 * is 16-byte aligned and the strides are whole multiples of 16 bytes. */
typedef struct msa_rows {
  const void* data;
  int64_t token_stride;
  int64_t head_stride;
} msa_rows;

/* Per-head norm and rotation of msa_qk_norm_rope_append. */
typedef struct msa_norm_rope_cfg {
  int32_t norm;        /* bit 0 (1): normalise the queries; bit 1 (2): the keys */
  int32_t rotary_dim;  /* leading dims of a head that are rotated: 0, 16, 32, ... 128 */
  int32_t interleaved; /* 0: pairs (i, i + rotary_dim/2); 1: pairs (2i, 2i + 1) */
  float eps;           /* added to the mean square, >= 0 */
  float weight_offset; /* norm weights enter as weight_offset + w (0 or 1 in use; any finite value) */
} msa_norm_rope_cfg;

/* Step-1 selection parameters. */
typedef struct msa_select_cfg {
  int32_t k_scored;    /* number of scored blocks to keep per unit, >= 0 */
  int32_t force_local; /* bit 0 (1): always keep the newest / diagonal block; bit 1 (2): always keep
                          block 0, an attention sink (guide §2 names a sink among the likely
                          replacements of the sliding window). Kept blocks are not scored. */
  int32_t q_tile;      /* 1: decode (one token per sequence); 64: prefill tiles */
  int32_t mode;        /* msa_score_mode */
  int64_t q_start;     /* prefill: absolute position of the first query token (any position) */
} msa_select_cfg;

/* Operation ids for msa_workspace_size. */
typedef enum msa_op {
  MSA_OP_POOL = 0,
  MSA_OP_SELECT = 1,         /* msa_select_topk_blocks with q_tile 1 (decode) */
  MSA_OP_DECODE = 2,
  MSA_OP_PREFILL = 3,
  MSA_OP_DENSE_DECODE = 4,
  MSA_OP_DENSE_PREFILL = 5,
  MSA_OP_SELECT_PREFILL = 6, /* msa_select_topk_blocks with q_tile 64 (n_q_tokens =
                                the chunk's tokens), and
                                msa_select_topk_blocks_varlen with n_q_tokens =
                                64 * the batch's query tiles (see
                                msa_select_topk_blocks_varlen) */
  MSA_OP_DECODE_STEP = 7,    /* msa_sparse_decode_step */
  MSA_OP_EXTEND = 8,         /* msa_extend_sequences */
  MSA_OP_TRIM = 9,           /* msa_trim_sequences */
  MSA_OP_APPEND = 10         /* msa_qk_norm_rope_append */
} msa_op;

/* Bytes of workspace `op` needs for these shapes (host call, no GPU work).
 * n_q_tokens is 1 for decode ops; k_total is the index-list length (ignored by
 * dense ops). Returns 0 when the arguments are invalid. A workspace must be
 * zero-filled once before its first use (msa_workspace_init); the library
 * leaves it ready for the next call. One workspace of the largest size serves
 * every op. */
size_t msa_workspace_size(int32_t op, const msa_kv_desc* kv /* host */, int32_t num_q_heads,
                          int32_t n_q_tokens, int32_t k_total);

/* Zero-fill `bytes` of workspace on `stream` (a memset; no allocation). */
msa_status msa_workspace_init(void* ws, size_t bytes, msa_stream_t stream);

/* Step 1a -- block summary keys (guide §1, Step 1, block pooling of the index
 * branch). For every complete block b (64 b + 63 < seq_len) of every
 * (sequence, KV head) with first_block <= b < first_block + n_blocks
 * (n_blocks = -1: all), writes pooled[b] = (1/64) * sum_{i<64} K[64 b + i]:
 * fp32 sum in row order, one multiply by 1/64, rounded to nearest even into
 * the KV dtype (bf16 for e4m3 rows, each code times its scale). Partial blocks are left untouched. Bad page ids set
 * MSA_ERR_DEVICE_BOUNDS in the status word when `ws` is given (ws may be NULL:
 * then bad pages are skipped silently); a skipped block's summary is not
 * written, the selection scores whatever that row holds, and the attention
 * reports the page again when the block is selected. */
msa_status msa_pool_block_keys(const msa_kv_desc* kv /* host */, int64_t first_block, int64_t n_blocks,
                               void* pooled, void* ws, size_t ws_bytes, msa_stream_t stream);

/* Step 1b/1c -- group index query, block scores and top-k (guide §1, Step 1:
 * one index query per GQA group, scores per block, TopK keeps the k best
 * blocks per layer and group).
 * Decode (cfg->q_tile == 1): q [batch, Hq, 128]; unit = (sequence, KV head);
 *   q_idx = sum of the group's G query heads (fp32); candidates are the
 *   complete blocks, minus the newest block nb-1 (nb = ceil(seq_len/64)) when
 *   force_local. Output idx_out [batch, Hkv, k_total].
 * Prefill (cfg->q_tile == 64, batch 1, contiguous or paged cache): q [n_q_tokens, Hq, 128] at
 *   absolute positions cfg->q_start + r (any q_start). The chunk's query
 *   tiles are its tokens grouped by the 64-token block they sit in: tile j
 *   holds the tokens whose position is in block q_start/64 + j (its diagonal
 *   block), so a chunk that starts inside a block has a shorter first tile;
 *   there are n_tiles = (q_start + n_q_tokens - 1)/64 - q_start/64 + 1 tiles.
 *   Unit = (tile j, KV head); q_idx = sum over the tile's tokens and the
 *   group's heads; candidates are the blocks before the diagonal block.
 *   Output idx_out [n_tiles, Hkv, k_total].
 * Scores are q_idx . pooled[b] in fp32 (unscaled). The top min(k_scored, n)
 * candidates by (score descending, block ascending) plus the forced block are
 * written sorted ascending, padded with -1;
 * k_total >= min(k_scored, max_blocks) + the number of kept blocks (bits of
 * force_local), and, as in every call with lists, <= 2^30 (MSA_ERR_UNSUPPORTED above). With the sink bit, block 0 leads the list and the candidates
 * start at block 1.
 * scores_out (nullable): [units, max_blocks] fp32 raw scores of the candidate
 * blocks (max_blocks = max_tokens/64 or max_pages_per_seq); other entries are
 * left unspecified.
 * cfg->mode == MSA_SCORE_TOKEN_MAX (bf16 or e4m3, Hkv <= 8; else
 *   MSA_ERR_UNSUPPORTED): `pooled` is the index-key cache instead, bf16, one shared
 *   head laid out like one KV head of the cache -- contiguous
 *   [batch, max_tokens, 128], paged [num_pages, 64, 128] on the cache's pages
 *   -- and the score of block b is max_{t in b} q_idx . K_idx[t] (fp32), for
 *   decode and for prefill tiles alike. The index keys of a sequence are read
 *   once for all of its KV heads (decode) or once per group of 16 tiles
 *   (prefill). */
msa_status msa_select_topk_blocks(const void* q, int32_t num_q_heads, int32_t n_q_tokens,
                                  const void* pooled, const msa_kv_desc* kv /* host */,
                                  const msa_select_cfg* cfg /* host */, int32_t* idx_out, int32_t k_total,
                                  float* scores_out, void* ws, size_t ws_bytes, msa_stream_t stream);

/* Step 1b/1c for a batch of chunks (guide §1, Step 1, applied to the prefill
 * chunk of every sequence of a batch at once): sequence s (n_seqs ==
 * kv->batch, at most 64) has q_counts[s] >= 0 new tokens at absolute positions
 * q_starts[s] + r (q_starts[s] + q_counts[s] within the sequence's capacity;
 * both arrays on the host). q holds the sequences' tokens back to back:
 * [sum q_counts, Hq, 128], sequence s from row q_off[s] = q_counts[0] + ... +
 * q_counts[s-1]. Its query tiles (tokens grouped by the 64-token block they sit
 * in, as for msa_select_topk_blocks: n_s = (q_starts[s] + q_counts[s] - 1)/64 -
 * q_starts[s]/64 + 1 tiles, none for an empty chunk) are numbered globally in
 * the same order (tile_off[s] + j), and idx_out [total tiles, Hkv, k_total]
 * gets, for global tile
 * tile_off[s] + j, exactly what msa_select_topk_blocks (q_tile 64, q_start =
 * q_starts[s]) gives for tile j of sequence s alone, scored against sequence
 * s's summaries (pooled [batch, Hkv, max_blocks, 128]; in token-max mode the
 * index-key cache). cfg->q_tile must be
 * 64 (cfg->q_start is ignored); fp32 caches take one sequence only
 * (MSA_ERR_UNSUPPORTED above). A batch with no new tokens queues nothing. */
msa_status msa_select_topk_blocks_varlen(const void* q, int32_t num_q_heads, int32_t n_seqs,
                                         const int64_t* q_starts /* host */, const int32_t* q_counts /* host */,
                                         const void* pooled, const msa_kv_desc* kv /* host */,
                                         const msa_select_cfg* cfg /* host */, int32_t* idx_out, int32_t k_total,
                                         float* scores_out, void* ws, size_t ws_bytes, msa_stream_t stream);

/* Step 2, decode (guide §1, Step 2: attention over the gathered selected
 * blocks; all heads of a group share the group's list).
 * For each sequence s and query head j (KV head h = j / G):
 *   o = sum_t softmax_t(scale * q_j . K[t]) V[t]
 * over the tokens t < seq_len[s] of the blocks idx[s, h, 0..k_total) (-1
 * entries ignored; duplicates are not allowed; bf16 caches: lists of up to 8192
 * entries always fit, a longer one is dealt in at most 16 equal runs, each of which
 * is cut after 512 valid blocks, and the device status records
 * MSA_ERR_UNSUPPORTED; e4m3 caches: batch * Hkv * k_total < 2^31 - 1,
 * MSA_ERR_UNSUPPORTED otherwise); batch * Hkv <= 16384 units
 * (MSA_ERR_UNSUPPORTED above). out [batch, Hq, 128] in q's dtype; lse (nullable)
 * [batch, Hq] fp32 natural-log sum of exp(scale q.k).
 * An empty selection gives out = 0 and lse = -inf; a NaN among a row's scores gives NaN
 * in both (in a prefill alike). */
msa_status msa_sparse_attn_decode(const void* q, int32_t num_q_heads, const msa_kv_desc* kv /* host */,
                                  const int32_t* idx, int32_t k_total, float scale, void* out,
                                  float* lse, void* ws, size_t ws_bytes, msa_stream_t stream);

/* Step 2, chunked prefill (guide §1, Step 2, and §3: during prefill the
 * savings fall on the main attention). Batch 1, bf16 or e4m3, contiguous or paged
 * cache (q_start + n_q_tokens within its capacity, any q_start); query token r
 * sits at absolute position p = q_start + r and attends to the tokens t <= p
 * of the blocks idx[p / 64 - q_start / 64, h, :] (its tile's list, idx from
 * msa_select_topk_blocks with q_tile 64).
 * At most 512 entries of a list may be valid blocks (-1 padding is free); a
 * longer list is cut there and the device status records MSA_ERR_UNSUPPORTED.
 * The rows of the chunk's own tokens have to be finite: a later token's key and
 * scales do not reach an earlier query, but a NaN or an infinity among its values
 * may, in the block that both lie in. kv->seq_lens is not read: the tokens up to the
 * chunk's end are taken as present, whether the lengths count them yet or not.
 * e4m3: the weight of a token (its softmax weight times its V scale) is rounded to 11
 * bits, or, where it is small against the row's largest, to a multiple of a fixed fraction of
 * that, such that the roundings of all small weights of a row add up to at most 2^-12 of the
 * largest (rows of up to 2^28 tokens); V scales may be as large as 2^80 (where a larger one leaves
 * a row's sum too small to be sure of, the device status records MSA_ERR_UNSUPPORTED). For every cache type the output is summed in fp32 on
 * the tensor cores, where a token whose share of a dim is below 2^-23 of that dim's sum so far
 * may be cut off.
 * out [n_q_tokens, Hq, 128] KV dtype (e4m3: bf16); lse (nullable) [n_q_tokens, Hq] fp32. */
msa_status msa_sparse_attn_prefill(const void* q, int32_t num_q_heads, int32_t n_q_tokens, int64_t q_start,
                                   const msa_kv_desc* kv /* host */, const int32_t* idx, int32_t k_total,
                                   float scale, void* out, float* lse, void* ws, size_t ws_bytes,
                                   msa_stream_t stream);

/* Step 2 for a batch of chunks: msa_sparse_attn_prefill for every sequence s
 * of the cache (n_seqs == kv->batch, at most 64) at once, in one launch. The
 * sequences, q, out and lse are laid out as for msa_select_topk_blocks_varlen:
 * tokens back to back (out [sum q_counts, Hq, 128], lse [sum q_counts, Hq]),
 * idx [total tiles, Hkv, k_total] with global tile numbers; token r of
 * sequence s sits at absolute position q_starts[s] + r and attends to the
 * tokens t <= that position of sequence s's listed blocks. Results equal those
 * of msa_sparse_attn_prefill on each sequence alone. */
msa_status msa_sparse_attn_prefill_varlen(const void* q, int32_t num_q_heads, int32_t n_seqs,
                                          const int64_t* q_starts /* host */, const int32_t* q_counts /* host */,
                                          const msa_kv_desc* kv /* host */, const int32_t* idx, int32_t k_total,
                                          float scale, void* out, float* lse, void* ws, size_t ws_bytes,
                                          msa_stream_t stream);

/* One whole decode step (guide §1, Step 1 then Step 2): the index lists of
 * msa_select_topk_blocks (decode, cfg->q_tile == 1) written to idx_out, and
 * the attention of msa_sparse_attn_decode over them written to out / lse,
 * with the same results. For a bf16 or e4m3 cache with k_scored <= 64 it runs as one
 * kernel (for a paged cache, when the step's grid fits one wave of the
 * device): one thread-block cluster per (sequence, KV head) scores the
 * summaries, selects and attends, exchanging the lists and the partial
 * results through distributed shared memory (nothing round-trips through the
 * workspace); otherwise it launches the two kernels in turn. In token-max mode
 * (cfg->mode, pooled = the index-key cache, Hkv <= 8) the token scores are
 * written to the workspace by their own kernel first and the cluster kernel
 * selects and attends on them. ws must hold
 * msa_workspace_size(MSA_OP_DECODE_STEP, ...) bytes. */
msa_status msa_sparse_decode_step(const void* q, int32_t num_q_heads, const void* pooled,
                                  const msa_kv_desc* kv /* host */, const msa_select_cfg* cfg /* host */,
                                  int32_t* idx_out, int32_t k_total, float scale, void* out, float* lse, void* ws,
                                  size_t ws_bytes, msa_stream_t stream);

/* The decode step of a generation loop (guide, introduction: decode writes the
 * output token by token, each new token checked against everything before
 * it; the summaries of Step 1 must keep up as blocks fill). Same as
 * msa_sparse_decode_step
 * (cfg->mode must be MSA_SCORE_MEAN_POOLED_KEYS), and `pooled` is also
 * written: for every (sequence, KV head) whose seq_len is a multiple of 64 --
 * its newest block has just filled with the current token -- the summary of
 * that block is written exactly as msa_pool_block_keys would, so the next step
 * (one token longer) can score it. In the fused kernel an otherwise idle warp
 * of the unit's first CTA does this while the attention runs; otherwise one
 * small pooling launch follows the step. No other summary is touched. */
msa_status msa_sparse_decode_step_pool(const void* q, int32_t num_q_heads, void* pooled,
                                       const msa_kv_desc* kv /* host */, const msa_select_cfg* cfg /* host */,
                                       int32_t* idx_out, int32_t k_total, float scale, void* out, float* lse,
                                       void* ws, size_t ws_bytes, msa_stream_t stream);

/* Dense causal GQA decode: the full-attention comparator (guide §3 quotes
 * the sparse speed-ups against full attention). Same as msa_sparse_attn_decode
 * with every block 0..ceil(seq_len/64)-1 selected. */
msa_status msa_dense_gqa_decode(const void* q, int32_t num_q_heads, const msa_kv_desc* kv /* host */,
                                float scale, void* out, float* lse, void* ws, size_t ws_bytes,
                                msa_stream_t stream);

/* Dense causal GQA prefill: msa_sparse_attn_prefill with every block up to the
 * diagonal selected for every tile. */
msa_status msa_dense_gqa_prefill(const void* q, int32_t num_q_heads, int32_t n_q_tokens, int64_t q_start,
                                 const msa_kv_desc* kv /* host */, float scale, void* out, float* lse,
                                 void* ws, size_t ws_bytes, msa_stream_t stream);

/* msa_sparse_attn_decode without a workspace argument, for callers that
 * cannot allocate device memory (an engine or plugin host that owns every
 * allocation, or a serving loop that must not call cudaMalloc/cudaFree once
 * running, since those can synchronise the device). The guide has no
 * counterpart to this call; it only changes where the split-K scratch lives.
 * Same arguments, layouts and results as msa_sparse_attn_decode, minus ws.
 *  - Scratch: a fixed 4 MiB device array inside this library, held by every
 *    GPU that loads it until the process exits. bf16 caches combine their
 *    splits inside a thread-block cluster and use none of it beyond a 256-byte
 *    header. fp32 and e4m3 caches keep split-K tickets and partial results there: a
 *    shape whose msa_workspace_size(MSA_OP_DECODE, ...) exceeds 4 MiB (fp32
 *    alone can) is rejected with MSA_ERR_WORKSPACE before any work is queued.
 *  - The first call on a device looks up the array's device address (a
 *    one-time set-up per device, cached for the life of the process); make
 *    that first call before any stream capture, and do not call this entry
 *    on a device after cudaDeviceReset (the cached address is then stale).
 *  - Every call on a device shares the one array and (fp32, e4m3) clears its
 *    counters at the start (a memset on `stream`): calls whose work overlaps
 *    on the GPU race; order them on one stream.
 *  - No device memory is allocated or freed. There is no status word:
 *    data-dependent errors (bad page ids, lengths above capacity) are skipped
 *    and a bounded wait that gives up leaves its output incomplete, neither
 *    reported. Use msa_sparse_attn_decode where those must be detected. */
msa_status msa_sparse_attn_decode_noalloc(const void* q, int32_t num_q_heads, const msa_kv_desc* kv /* host */,
                                          const int32_t* idx, int32_t k_total, float scale, void* out, float* lse,
                                          msa_stream_t stream);

/* The new tokens of a step find their place (the guide has no counterpart: its
 * cache is there already). Sequence s of the batch holds n_s = kv->seq_lens[s]
 * tokens and receives q_counts[s] >= 0 more (device array; 1 for a decode step,
 * a chunk's tokens for a prefill, 0 for none):
 *  - paged: every block it newly reaches gets a page from the top of the stack
 *    free_pages[0 .. *free_count) (device; the array has room for num_pages
 *    entries): the j-th new block, counted over the sequences in order and a
 *    sequence's blocks ascending, gets free_pages[*free_count - 1 - j]; it is
 *    written to page_table (normally kv->page_table itself), and
 *    *free_count_out is what is left. Contiguous caches ignore page_table and
 *    the three free-list arguments (NULL is fine).
 *  - seq_lens_out[s] = n_s + q_counts[s].
 *  - q_off [batch + 1]: the first row of each sequence's new tokens, which lie
 *    back to back: token r of s is row q_off[s] + r; q_off[batch] is their
 *    number. The decode calls take row s of q for sequence s: with one token each
 *    these rows are that; otherwise gather the rows q_off[s + 1] - 1.
 *  - positions [n_slots] int32: n_s + r for that row; slots [n_slots] int64: its
 *    cache slot, page * 64 + offset (paged) or s * max_tokens + position
 *    (contiguous), what msa_qk_norm_rope_append takes. n_slots is the row count
 *    of a padded step: rows from q_off[batch] on get position 0 and slot -1.
 * seq_lens_out may be kv->seq_lens and free_count_out may be free_count (the step
 * then happens in place); no other overlap is allowed. batch <= 8192
 * (MSA_ERR_UNSUPPORTED above).
 * All or nothing: when a length or count is negative or ends past the
 * capacity (or past 2^31 - 1 tokens), when the tokens exceed n_slots, or
 * *free_count is not in [0, num_pages], the device status gets
 * MSA_ERR_DEVICE_BOUNDS; when the stack holds too few pages,
 * MSA_ERR_OUT_OF_PAGES; then no sequence grows: lengths and count are copied,
 * q_off is all 0, slots all -1, and page_table and the stack are untouched. A
 * page id outside [0, num_pages) (on the stack, or in the table at a block
 * that is filled further) sets MSA_ERR_DEVICE_BOUNDS and its tokens get slot
 * -1, a new block's table entry -1.
 * ws: msa_workspace_size(MSA_OP_EXTEND, ...) bytes. */
msa_status msa_extend_sequences(const msa_kv_desc* kv /* host */, const int32_t* q_counts, const int32_t* free_pages,
                                const int32_t* free_count, int32_t n_slots, int32_t* page_table,
                                int32_t* seq_lens_out, int32_t* free_count_out, int32_t* q_off, int32_t* positions,
                                int64_t* slots, void* ws, size_t ws_bytes, msa_stream_t stream);

/* The inverse: sequences shrink -- to 0 when a request is finished, to an
 * earlier length when drafted tokens are rejected -- and return their pages.
 * seq_lens_out[s] = min(n_s, keep_lens[s]) with keep_lens [batch] (device) >= 0
 * (a value of n_s or more keeps the sequence). Paged: the pages of the blocks
 * past the new length, over the sequences in order and a sequence's blocks
 * ascending, are pushed on the stack: the j-th to free_pages[*free_count + j];
 * *free_count_out is the new height. Pages must belong to one sequence
 * only (a shared one would be pushed twice). The page table is left as it is:
 * its entries past a sequence's length (or its chunk's end) are not read by any call. In place use
 * and contiguous caches as for msa_extend_sequences; batch <= 8192.
 * All or nothing: a negative value, a length past the capacity, or a stack
 * that would exceed num_pages entries sets MSA_ERR_DEVICE_BOUNDS, lengths and
 * count are copied and nothing is pushed. A page id out of range is pushed as
 * -1 and sets MSA_ERR_DEVICE_BOUNDS.
 * ws: msa_workspace_size(MSA_OP_TRIM, ...) bytes. */
msa_status msa_trim_sequences(const msa_kv_desc* kv /* host */, const int32_t* keep_lens, int32_t* free_pages,
                              const int32_t* free_count, int32_t* seq_lens_out, int32_t* free_count_out, void* ws,
                              size_t ws_bytes, msa_stream_t stream);

/* The new tokens' queries, keys and values on their way from the projections to
 * the attention and the cache, in one pass. For token t and each query head
 * and key head x (128 elements, fp32 arithmetic, one rounding at the end):
 *   y = x / sqrt(mean(x^2) + eps) * (weight_offset + w)     where cfg->norm asks
 *   (a, b) -> (a cos - b sin, b cos + a sin), angle positions[t] * inv_freq[i],
 *   for the pairs i < rotary_dim/2 of the head's leading rotary_dim dims
 *   (cfg->interleaved says which two elements pair i holds).
 * Angles are exact to 2^-24 of half a turn at any position and for any finite inv_freq.
 * Query heads go to q_out, key
 * heads and value heads (unchanged) to the cache rows of slots[t]: row
 * slot % W of head h of run slot / W, W = max_tokens (contiguous; the run is the
 * sequence) or 64 (paged; the page). An e4m3 cache gets, per row, scale =
 * max(max|y|, 2^-100) / 448 and code = y * (448 / max(max|y|, 2^-100)) rounded
 * to nearest even; NaN stays NaN, a row with an infinity reads as NaN.
 *  - q, k, v, q_out: [n_tokens, heads, 128] rows with strides, e.g. views of one
 *    fused projection; type as kv->dtype, bf16 for e4m3. q->data may be NULL
 *    (no queries: writing rows to a cache, e.g. converting a bf16 cache to e4m3
 *    with norm 0 and rotary_dim 0; q_out is then ignored), or k->data and
 *    v->data both NULL (queries only; slots may then be NULL); an absent
 *    msa_rows pointer counts as data NULL.
 *    q_out may be q itself; otherwise outputs must not overlap inputs.
 *  - q_weight, k_weight [128], type of q, read where cfg->norm asks; NULL: no scaling.
 *  - positions [n_tokens] int32 and inv_freq [rotary_dim/2] fp32 (finite);
 *    not read when rotary_dim is 0.
 *  - slots [n_tokens] int64 (msa_extend_sequences writes them): -1 marks a padding
 *    token, of which nothing is read or written (its q_out rows stay as they
 *    were); any other value outside the cache sets MSA_ERR_DEVICE_BOUNDS and is
 *    treated the same. Of two tokens with one slot, either may win each row.
 * kv->page_table and kv->seq_lens are not read; num_q_heads is any count >= 1
 * (0 without queries). Nothing is queued for n_tokens 0.
 * ws: the 256-byte header (msa_workspace_size(MSA_OP_APPEND, ...)). */
msa_status msa_qk_norm_rope_append(const msa_rows* q /* host */, const msa_rows* k /* host */,
                                   const msa_rows* v /* host */, int32_t num_q_heads, int32_t n_tokens,
                                   const void* q_weight, const void* k_weight, const int32_t* positions,
                                   const float* inv_freq, const int64_t* slots, const msa_kv_desc* kv /* host */,
                                   const msa_norm_rope_cfg* cfg /* host */, const msa_rows* q_out /* host */, void* ws,
                                   size_t ws_bytes, msa_stream_t stream);

/* Failure-detection self test (the guide has no counterpart; it checks the
 * library's own error path): launches one warp that waits, with the same
 * bounded spin every kernel of the library uses, on a barrier that nothing
 * signals. After `limit_cycles` SM cycles (1000 .. 4e9; MSA_ERR_INVALID_ARG
 * outside) the wait gives up, the status word of `ws` gets MSA_ERR_TIMEOUT and
 * the kernel ends normally: no fault, no trap, the context stays usable.
 * ws: at least the 256-byte header (MSA_ERR_WORKSPACE otherwise). */
msa_status msa_selftest_wait_timeout(void* ws, size_t ws_bytes, int64_t limit_cycles, msa_stream_t stream);

/* Reads (and clears) the sticky device status word of `ws`: synchronises
 * `stream`, stores an msa_status in *status_out (host). */
msa_status msa_read_device_status(const void* ws, msa_stream_t stream, int32_t* status_out /* host */);

/* Static English text for a status code. */
const char* msa_status_string(int32_t status);

/* Library version, e.g. 0x000100 for 0.1.0. */
int32_t msa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
