/*
 * dsa.h - two-tier sparse attention on one GB300 (sm_103a): C ABI.
 *
 * The method is the two-tier sparse-attention step of DeepSeek-V4.1:
 *   - recipes.vllm.ai "DeepSeek-V4.1-Flash", Overview, bullet "Two-tier sparse
 *     attention": every layer attends over a 128-token sliding window; layers
 *     with a compression ratio (1 or 2) add compressed KV latents; an indexer
 *     side attention scores the latents and keeps the best 512 per query,
 *     pre-filtered by a candidate stage that keeps 2048 blocks of 8.
 *   - miles.radixark.com "DeepSeek-V4.1 Flash", §1 Model Introduction,
 *     "Architecture": one 512-wide latent per position is both key and value
 *     for all 64 query heads (no value projection); "Sparse retrieval": a
 *     top-512 candidate set per retrieving layer and a coarser candidate-block
 *     pass.
 * The pages leave the indexer open; this library fixes it as
 *     score(k) = sum_h w_h * ReLU(q_h . k)        (16 index heads x 128),
 * the block key as the mean of the block's 8 index keys, and ties in both
 * top-k stages to the lower index.
 *
 * Conventions shared by every call
 *   - Memory: every tensor pointer is DEVICE memory owned by the caller. The
 *     library allocates nothing and keeps no pointer after a call returns.
 *     Scratch lives in a caller-supplied workspace (see dsa_workspace_size);
 *     one workspace must not serve two calls that may run at the same time.
 *   - Streams: calls enqueue work on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream) and return without synchronising, except
 *     dsa_read_device_status.
 *   - Threads: calls may come from several host threads at once, each with
 *     its own workspace; the library's host-side caches and launch counters
 *     are atomic. The profiling hook dsa_profile_events is the exception.
 *   - Layout: row-major, innermost dimension last. bf16 tensors are passed as
 *     raw 16-bit patterns. Every base pointer must be 16-byte aligned (32-bit
 *     arrays of dsa_plan_step, dsa_norm_rope, dsa_kv_write and dsa_kv_read 4-byte
 *     aligned where nothing else is said).
 *   - Dimensions: the kernels are built for 64 query heads, latent width 512,
 *     16 index heads of width 128, blocks of 8. Other values of those fields
 *     return DSA_ERR_UNSUPPORTED. k_blocks (1..4096), k_tokens (1..512),
 *     window (1..128), ratio (>= 1) and sm_scale are free.
 *   - Errors: every call returns a status and never aborts. Argument errors are
 *     found on the host before any launch. Conditions only the device can see
 *     (an n_latents entry above max_latents, a token id outside its sequence,
 *     block ids not ascending) are recorded in a status word inside the
 *     workspace, the offending element is skipped, and
 *     dsa_read_device_status reports DSA_ERR_DEVICE_CHECK.
 *   - Determinism: results are bit-identical from run to run (no floating-point
 *     atomics; every reduction has a fixed order).
 *   - Tracing: each call marks its phases as NVTX ranges (dsa.decode_step,
 *     dsa.decode_multi, dsa.prefill, dsa.compress_append, dsa.pool, dsa.block_stage,
 *     dsa.token_stage, dsa.attention, dsa.full_attn, dsa.plan, dsa.norm_rope,
 *     dsa.kv_write, dsa.kv_read, dsa.verify_drafts) that a profiler shows on its timeline;
 *     with no tool attached a range costs two calls into empty stubs.
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* dsa_stream_t; /* a cudaStream_t */

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad enum, ... */
  DSA_ERR_MISALIGNED = 2,   /* a base pointer is not 16-byte aligned */
  DSA_ERR_UNSUPPORTED = 3,  /* dimensions the kernels are not built for */
  DSA_ERR_WORKSPACE = 4,    /* workspace missing or smaller than required */
  DSA_ERR_CUDA = 5,         /* a CUDA runtime call failed */
  DSA_ERR_DEVICE_CHECK = 6, /* a kernel flagged bad input (dsa_read_device_status) */
  DSA_ERR_TIMEOUT = 7       /* a bounded device wait ran out (dsa_read_device_status) */
} dsa_status_t;

/* Storage format of index keys and of block-pooled keys (recipes.vllm.ai
 * "DeepSeek-V4.1-Flash" names an MXFP8 and an MXFP4 indexer cache: the
 * "Mixed MXFP4/MXFP8 checkpoint" bullet and indexer_kv_dtype mxfp4 in its
 * serving configurations). */
typedef enum {
  DSA_FMT_BF16 = 0,  /* data: bf16 [rows, 128]; scales: NULL */
  DSA_FMT_MXFP8 = 1, /* data: e4m3 bytes [rows, 128]; scales: UE8M0 bytes [rows, 4]
                        (OCP MX v1.0: one power-of-two scale 2^(s-127) per 32 values) */
  DSA_FMT_MXFP4 = 2  /* data: e2m1 codes two a byte [rows, 64], element 2i in the low
                        nibble of byte i; scales: UE8M0 bytes [rows, 4] (OCP MX v1.0).
                        The kernels read these arrays in pairs of rows: seq_stride_rows
                        must be even, and a buffer whose last sequence's rows are odd in
                        number must hold one row more (it is read, never used). */
} dsa_fmt_t;

typedef struct {
  int n_heads;     /* query heads: 64 */
  int latent_dim;  /* latent width, key = value: 512 */
  int n_idx_heads; /* indexer heads: 16 */
  int idx_dim;     /* indexer width: 128 */
  int block;       /* latents per candidate block: 8 */
  int k_blocks;    /* blocks kept by the candidate stage: 2048 */
  int k_tokens;    /* latents kept per query: 512 */
  int window;      /* sliding-window rows: 128 */
  int ratio;       /* positions per compressed latent: 1 or 2 */
  float sm_scale;  /* softmax scale tau; <= 0 selects 1/sqrt(latent_dim) */
  int kv_fmt;      /* dsa_kv_fmt_t of the latents and window rows the attention reads */
  float kv_scale;  /* DSA_KV_FP8_E4M3: a row holds code * kv_scale; finite, > 0 */
} dsa_config_t;

/* Storage of the latent cache and of the window rows (key = value rows of
 * the attention). The serving pages run an fp8 KV cache (recipes.vllm.ai
 * "DeepSeek-V4.1-Flash", serving configurations, --kv-cache-dtype fp8) and
 * name no scale granularity; this library reads it as OCP E4M3 codes with one
 * scale for the whole cache. fp8 rows are taken by dsa_sparse_attn_decode, its
 * paged form, dsa_decode_step and the dsa_full_attn calls; the prefill, multi-query and append calls
 * return DSA_ERR_UNSUPPORTED for them. The sparse attention converts each code to f16
 * exactly and takes the query to f16 with a power-of-two scale per head (exact
 * unless an element is below 2^-24 of its head's largest), so its MMAs run on
 * f16 operands; the probabilities are f16 too (bf16 with bf16 rows). The dsa_full_attn
 * calls multiply the codes as they are: the query enters as the sum of two E4M3 values a
 * element, exact down to 2^-10 of its head's largest element and within 2^-18 of that below, and so do
 * the probabilities, rounded as to bf16 but for small ones, of which the roundings together
 * change the sum by at most 2^-8 + 2^-9 of it, however many rows there are.
 * Latents "trained to be stored in FP4" (miles.radixark.com "DeepSeek-V4.1
 * Flash") are read as OCP MXFP4, the format of the 4-bit index keys. 4-bit
 * rows are taken by the calls above and by dsa_compress_append; prefill and
 * multi-query calls return DSA_ERR_UNSUPPORTED (dsa_kv_read gives a sequence's
 * rows back as the bf16 rows they take). The attention converts codes times
 * scale to bf16 exactly (scale bytes up to 252; 255 stands for NaN).
 * dsa_kv_write puts rows into a cache of any of the formats. */
typedef enum {
  DSA_KV_BF16 = 0,      /* bf16 rows of 512: 1024 bytes a row */
  DSA_KV_FP8_E4M3 = 1,  /* E4M3 codes, 512 bytes a row, standing for code * kv_scale */
  DSA_KV_MXFP4 = 3      /* 272 bytes a row: 256 of e2m1 codes two a byte (element 2i in the
                           low nibble of byte i), then 16 UE8M0 bytes, byte g the scale
                           2^(s-127) of elements 32 g .. 32 g + 31; kv_scale not used */
} dsa_kv_fmt_t;

/*
 * Paged layout of a decode batch's caches (a block table, as serving engines
 * keep KV caches in fixed-size pages; the candidate-block indexer reads its
 * keys through one, miles.radixark.com "DeepSeek-V4.1 Flash", §4.1). Each
 * cache is a pool of physical pages shared by the B sequences: logical row r
 * of sequence b lives in physical page
 *     page_table[b * pages_per_seq + r / R]   at row r % R of that page,
 * with R = page_rows for index keys and latents and R = page_rows / 8 for
 * block keys (a page of page_rows tokens holds page_rows / 8 blocks). So the
 * pools are laid out as [n_pages * R] rows of the cache's own row format
 * (latents: the row of cfg->kv_fmt; keys: their dsa_fmt_t row, MX scales
 * [n_pages * R, 4]).
 *   page_table:    device int32 [B, pages_per_seq]; an entry outside
 *                  [0, n_pages) is a device-detected error (DSA_ERR_DEVICE_CHECK,
 *                  the rows of that page are skipped)
 *   page_rows:     tokens per page, a positive multiple of 64
 *   pages_per_seq: row stride of page_table, at least ceil(max_latents / page_rows)
 *   n_pages:       physical pages in each pool; n_pages * page_rows < 2^31
 */
typedef struct {
  const int32_t* page_table;
  int32_t page_rows;
  int32_t pages_per_seq;
  int64_t n_pages;
} dsa_pages_t;

/* A key cache (index keys or block-pooled keys) of B sequences. Contiguous
 * (pages == NULL): sequence b's row r is at data + (b * seq_stride_rows + r) *
 * row_bytes, and MX scales are laid out the same way with 4 bytes per row.
 * Paged (pages != NULL): rows are found through the page table above and
 * seq_stride_rows is not used. Paged caches are taken by dsa_pool_index_keys,
 * dsa_index_blocks, dsa_topk, dsa_topk_noalloc and dsa_decode_step (decode
 * only; prefill reads one contiguous sequence). */
typedef struct {
  dsa_fmt_t fmt;
  const void* data;
  const uint8_t* scales;
  int64_t seq_stride_rows;
  const dsa_pages_t* pages;
} dsa_keys_t;

/* The writable form, for dsa_pool_index_keys' output. */
typedef struct {
  dsa_fmt_t fmt;
  void* data;
  uint8_t* scales;
  int64_t seq_stride_rows;
  const dsa_pages_t* pages;
} dsa_keys_out_t;

/* Fills *cfg with the DeepSeek-V4.1 values above (ratio 1, sm_scale 0). */
void dsa_default_config(dsa_config_t* cfg);

/* Human-readable name of a status. Never NULL. */
const char* dsa_status_string(dsa_status_t s);

/*
 * Workspace bytes needed by any call below for up to `n_queries` queries
 * (decode: the batch B; prefill: n_q) whose sequences hold at most
 * `max_latents` latents each. Any larger workspace works too. The buffer must
 * be 256-byte aligned device memory, zeroed once before its first use (its
 * first 16 bytes hold the device status word), and is reused across calls.
 */
dsa_status_t dsa_workspace_size(const dsa_config_t* cfg, int n_queries, int64_t max_latents,
                                size_t* bytes);

/*
 * S0, block keys (the candidate stage's "blocks of 8", recipes.vllm.ai
 * "DeepSeek-V4.1-Flash", Overview, "Two-tier sparse attention"; the block key is
 * the mean of the block's index keys, the rule this library fixes).
 * For each sequence b and each block j < ceil(n_latents[b] / 8) (or only the
 * block holding latent n_latents[b] - 1 when tail_only != 0):
 *     pooled[b][j] = RN_fmt( fp32_sum_in_order(keys[b][8j .. 8j+c-1]) / c ),
 * c = min(8, n_latents[b] - 8j). RN_fmt is round-to-nearest-even to bf16, or
 * the OCP MX conversion (X = floor(log2 amax) - emax per 32 values, emax 8
 * for e4m3 and 2 for e2m1, elements rounded to nearest even with saturation).
 * pooled->fmt must equal keys->fmt.
 *   n_latents: device int32 [B], each in [0, max_latents].
 */
dsa_status_t dsa_pool_index_keys(const dsa_config_t* cfg, const dsa_keys_t* keys,
                                 const int32_t* n_latents, int B, int64_t max_latents,
                                 int tail_only, const dsa_keys_out_t* pooled, void* workspace,
                                 size_t workspace_bytes, dsa_stream_t stream);

/*
 * S1 + S2, candidate-block stage: per query b, score every block j <
 * ceil(n_latents[b] / 8) with score = sum_h w_h ReLU(q_idx[b][h] . pooled[b][j])
 * and keep the k_blocks best by (score desc, j asc). When a query has at most
 * k_blocks blocks, all are kept.
 *   q_idx:        device bf16 [B, 16, 128]
 *   w:            device fp32 [B, 16]
 *   pooled:       block keys, as written by dsa_pool_index_keys
 *   n_latents:    device int32 [B]
 *   block_ids:    out, device int32 [B, k_blocks], ascending, -1 padded
 *   block_scores: out (optional, may be NULL), device fp32 [B, ceil(max_latents/8)];
 *                 entries past a query's block count are -inf
 */
dsa_status_t dsa_index_blocks(const dsa_config_t* cfg, const void* q_idx, const float* w,
                              const dsa_keys_t* pooled, const int32_t* n_latents, int B,
                              int64_t max_latents, int32_t* block_ids, float* block_scores,
                              void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * S3 + S4, token stage: per query b, score every visible latent t of the kept
 * blocks (t = 8 * block_ids[b][i] + r, r < 8, t < n_latents[b]) and keep the
 * k_tokens best by (score desc, t asc).
 *   block_ids:    device int32 [B, k_blocks], ascending with -1 padding at the
 *                 end (as dsa_index_blocks writes it), or NULL for "every block"
 *   token_ids:    out, device int32 [B, k_tokens], ascending, -1 padded
 *   token_scores: out (optional), device fp32 [B, n_cand]: the score of
 *                 candidate i (i.e. latent 8 * block_ids[b][i / 8] + i % 8), or of
 *                 latent i when block_ids is NULL; -inf where no latent exists.
 *                 n_cand = 8 * k_blocks, or max_latents rounded up to 8 when
 *                 block_ids is NULL.
 */
dsa_status_t dsa_topk(const dsa_config_t* cfg, const void* q_idx, const float* w,
                      const dsa_keys_t* keys, const int32_t* block_ids,
                      const int32_t* n_latents, int B, int64_t max_latents, int32_t* token_ids,
                      float* token_scores, void* workspace, size_t workspace_bytes,
                      dsa_stream_t stream);

/*
 * S5 - S7, attention (miles.radixark.com "DeepSeek-V4.1 Flash", §1: the latent
 * is key and value for all 64 heads). For query b the rows are
 *     KV = latents[b][token_ids[b][i]] for every id >= 0, then swa[b][0 .. swa_len[b]-1]
 * (selected latents and the sliding window, concatenated), and every head h
 *     z_j = tau * q[b][h] . KV_j,   out[b][h] = sum_j softmax(z)_j KV_j,
 *     lse[b][h] = log sum_j exp(z_j)   (natural log; -inf when there are no rows).
 *   q:        device bf16 [B, 64, 512]
 *   latents:  device bf16, sequence b's row r at (b * latent_seq_stride_rows + r) * 512
 *             (cfg->kv_fmt DSA_KV_FP8_E4M3: uint8 E4M3 codes, the same row layout;
 *             DSA_KV_MXFP4: 272-byte rows, row r at (b * latent_seq_stride_rows + r) * 272)
 *   n_latents: device int32 [B]; an id >= n_latents[b] is flagged and skipped
 *   token_ids: device int32 [B, k_tokens], -1 entries are skipped
 *   swa:      device bf16 [B, window, 512]; slot s holds position T - swa_len[b] + s
 *             (DSA_KV_FP8_E4M3: uint8 E4M3 codes [B, window, 512]; DSA_KV_MXFP4: uint8
 *             [B, window, 272]). The rows' order does not matter to the result, so a
 *             sequence's slots may also be a ring (position p in slot p % window).
 *   swa_len:  device int32 [B], each in [0, window]
 *   out:      out, device bf16 [B, 64, 512]
 *   lse:      out (optional), device fp32 [B, 64]
 */
dsa_status_t dsa_sparse_attn_decode(const dsa_config_t* cfg, const void* q, const void* latents,
                                    int64_t latent_seq_stride_rows, const int32_t* n_latents,
                                    const int32_t* token_ids, const void* swa,
                                    const int32_t* swa_len, int B, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes,
                                    dsa_stream_t stream);

/*
 * dsa_sparse_attn_decode over a paged latent pool: latent id t of sequence b
 * is row page_table[b * pages_per_seq + t / page_rows] * page_rows + t % page_rows
 * of `latents` (bf16 [pages->n_pages * page_rows, 512], or rows of the other cache
 * formats). Ids whose page entry is out of range are skipped and reported like ids past n_latents.
 */
dsa_status_t dsa_sparse_attn_decode_paged(const dsa_config_t* cfg, const void* q,
                                          const void* latents, const dsa_pages_t* pages,
                                          const int32_t* n_latents, const int32_t* token_ids,
                                          const void* swa, const int32_t* swa_len, int B,
                                          void* out, float* lse, void* workspace,
                                          size_t workspace_bytes, dsa_stream_t stream);

/*
 * The whole decode step for B sequences, the query of sequence b at position
 * T_b - 1 with n_latents[b] = T_b / ratio visible latents: pool the newest
 * block (when update_pool != 0), the candidate-block stage (skipped when no
 * sequence can have more than k_blocks blocks), the token stage and the
 * attention, as the four calls above would in sequence.
 *   pooled:        block keys, read by the block stage; also written (newest
 *                  block only) when update_pool != 0
 *   keys, pooled:  both contiguous, or both paged with the same page table;
 *                  paged keys make the latents paged by that table too (and
 *                  latent_seq_stride_rows is then not used)
 *   block_ids:     out (optional), device int32 [B, k_blocks]
 *   token_ids:     out (optional), device int32 [B, k_tokens]
 */
dsa_status_t dsa_decode_step(const dsa_config_t* cfg, const void* q, const void* q_idx,
                             const float* w, const dsa_keys_t* keys, const dsa_keys_out_t* pooled,
                             int update_pool, const void* latents,
                             int64_t latent_seq_stride_rows, const int32_t* n_latents,
                             int64_t max_latents, const void* swa, const int32_t* swa_len, int B,
                             int32_t* block_ids, int32_t* token_ids, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * Prefill: n_q queries appended after ctx_len tokens of one sequence, query i
 * at position P = ctx_len + i. Each query has its own causal selection: it sees
 * floor((P + 1) / ratio) latents; a block that it sees only in part is pooled
 * over its visible members on the fly; its window is positions
 * max(0, P - window + 1) .. P.
 *   q:         device bf16 [n_q, 64, 512]
 *   q_idx:     device bf16 [n_q, 16, 128];  w: device fp32 [n_q, 16]
 *   latents:   device bf16 [n_lat, 512], n_lat = (ctx_len + n_q) / ratio
 *   keys:      index keys [n_lat, 128] (seq_stride_rows ignored)
 *   pooled:    block keys of the complete blocks [n_lat / 8, 128]
 *   swa:       device bf16 [n_q + window - 1, 512]; row r holds position
 *              ctx_len - window + 1 + r (rows before position 0 are never read)
 *   out:       out, device bf16 [n_q, 64, 512];  lse: out (optional) fp32 [n_q, 64]
 *   token_ids: out (optional), device int32 [n_q, k_tokens]
 */
dsa_status_t dsa_sparse_attn_prefill(const dsa_config_t* cfg, int n_q, int64_t ctx_len,
                                     const void* q, const void* q_idx, const float* w,
                                     const void* latents, const dsa_keys_t* keys,
                                     const dsa_keys_t* pooled, const void* swa, void* out,
                                     float* lse, int32_t* token_ids, void* workspace,
                                     size_t workspace_bytes, dsa_stream_t stream);

/*
 * Cache append at the compression step (recipes.vllm.ai "DeepSeek-V4.1-Flash",
 * Overview, "Two-tier sparse attention": layers with a compression ratio keep
 * latents "pooled by a learned softmax gate", one latent per ratio positions).
 * For each sequence b whose token count T_b = n_tokens[b] completes a latent
 * (T_b % ratio == 0), latent j = T_b / ratio - 1 becomes
 *     RN( sum_i softmax(gate[b])_i * kv[b][i] ),   i = 0 .. ratio - 1,
 * rounded once from fp32 to bf16, or with cfg->kv_fmt DSA_KV_MXFP4 to that format
 * (softmax over the group's ratio logits, in fp32), its index key row becomes
 * new_keys' row b, and the block key of the block holding j is re-pooled as
 * dsa_pool_index_keys(tail_only) does. Sequences that complete no latent are
 * left as they are. The gate's learned projection is not on the pages: its
 * logits are inputs.
 *   n_tokens:  device int32 [B]
 *   kv:        device bf16 [B, ratio, 512]: the group's per-position KV vectors
 *   gate:      device fp32 [B, ratio]
 *   new_keys:  the new index key of each sequence, one row per sequence (data
 *              [B, row], MX scales [B, 4]; seq_stride_rows not used)
 *   latents:   rows of cfg->kv_fmt (bf16 or MXFP4), contiguous with
 *              latent_seq_stride_rows rows a sequence, or paged by keys->pages like the keys
 *   keys, pooled: the index-key and block-key caches (written)
 *   max_latents: the caches' capacity; a latent at or past it is a device check
 * ratio must be at most 32 (DSA_ERR_UNSUPPORTED otherwise). The workspace is
 * sized for B queries.
 */
dsa_status_t dsa_compress_append(const dsa_config_t* cfg, int B, const int32_t* n_tokens,
                                 const void* kv, const float* gate, const dsa_keys_t* new_keys,
                                 void* latents, int64_t latent_seq_stride_rows,
                                 const dsa_keys_out_t* keys, const dsa_keys_out_t* pooled,
                                 int64_t max_latents, void* workspace, size_t workspace_bytes,
                                 dsa_stream_t stream);

/*
 * Multi-query decode: n_q queries per sequence at its last n_q positions, as
 * when a block of draft tokens is verified in one pass (recipes.vllm.ai
 * "DeepSeek-V4.1-Flash", Overview, bullet "DSpark draft head"). Sequence b
 * holds T_b = n_tokens[b] tokens and its query i sits at position
 * P = T_b - n_q + i. Each query is causal with its own two-tier selection over
 * floor((P + 1) / ratio) latents (a block it sees in part is pooled over its
 * visible members on the fly, as in prefill) and its own window of positions
 * max(0, P - window + 1) .. P; the queries of a sequence read the same caches.
 *   n_tokens:    device int32 [B], each >= n_q (the queries of a shorter
 *                sequence that have no position get no rows, reported as
 *                DSA_ERR_DEVICE_CHECK)
 *   q:           device bf16 [B, n_q, 64, 512]; q_idx bf16 [B, n_q, 16, 128];
 *                w fp32 [B, n_q, 16]
 *   keys:        index keys of each sequence, contiguous (seq_stride_rows >=
 *                max_latents)
 *   pooled:      block keys of each sequence's complete blocks, as
 *                dsa_pool_index_keys writes them (seq_stride_rows >= max_latents / 8)
 *   latents:     bf16, sequence b's row r at (b * latent_seq_stride_rows + r) * 512
 *   max_latents: at least floor(n_tokens[b] / ratio) for every b
 *   swa:         device bf16 [B, window + n_q - 1, 512]; row r of sequence b
 *                holds position T_b - n_q - window + 1 + r (rows before
 *                position 0 are never read)
 *   out:         out, bf16 [B, n_q, 64, 512]; lse: out (optional) fp32 [B, n_q, 64]
 *   token_ids:   out (optional), int32 [B, n_q, k_tokens]
 * The workspace is sized for B * n_q queries (dsa_workspace_size).
 */
dsa_status_t dsa_decode_multi(const dsa_config_t* cfg, int n_q, const int32_t* n_tokens,
                              const void* q, const void* q_idx, const float* w,
                              const dsa_keys_t* keys, const dsa_keys_t* pooled,
                              const void* latents, int64_t latent_seq_stride_rows,
                              int64_t max_latents, const void* swa, int B, void* out, float* lse,
                              int32_t* token_ids, void* workspace, size_t workspace_bytes,
                              dsa_stream_t stream);

/*
 * Attention over the whole cache: every latent of the sequence instead of a selection, and
 * the window rows, under one softmax (miles.radixark.com "DeepSeek-V4.1 Flash", §1: the
 * latent is key and value for all 64 heads). For caches of at most k_tokens latents it is what
 * the sparse calls compute; over longer ones it measures what a selection leaves out. The rows
 * of query b are
 *     KV = latents of sequence b, 0 .. n_latents[b] - 1, then swa[b][0 .. swa_len[b] - 1],
 * and out and lse are those of dsa_sparse_attn_decode.
 *   q:           device bf16 [B, 64, 512]
 *   latents:     rows of cfg->kv_fmt, contiguous (pages NULL: sequence b's row r is row
 *                b * latent_seq_stride_rows + r) or in pages->page_rows pages of a pool; the
 *                contiguous array has less than 2^31 rows (DSA_ERR_UNSUPPORTED); may be NULL
 *                with max_latents 0
 *   n_latents:   device int32 [B], each in [0, max_latents]; another is reported (DSA_ERR_DEVICE_CHECK)
 *                and taken to the nearer end. Rows past it are not used, whatever they hold.
 *   max_latents: latents that a sequence's cache can hold: at most latent_seq_stride_rows, or
 *                pages_per_seq * page_rows
 *   swa, swa_len: the window rows as in dsa_sparse_attn_decode (cfg->window rows a sequence, in any
 *                order), or both NULL: no window
 *   out:         out, device bf16 [B, 64, 512]; lse: out (optional), device fp32 [B, 64]. A
 *                query without rows gets zeros and -inf.
 * Rows of a page whose table entry is outside the pool are skipped and reported. out, lse and
 * the workspace overlap no input and not one another (DSA_ERR_INVALID_ARG). B (in
 * dsa_full_attn_multi B * n_q) is at most 2^20, and B * (max_latents / 64 + 8) below 2^31
 * (DSA_ERR_UNSUPPORTED).
 * The workspace has the size dsa_full_attn_workspace_size gives, the same for
 * every n_queries and format (42 MB: partial outputs of the queries that several SMs share); it is
 * aligned and zeroed like the others, and the calls that need none but a status word
 * (dsa_plan_step, dsa_kv_write, ...) take it too.
 */
dsa_status_t dsa_full_attn_workspace_size(const dsa_config_t* cfg, int n_queries, size_t* bytes);
dsa_status_t dsa_full_attn_decode(const dsa_config_t* cfg, const void* q, const void* latents,
                                  int64_t latent_seq_stride_rows, const dsa_pages_t* pages,
                                  const int32_t* n_latents, int64_t max_latents, const void* swa,
                                  const int32_t* swa_len, int B, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * The same for n_q queries a sequence at its last n_q positions, as when a block of draft
 * tokens is verified in one pass: positions, causality and the window rows are those of
 * dsa_decode_multi (query i of sequence b at P = n_tokens[b] - n_q + i sees
 * floor((P + 1) / ratio) latents and its own window), over a contiguous or paged cache of any
 * format. Each query reads its rows anew: this is for a few, not for prompts.
 *   n_tokens: device int32 [B], each >= n_q (the queries of a shorter sequence that have
 *             no position get no rows, reported as DSA_ERR_DEVICE_CHECK); with at most
 *             max_latents latents each (reported; the first max_latents are used)
 *   q, out:   device bf16 [B, n_q, 64, 512]; lse: fp32 [B, n_q, 64] or NULL
 *   swa:      rows of cfg->kv_fmt [B, window + n_q - 1], row r of sequence b at position
 *             n_tokens[b] - n_q - window + 1 + r (rows before position 0 are not used), or NULL
 */
dsa_status_t dsa_full_attn_multi(const dsa_config_t* cfg, int n_q, const int32_t* n_tokens,
                                 const void* q, const void* latents,
                                 int64_t latent_seq_stride_rows, const dsa_pages_t* pages,
                                 int64_t max_latents, const void* swa, int B, void* out,
                                 float* lse, void* workspace, size_t workspace_bytes,
                                 dsa_stream_t stream);

/*
 * dsa_topk without a workspace. The pages have no counterpart to this call; it
 * serves callers that cannot allocate device memory: a plugin that runs inside
 * a host framework which owns all device memory and lends it none, or a
 * serving loop under a fixed memory budget that forbids allocation once it has
 * started. It computes exactly what dsa_topk computes (same kernels, same
 * arguments, bit-identical token_ids) but keeps its candidate scores in a
 * scratch array that the library defines statically in device memory:
 * DSA_TOPK_NOALLOC_MAX_SCORES fp32 values (8 MiB), held on every GPU that
 * loads the library until the process exits. It calls no allocator.
 *   - Limit: B * n_cand <= DSA_TOPK_NOALLOC_MAX_SCORES, where n_cand is
 *     8 * k_blocks (block_ids given) or max_latents rounded up to 8 (block_ids
 *     NULL); larger requests return DSA_ERR_WORKSPACE before any launch.
 *   - Set-up: the first call on each device looks up that device's address of
 *     the scratch array (the calling thread's current device must be the one
 *     the stream belongs to); make that first call before any stream capture.
 *   - Sharing: every call on a device uses the same scratch array, which keeps
 *     the last call's contents (every score the kernels read is written first
 *     by the same call, so nothing needs clearing). Calls that may overlap on
 *     the GPU (different streams without ordering) race on it: serialise them.
 *   - No status word: device-side input checks (ids outside a sequence,
 *     unordered block ids) skip the offending elements and report nothing,
 *     and a bounded device wait that runs out (DSA_ERR_TIMEOUT in the other
 *     calls) is not reported either. After such a timeout the scan leaves
 *     score slots unwritten, so the selection may rank scores left in the
 *     scratch by an earlier call while the call still returns DSA_OK. Use
 *     dsa_topk with a workspace where these conditions must be seen.
 */
#define DSA_TOPK_NOALLOC_MAX_SCORES (1 << 21)
dsa_status_t dsa_topk_noalloc(const dsa_config_t* cfg, const void* q_idx, const float* w,
                              const dsa_keys_t* keys, const int32_t* block_ids,
                              const int32_t* n_latents, int B, int64_t max_latents,
                              int32_t* token_ids, dsa_stream_t stream);

/*
 * Around the attention of a serving step: the step's plan, the queries and
 * keys it takes, and the cache rows it reads. A decode loop calls
 *     dsa_plan_step -> dsa_norm_rope -> dsa_compress_append and dsa_kv_write
 *     -> dsa_decode_step
 * on one stream, all from device memory, and captures into a CUDA graph. dsa_norm_rope and
 * dsa_kv_write do nothing in a step that the plan refuses (it counts no token and gives no slot).
 * dsa_compress_append goes by the token counts that it is given, and would write a complete group's
 * latent again: give it 0 for a request without a new token (where cu_new does not grow).
 */

/* A pool of pages that requests share, and its free pages. */
typedef struct {
  int32_t* page_table;       /* device [B, pages_per_seq], updated in place */
  int32_t page_rows;         /* latents per page, a positive multiple of 64 */
  int32_t pages_per_seq;     /* row stride of page_table */
  int64_t n_pages;           /* n_pages * page_rows < 2^31 */
  int32_t* free_ring;        /* device [n_pages]: free pages at positions head .. tail - 1,
                                modulo n_pages; updated in place */
  const int64_t* ring_state; /* device {head, tail}, 0 <= tail - head <= n_pages */
  int64_t* ring_state_out;   /* {head, tail} after the step; may be ring_state itself */
} dsa_page_pool_t;

/* What a step's plan writes (device arrays; n_tokens may be the input lengths
 * themselves, no others may overlap). Token arrays hold max_new entries, the
 * new tokens of request 0 first; entries past the last token hold position 0
 * and -1 elsewhere. */
typedef struct {
  int32_t* n_tokens;     /* [B] lengths after the step */
  int32_t* n_latents;    /* [B] n_tokens / ratio */
  int32_t* swa_len;      /* [B] min(n_tokens, window) */
  int32_t* cu_new;       /* [B + 1] index of each request's first new token; the total last */
  int32_t* token_seq;    /* [max_new] request of each token */
  int32_t* positions;    /* [max_new] its position */
  int32_t* latent_slots; /* [max_new] pool row of the latent it completes, or -1 */
  int32_t* window_slots; /* [max_new] request * window + position % window for the request's
                            last `window` positions, -1 for earlier ones */
  int32_t max_new;       /* 0 .. 2^30; the arrays above are 16-byte aligned */
} dsa_step_plan_t;

#define DSA_PLAN_MAX_REQUESTS 4096

/*
 * Block tables and slot maps of a step, built on the GPU from the requests'
 * lengths (the pages keep caches in pages of a shared pool; how pages are
 * given out is this library's choice).
 *   n_tokens: device int32 [B], lengths before the step
 *   n_new:    device int32 [B], tokens that the step adds to each request (0 is
 *             fine); a negative number ends the request: its length becomes 0
 *             and its pages go back to the ring (its table entries are left as
 *             they are and mean nothing any more)
 * A request of n tokens holds ceil((n / ratio) / page_rows) pages, entries 0 ..
 * of its table row. New pages are popped from the ring in request order, then
 * page order, and ended requests' pages pushed in the same order; a page freed
 * in a step is not given out in the same step.
 * All or nothing: when lengths or additions are impossible (negative lengths, more
 * latents than pages_per_seq pages hold, more new tokens than max_new), the
 * free pages are too few or the ring's counters are not those of a ring, the
 * call changes no length, no table entry and nothing of the ring, cu_new is 0,
 * every token entry is that of a row past the last token, and
 * dsa_read_device_status reports DSA_ERR_DEVICE_CHECK.
 * A page id outside the pool (0 .. n_pages - 1) is not passed on; -1, no page, takes its
 * place. Tokens that fall on such an entry, of the table or newly popped from the ring, get -1
 * slots and are reported with their request, in whose row the ring's entry is -1. When a
 * request ends that holds such an entry, the request is reported, and the page's position in
 * the ring holds -1 (an entry that is -1 already goes back as it is: its tokens were reported).
 * B is at most DSA_PLAN_MAX_REQUESTS (DSA_ERR_UNSUPPORTED above). The workspace
 * may be of any size that dsa_workspace_size gives.
 */
dsa_status_t dsa_plan_step(const dsa_config_t* cfg, int B, const int32_t* n_tokens,
                           const int32_t* n_new, const dsa_page_pool_t* pool,
                           const dsa_step_plan_t* plan, void* workspace, size_t workspace_bytes,
                           dsa_stream_t stream);

/* Element type of the heads of dsa_norm_rope. */
typedef enum { DSA_DT_BF16 = 0, DSA_DT_F16 = 1, DSA_DT_F32 = 2 } dsa_dtype_t;

/* A group of heads: token t's head h has elements x[t * x_token_stride + h *
 * x_head_stride + 0 .. dim - 1], and goes to out by out's strides. Strides count
 * elements and, like the base pointers, are multiples of 16 bytes; that of a single
 * token or head is not used. out's heads do not overlap (DSA_ERR_INVALID_ARG). out may be
 * x with the same strides (in place); they must not overlap otherwise. Nor may a group's out
 * overlap another's x or out, since nothing orders the groups of a call (that is refused
 * where two of them start at one address); groups may read the same x. */
typedef struct {
  const void* x;
  void* out;
  int heads;                 /* >= 0 */
  int dim;                   /* elements of a head: a multiple of 8, 8 .. 1024 */
  int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;
  const float* weight;       /* device fp32 [dim], 16-byte aligned, or NULL (all 1) */
  float eps;                 /* >= 0, finite */
  int norm;                  /* 0: no norm (weight and eps are not used) */
  int rope_start;            /* first rotated element, a multiple of 8; < 0: no rotation */
} dsa_heads_t;

#define DSA_MAX_HEAD_GROUPS 8

/* A rotation: pair i of a token at position p turns by p * inv_freq[i]; cosine
 * and sine are multiplied by `scale` (1 for plain RoPE, YaRN's factor with it). */
typedef struct {
  const double* inv_freq;    /* device fp64 [rope_dim / 2], radians per position, of either
                                sign; an infinity or NaN makes its pair NaN */
  int rope_dim;              /* rotated elements: a multiple of 8 (interleaved) or 16, <= 1024 */
  int interleaved;           /* pair i: elements 2i and 2i + 1; else i and i + rope_dim / 2 */
  float scale;
} dsa_rope_t;

/*
 * Norms of queries and keys for each head, with the position rotation in the
 * same pass, over n_groups groups of heads in one launch (the step's queries,
 * latents, index queries and index keys, for instance):
 *     y = x / sqrt(mean(x^2) + eps) * weight   over each head's dim elements,
 *     then elements rope_start .. rope_start + rope_dim - 1 turned in pairs:
 *     (y0, y1) -> (y0 c - y1 s, y0 s + y1 c).
 * The pages name a KV norm and RoPE (theta 160000, YaRN x16) and give no
 * formula; RMS norm and both pairings are the common forms. Arithmetic in fp32,
 * one rounding to the elements' type. An angle p * inv_freq[i] is reduced to its fraction of
 * a turn in 64-bit integers, right to within 2^-33 turns and 2^-63 of the whole
 * angle, and its cosine and sine are taken in fp32.
 *   positions: device int32 [n], of either sign
 *   n_valid:   device int32 or NULL: only tokens below *n_valid are done, the
 *              rows behind them are left as they were (cu_new + B of a plan)
 *   groups:    host array of n_groups <= DSA_MAX_HEAD_GROUPS
 *   rope:      NULL: norms only
 */
dsa_status_t dsa_norm_rope(int n, const int32_t* n_valid, const int32_t* positions,
                           dsa_dtype_t dtype, const dsa_heads_t* groups, int n_groups,
                           const dsa_rope_t* rope, dsa_stream_t stream);

/*
 * Rows into a cache: bf16 row r of `rows` (r * row_stride elements from its
 * start) becomes row slots[r] of `cache` in cfg->kv_fmt.
 *   DSA_KV_BF16: as it is. DSA_KV_FP8_E4M3: RN_e4m3(x / kv_scale, divided in fp32),
 *   saturating: an infinity becomes +-448, a NaN a NaN code.
 *   DSA_KV_MXFP4: the OCP MX conversion (scale 2^X, X = floor(log2 amax) - 2 per
 *   32 elements, at least -127; 2^0 for zeros; elements to nearest, ties to the
 *   even code, at most 6); a group that holds a NaN or an infinity gets the NaN
 *   scale.
 * A negative slot skips its row. The other slots are distinct (of two rows with
 * one slot, either's bytes may stay). A slot >= n_rows is skipped and reported
 * (DSA_ERR_DEVICE_CHECK).
 *   n_valid: as in dsa_norm_rope
 *   slots:   device int32 [n] (a plan's latent_slots or window_slots)
 *   cache:   n_rows rows of the format (n_pages * page_rows for a pool,
 *            B * window for the window rows); n_rows < 2^31; `rows` does not overlap it
 *            (here and in dsa_kv_read)
 * The workspace may be of any size that dsa_workspace_size gives: its status word alone is
 * used here and in dsa_kv_read, however many rows there are.
 */
dsa_status_t dsa_kv_write(const dsa_config_t* cfg, int n, const int32_t* n_valid, const void* rows,
                          int64_t row_stride, const int32_t* slots, void* cache, int64_t n_rows,
                          void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * Rows out of a cache: row slots[r] of `cache` as bf16 to row r of `rows`, code
 * times scale (exact for MXFP4 scales up to 2^125; rounded once for E4M3, products
 * of at least 2^-122). Rows with a negative slot are left as they were. A cache of any format so serves
 * the calls that read bf16 rows (a sequence's latents for dsa_sparse_attn_prefill).
 */
dsa_status_t dsa_kv_read(const dsa_config_t* cfg, int n, const int32_t* n_valid, const void* cache,
                         int64_t n_rows, const int32_t* slots, void* rows, int64_t row_stride,
                         void* workspace, size_t workspace_bytes, dsa_stream_t stream);

/*
 * Tokens taken off the requests' ends, as when drafted tokens are rejected: request b of
 * n_tokens[b] tokens keeps n_tokens[b] - n_drop[b] of them, and the pages that it then needs no
 * more go back to the ring in request order, then page order (their table entries are left as they are and
 * mean nothing any more). Written are the plan's n_tokens (which may be the input lengths),
 * n_latents and swa_len; its token arrays and cu_new are not used and may be NULL.
 *   n_drop: device int32 [B], each in [0, n_tokens[b]]
 * All or nothing as in dsa_plan_step: when a length or a number to drop is impossible or the
 * ring's counters are not those of a ring, no length and nothing of the ring changes
 * (DSA_ERR_DEVICE_CHECK). Page ids outside the pool are treated as there. Latents of
 * the tokens dropped stay in the cache's rows until others are written there; nothing reads them. The window rows
 * that a ring of `window` slots lost to the dropped tokens are lost: a caller that drops tokens
 * writes the window rows once it knows which stay, or keeps the rows of n_drop more positions.
 */
dsa_status_t dsa_plan_trim(const dsa_config_t* cfg, int B, const int32_t* n_tokens,
                           const int32_t* n_drop, const dsa_page_pool_t* pool,
                           const dsa_step_plan_t* plan, void* workspace, size_t workspace_bytes,
                           dsa_stream_t stream);

#define DSA_MAX_DRAFTS 255
#define DSA_MAX_VOCAB 500000

/*
 * Verification of drafted tokens (recipes.vllm.ai "DeepSeek-V4.1-Flash", Overview, bullet
 * "DSpark draft head", names blocks of drafted tokens; the rule is speculative sampling's).
 * Request b has N = n_drafts[b] drafts x_0 .. x_{N-1}, the drafter's probabilities q_i they were
 * drawn from and the target's probabilities p_0 .. p_N at their positions and the one behind:
 *     draft i stands when u_i q_i(x_i) < p_i(x_i) and every one before it stands;
 *     with k drafts standing, the token behind them is drawn from max(p_k - q_k, 0) if k < N
 *     (from p_k if nothing of that is left), from p_N if k = N: the first t with
 *     sum_{s <= t} w_s > u sum_s w_s.
 * Tokens so drawn follow the target's distribution when the u are independent and uniform
 * on [0, 1). A value counts as a probability in [0, 1] (a NaN or a negative one as 0, one above 1 as
 * 1), to the nearest multiple of 2^-44 in the sums, which are exact; rows need not sum to 1.
 *   target:       device [B, n_draft + 1, vocab] of dtype, row (b, i) at (b (n_draft + 1) + i) *
 *                 target_stride elements
 *   draft:        device [B, n_draft, vocab], row (b, i) at (b n_draft + i) * draft_stride; or NULL: each
 *                 draft had probability 1 (a drafter that takes its likeliest token)
 *                 (strides of at least vocab; that of a single row is not used)
 *   draft_tokens: device int32 [B, n_draft]; an id outside the vocabulary does not stand and is
 *                 reported (DSA_ERR_DEVICE_CHECK)
 *   n_drafts:     device int32 [B], or NULL: n_draft each; above n_draft: reported, n_draft;
 *                 negative: the request has no step (tokens -1, counts 0)
 *   uniform:      device fp32 [B, n_draft + 1]: u_i of draft i, and last the u of the drawn token
 *   tokens:       out, device int32 [B, n_draft + 1]: the drafts that stand, the drawn token,
 *                 then -1. A row without any probability gives -1, reported.
 *   n_kept:       out, device int32 [B]: tokens of the request (k + 1)
 *   n_drop:       out (optional), device int32 [B]: N - k, the drafts that do not stand (what
 *                 dsa_plan_trim takes off a step of N + 1 tokens)
 * Outputs and the status word overlap no input and not one another (DSA_ERR_INVALID_ARG). n_draft
 * is at most DSA_MAX_DRAFTS (0 draws one token from p), vocab at most DSA_MAX_VOCAB, B at most 2^20
 * (DSA_ERR_UNSUPPORTED). The workspace may be of
 * any size that dsa_workspace_size gives (its status word is used).
 */
dsa_status_t dsa_verify_drafts(int B, int n_draft, int64_t vocab, dsa_dtype_t dtype,
                               const void* target, int64_t target_stride, const void* draft,
                               int64_t draft_stride, const int32_t* draft_tokens,
                               const int32_t* n_drafts, const float* uniform, int32_t* tokens,
                               int32_t* n_kept, int32_t* n_drop, void* workspace,
                               size_t workspace_bytes, dsa_stream_t stream);

/* Kernel kinds, for the timing hook and the launch counters below. */
typedef enum {
  DSA_KERNEL_POOL = 0,    /* block-key pooling */
  DSA_KERNEL_SCAN = 1,    /* indexer scores (block stage and token stage) */
  DSA_KERNEL_SELECT = 2,  /* top-k selection */
  DSA_KERNEL_ATTN = 3,    /* attention */
  DSA_KERNEL_OTHER = 4,   /* identity block lists, step plans, norms, cache rows */
  DSA_KERNEL_KINDS = 5
} dsa_kernel_kind_t;

/*
 * Optional timing hook for profiling and benchmarks (no counterpart on the
 * pages). With n > 0, each later launch of kernel `kind` is bracketed on its
 * stream by cudaEventRecord(starts[i % n]) and cudaEventRecord(ends[i % n]),
 * where i counts that kind's launches since this call; n = 0 switches it off.
 * starts/ends hold caller-owned cudaEvent_t handles and must outlive their use.
 * The setting is process-wide and not thread-safe. Recording inside CUDA-graph
 * capture does not give timings; use it on plain stream launches.
 */
dsa_status_t dsa_profile_events(int kind, void* const* starts, void* const* ends, int n);

/*
 * Number of kernel launches per kind (counts[DSA_KERNEL_KINDS]) issued by this
 * process since it started or since the last call with reset != 0.
 */
dsa_status_t dsa_launch_counts(uint64_t* counts, int reset);

/*
 * Waits for `stream`, then reads and clears the status word in `workspace`:
 * DSA_OK, DSA_ERR_DEVICE_CHECK or DSA_ERR_TIMEOUT (the earliest recorded).
 * If info is not NULL it receives the recorded detail word (0 if none): bits
 * 24..31 name the kernel (1 block-key pooling, 2 indexer scan, 3 top-k
 * selection, 4 attention, 5 prefill partial block, 6 the self-test below, 7 step
 * plan, 8 cache rows, 9 attention over the whole cache, 10 draft
 * verification),
 * bits 0..23 a detail (for
 * DSA_ERR_TIMEOUT the shared-memory address of the barrier waited on; for
 * DSA_ERR_DEVICE_CHECK the offending sequence index or id).
 */
dsa_status_t dsa_read_device_status(void* workspace, dsa_stream_t stream, uint32_t* info);

/*
 * Self-test of the device failure report (no counterpart on the pages): a
 * kernel waits on a barrier that nothing arrives at, under the bounded-wait
 * scheme the step's kernels use but with a limit of about one millisecond,
 * gives up and records DSA_ERR_TIMEOUT in `workspace`'s status word. A
 * following dsa_read_device_status returns DSA_ERR_TIMEOUT with site 6; the
 * device stays usable. Returns DSA_ERR_INVALID_ARG without a workspace.
 */
dsa_status_t dsa_selftest_timeout(void* workspace, size_t workspace_bytes, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H_ */
