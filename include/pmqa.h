/*
 * pmqa.h -- C ABI of libpmqa: the FP8 paged MQA-logits indexer and its per-row
 * top-k, the non-paged (prefill) MQA logits, and the sparse MLA decode that
 * consumes the top-k positions, as hand-written CUDA kernels for sm_103a
 * (GB300).
 *
 * What is computed. Sources: the page "[Bug] aiter ops triton attention pa"
 * (stepcodex.com issue mirror), section "Minimal reproduction" (the reference
 * function `torch_ref` and the `test` driver); the page "[Bugfix][Hardware][AMD]
 * Fix last_page_len calculation in AITER MLA decode" (vLLM PR 31282), section
 * "Comparison with Other Backends" (tokens held by a request's last page).
 *
 *   For request i < bs, draft row j < next_n (row r = i*next_n + j) and
 *   logical token t:
 *     valid(r, t)  <=>  t < ctx_i  and  t <= ctx_i - next_n + j
 *     phys         =   block_tables[i][t / P] * P + t % P
 *     k_t          =   kv_cache[phys][0..127] as fp8 e4m3fn
 *     s_t          =   fp32 whose little-endian bytes are kv_cache[phys][128..131]
 *     logits[r][t] =   sum_h weights[r][h] * relu(s_t * dot(q[i][j][h], k_t))
 *                      if valid(r, t), else -inf, for 0 <= t < max_model_len
 *   Top-k of row r: the positions of the min(k, valid_len(r)) largest logits
 *   among t < valid_len(r) = clamp(ctx_i - next_n + j + 1, 0, ctx_i); remaining
 *   slots hold -1. The order of positions within a row is unspecified; among
 *   equal values any choice is returned. The last page of a request holds
 *   ((ctx_i - 1) mod P) + 1 tokens; its other slots are never read.
 *
 * Memory. Every pointer is a DEVICE pointer owned by the caller. The library
 * allocates nothing, keeps no global state between calls (the one exception is
 * the built-in scratch of pmqa_logits_topk_noalloc), never synchronises the
 * stream (except pmqa_read_device_status) and enqueues its work on the given
 * stream. Calls that share one workspace must not overlap on the GPU.
 *
 * Errors. Functions return PMQA_OK (0) or a negative PMQA_ERR_* code; on an
 * error nothing has been enqueued. Faults the host cannot see (a block table
 * entry outside the pool, a context longer than max_model_len or than the
 * table covers, a pipeline wait that ran out) never trap: the kernel skips the
 * access (a bad table entry reads as zeros), records a PMQA_DEV_* bit in the
 * workspace status word and finishes; pmqa_read_device_status reports it.
 */
#ifndef PMQA_H
#define PMQA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st *pmqa_stream_t;

enum {
    PMQA_OK = 0,
    PMQA_ERR_INVALID_ARG = -1,  /* null pointer, negative size, misalignment, k < 1 */
    PMQA_ERR_UNSUPPORTED = -2,  /* head_dim != 128, heads not in {16,32,64,128},
                                   next_n not in 1..4, k too large for the kernel */
    PMQA_ERR_WORKSPACE = -3,    /* workspace smaller than pmqa_workspace_bytes */
    PMQA_ERR_CUDA = -4,         /* a CUDA runtime call or a launch failed */
    PMQA_ERR_DEVICE = -5        /* reported by pmqa_read_device_status only */
};

/* Bits of the device status word. */
#define PMQA_DEV_BAD_BLOCK_ID 0x1u /* a block table entry outside [0, num_blocks) */
#define PMQA_DEV_BAD_CONTEXT 0x2u  /* ctx < 0, ctx > max_model_len, or ctx > P * max_blocks_per_seq;
                                      the kernel clamps it */
#define PMQA_DEV_TIMEOUT 0x4u      /* a pipeline wait exceeded its limit; results are invalid */
#define PMQA_DEV_OVERFLOW 0x8u     /* top-k candidate storage exceeded; results are invalid */
#define PMQA_DEV_INTERNAL 0x10u    /* a kernel found its shared memory misaligned and did no work;
                                      results are invalid */
#define PMQA_DEV_SCORE_RANGE 0x20u /* an attention score out of range; its row's result is invalid */

/* Workspace-size selector for pmqa_workspace_bytes. For PMQA_OP_MQA_LOGITS (the
   prefill entry point) bs is the number of query rows m and the other sizes
   are ignored. */
enum { PMQA_OP_LOGITS = 0, PMQA_OP_TOPK = 1, PMQA_OP_LOGITS_TOPK = 2, PMQA_OP_MQA_LOGITS = 3 };

/*
 * One decode-step problem, in the argument order of the reference function
 * (q, kv_cache, weights, context_lens, block_tables, max_model_len) plus sizes.
 *   q             fp8 e4m3fn [bs, next_n, heads, head_dim], contiguous, 16-byte aligned
 *   kv_cache      uint8 [num_blocks, block_size, head_dim + 4], contiguous, 16-byte
 *                 aligned (rows are read as 16-byte aligned windows): per token
 *                 head_dim fp8 bytes then a little-endian fp32 scale
 *   weights       fp32 [bs * next_n, heads], contiguous, 16-byte aligned
 *   context_lens  int32 [bs]
 *   block_tables  int32 [bs, max_blocks_per_seq], row-major; only the first
 *                 ceil(ctx_i / block_size) entries of row i are read
 */
typedef struct pmqa_problem {
    const void *q;
    const void *kv_cache;
    const float *weights;
    const int32_t *context_lens;
    const int32_t *block_tables;
    int32_t bs;
    int32_t next_n;
    int32_t heads;
    int32_t head_dim;
    int32_t block_size;
    int32_t max_blocks_per_seq;
    int32_t max_model_len;
    int64_t num_blocks;
} pmqa_problem;

/*
 * Bytes of device workspace an operation needs for rows = bs * next_n rows of
 * width max_model_len and top-k size k (k is ignored for PMQA_OP_LOGITS).
 * Returns 0 for invalid arguments. The workspace must be 256-byte aligned and
 * zero-filled before its first use (pmqa_workspace_init); every call leaves it
 * zero-filled again except for the status word.
 */
size_t pmqa_workspace_bytes(int32_t bs, int32_t next_n, int32_t max_model_len, int32_t k, int op);

/* Zero-fill a workspace (cudaMemsetAsync on the stream). */
int pmqa_workspace_init(void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * Logits, the definition above. logits: fp32 [bs * next_n, max_model_len],
 * 4-byte aligned; every entry of every row is written (-inf outside the mask),
 * so no caller pre-fill is needed.
 */
int pmqa_logits(const pmqa_problem *p, float *logits, void *ws, size_t ws_bytes,
                pmqa_stream_t stream);

/*
 * Per-row top-k of existing logits rows. logits: fp32 [bs * next_n, max_model_len];
 * only t < valid_len(r) is read (entries beyond are ignored whatever they hold).
 * idx: int32 [bs * next_n, k], -1 past min(k, valid_len(r)).
 * vals: fp32 [bs * next_n, k] or NULL; the logits at idx (-inf where idx is -1).
 */
int pmqa_topk(const float *logits, const int32_t *context_lens, int32_t bs, int32_t next_n,
              int32_t max_model_len, int32_t k, int32_t *idx, float *vals, void *ws,
              size_t ws_bytes, pmqa_stream_t stream);

/*
 * Fused logits + top-k in one pass over the KV cache: the logits rows need not
 * be written to memory. idx and vals as for pmqa_topk; logits may be NULL, or
 * a [bs * next_n, max_model_len] buffer that then receives the full logits.
 */
int pmqa_logits_topk(const pmqa_problem *p, int32_t k, int32_t *idx, float *vals, float *logits,
                     void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * pmqa_logits_topk in its two kernel launches, for callers that schedule or
 * time them apart. stages: PMQA_STAGE_SCORE (the KV pass: logits into the
 * workspace, or into logits when given, plus one key histogram per row),
 * PMQA_STAGE_SELECT (the per-row selection from that state, which also clears
 * it), or both (= pmqa_logits_topk). A SELECT call must follow the SCORE call
 * with the same arguments and workspace, with no other call on that workspace
 * in between; arguments are checked as for pmqa_logits_topk. The pages have no
 * counterpart: the split is the fused call's own launch boundary.
 */
enum { PMQA_STAGE_SCORE = 1, PMQA_STAGE_SELECT = 2 };
int pmqa_logits_topk_stages(const pmqa_problem *p, int32_t k, int32_t *idx, float *vals,
                            float *logits, void *ws, size_t ws_bytes, pmqa_stream_t stream,
                            int32_t stages);

/*
 * pmqa_logits_topk without a caller-supplied workspace. The pages have no
 * counterpart to this entry point: it exists for callers that are given device
 * buffers for their inputs and outputs but cannot allocate device memory of
 * their own (for example a plugin inside a host program that owns the whole
 * device-memory pool and offers no allocation hook, or a latency-critical loop
 * that must not call cudaMalloc, which may synchronise the device).
 * The workspace is a 32 MiB array that the library keeps in device memory on
 * every GPU where it is loaded, until the process exits. Problems whose
 * pmqa_workspace_bytes(bs, next_n, max_model_len, k, PMQA_OP_LOGITS_TOPK)
 * exceeds 32 MiB return PMQA_ERR_WORKSPACE with nothing enqueued: that size is
 * 12 bytes per (row, position) -- an 8-byte candidate entry and a 4-byte
 * compact logit -- plus 8 KB of histogram and 12 bytes of counters per row and
 * 256 bytes of status, so for example 16 rows of 131072 positions fit and 16
 * rows of 202752 do not.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before capturing
 * any stream. Every call shares the one array and clears its counters at the
 * start, so calls that overlap on the GPU (other streams, other threads) race
 * and must be serialised by the caller. Device-side status bits of these calls
 * are not reported. Allocates nothing: no cudaMalloc, cudaFree or allocating
 * library call.
 */
int pmqa_logits_topk_noalloc(const pmqa_problem *p, int32_t k, int32_t *idx, float *vals,
                             float *logits, pmqa_stream_t stream);

/*
 * The fused call restricted to a slice of every request's tokens: request i
 * scores only tokens token_begin[i] <= t < token_end[i] (device int32 [bs]
 * each, clamped to [0, ctx_i]; an empty slice scores nothing), with the
 * request's full context for the causal window, and selects per row the
 * positions (global t) of the min(k, admitted tokens of the slice) largest
 * logits; idx and vals as for pmqa_logits_topk. The block table is read only
 * for pages that hold tokens of the slice, so a GPU that keeps only its
 * slice's pages may leave the other entries unset. This is the per-GPU step
 * of a context-parallel split, whose lists pmqa_topk_merge combines; a call on
 * the whole range [0, ctx_i) equals pmqa_logits_topk. Workspace as for
 * PMQA_OP_LOGITS_TOPK; two kernel launches, as pmqa_logits_topk.
 */
int pmqa_logits_topk_range(const pmqa_problem *p, const int32_t *token_begin,
                           const int32_t *token_end, int32_t k, int32_t *idx, float *vals,
                           void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * Top-k of the union of candidate lists, per row: the merge step of a
 * context-parallel split of the indexer, in which each GPU holds a slice of
 * every request's tokens, scores it (pmqa_logits_topk_range) and keeps the
 * slice's top-k positions and logits; the lists are gathered from the GPUs
 * (an all-gather) and merged here. Every one of a row's k largest logits lies
 * in its own slice's top-k, so the union's top-k is the row's top-k. The pages
 * name decode context parallelism (DCP) among the configurations of the
 * sparse-MLA decode path (page "[Bug][ROCm]: ROCM_AITER_MLA can select an aiter
 * MLA decode kernel that silently returns uncorrelated output", chat-gpts.plus
 * summary, closing notes); the split and this merge are the library's design.
 *   idx       int32 [lists, rows, k_in]: positions, -1 for an empty slot (skipped)
 *   vals      fp32 [lists, rows, k_in]: their logits
 *   out_idx   int32 [rows, k]: the positions of the min(k, valid candidates)
 *             largest logits (order unspecified, ties either way), then -1
 *   out_vals  fp32 [rows, k] or NULL: their logits, then -inf
 * A position may appear in at most one of a row's lists. lists * k_in < 2^31
 * (PMQA_ERR_UNSUPPORTED otherwise). No workspace; one kernel launch.
 */
int pmqa_topk_merge(const int32_t *idx, const float *vals, int32_t lists, int32_t rows,
                    int32_t k_in, int32_t k, int32_t *out_idx, float *out_vals,
                    pmqa_stream_t stream);

/*
 * Prefill (non-paged) logits. Source: the page "[Bug] aiter ops triton
 * attention pa", section "Observations while narrowing it down", which names
 * the prefill indexer `fp8_mqa_logits` (heads 32, head_dim 128, up to 8192 keys,
 * query lengths up to 4096) beside the paged decode kernel. The pages give only
 * its name and shapes; it is read as the decode definition with the paging
 * removed and one key range per query row:
 *   logits[r][t] = sum_h weights[r][h] * relu(k_scale[t] * dot(q[r][h], k_t))
 *                  for max(ks[r], 0) <= t < min(ke[r], n), else -inf,
 * for every query row r < m and key t < n.
 *   q        fp8 e4m3fn [m, heads, head_dim], contiguous, 16-byte aligned
 *   k        fp8 e4m3fn [n, head_dim], contiguous, 16-byte aligned
 *   k_scale  fp32 [n], 4-byte aligned
 *   weights  fp32 [m, heads], contiguous, 16-byte aligned
 *   ks, ke   int32 [m]: row r's key range [ks[r], ke[r]); values outside [0, n]
 *            are clamped, ks >= ke gives an all -inf row
 * head_dim must be 128 and heads one of 16, 32, 64, 128; m * heads < 2^31 and
 * n <= 2^31 - 129 (PMQA_ERR_UNSUPPORTED otherwise).
 */
typedef struct pmqa_mqa_problem {
    const void *q;
    const void *k;
    const float *k_scale;
    const float *weights;
    const int32_t *ks;
    const int32_t *ke;
    int32_t m;
    int32_t n;
    int32_t heads;
    int32_t head_dim;
} pmqa_mqa_problem;

/*
 * logits: fp32 [m, n], 4-byte aligned; every entry is written. ws: at least
 * pmqa_workspace_bytes(m, 1, n, 0, PMQA_OP_MQA_LOGITS) bytes (256 + 8 per 4
 * query rows, rounded up to 256), 256-byte aligned, zero-filled before first
 * use; it holds the status word (a pipeline wait that ran out sets
 * PMQA_DEV_TIMEOUT) and per-call scratch. Two kernel launches.
 */
int pmqa_mqa_logits(const pmqa_mqa_problem *p, float *logits, void *ws, size_t ws_bytes,
                    pmqa_stream_t stream);

/*
 * Sparse MLA decode over the indexer's top-k positions: the attention step of
 * the same decode step, which attends only to the positions the top-k
 * selected. Sources: the page "[Bug] aiter ops triton attention pa", section
 * "Downstream impact" (the sparse MLA attention attends to the indexer's top-k
 * positions); the page "[Bug][ROCm]: ROCM_AITER_MLA can select an aiter MLA
 * decode kernel that silently returns uncorrelated output" (chat-gpts.plus
 * summary: fp8 Q and fp8 KV, 16 query heads per latent KV head, 1..4 query
 * rows per request, a log-sum-exp output for decode context parallelism); the
 * page "[Bugfix][Hardware][AMD] Fix last_page_len calculation in AITER MLA
 * decode", section "The Bug" (the MLA cache in pages of one token; larger
 * pages use the same lookup). The pages give no widths: a cached token is one
 * latent row of 576 fp8 values whose first 512 are its value vector (the MLA
 * layout of a 512-wide compressed KV plus a 64-wide rotary key), and q and the
 * cache carry one fp32 scale each.
 *
 *   For query row r = i*next_n + j, head h and each listed position t of row r
 *   (indices[r][e] >= 0; a position listed twice counts twice):
 *     phys    = block_tables[i][t / block_size] * block_size + t % block_size
 *     s_t     = sm_scale * sum_d (q_scale * q[r][h][d]) * (kv_scale * kv[phys][d]),  d < 576
 *     out[r][h][d] = sum_t softmax(s)_t * kv_scale * kv[phys][d],   d < 512
 *     lse[r][h]    = ln sum_t exp(s_t)
 *   A row with no listed position gives out = 0 and lse = -inf.
 *
 *   q             fp8 e4m3fn [bs * next_n, heads, head_dim], contiguous, 16-byte aligned
 *   kv_cache      fp8 e4m3fn [num_blocks, block_size, head_dim], contiguous,
 *                 16-byte aligned; only the rows of listed positions are read
 *   indices       int32 [bs * next_n, topk]: positions in the row's request
 *                 (what pmqa_logits_topk returns), -1 for an empty entry
 *   block_tables  int32 [bs, max_blocks_per_seq], row-major
 * heads must be 16, head_dim 576 and v_head_dim 512 (PMQA_ERR_UNSUPPORTED
 * otherwise); the scales must be finite.
 */
typedef struct pmqa_mla_problem {
    const void *q;
    const void *kv_cache;
    const int32_t *indices;
    const int32_t *block_tables;
    float q_scale;
    float kv_scale;
    float sm_scale;
    int32_t bs;
    int32_t next_n;
    int32_t heads;
    int32_t head_dim;
    int32_t v_head_dim;
    int32_t topk;
    int32_t block_size;
    int32_t max_blocks_per_seq;
    int64_t num_blocks;
} pmqa_mla_problem;

/* Bytes of workspace for pmqa_sparse_mla_decode over `rows` query rows (about
   17 MB, whatever the row count); 0 for rows < 0. */
size_t pmqa_sparse_mla_workspace_bytes(int32_t rows);

/*
 * out: bf16 [bs * next_n, heads, 512], 4-byte aligned; lse: fp32
 * [bs * next_n, heads] or NULL. ws: pmqa_sparse_mla_workspace_bytes(rows)
 * bytes, 256-byte aligned, its status word zero before the first use
 * (pmqa_workspace_init). A listed position past the block table sets
 * PMQA_DEV_BAD_CONTEXT, a table entry outside [0, num_blocks)
 * PMQA_DEV_BAD_BLOCK_ID (the position is then skipped); a pipeline wait that
 * ran out sets PMQA_DEV_TIMEOUT (results invalid). Two kernel launches: the
 * attention, and the combination of rows whose tiles were split over CTAs.
 */
int pmqa_sparse_mla_decode(const pmqa_mla_problem *p, void *out, float *lse, void *ws,
                           size_t ws_bytes, pmqa_stream_t stream);

/*
 * The decode restricted to a slice of every request's tokens: request i's rows
 * attend only to their listed positions t with token_begin[i] <= t <
 * token_end[i] (device int32 [bs] each); the other listed positions are
 * skipped, so the block table need only map the slice's pages. This is one
 * GPU's step of a decode split by context (decode context parallelism: the
 * chat-gpts.plus summary names an LSE output for it): the slices' outputs and
 * log-sum-exps are gathered and combined by pmqa_sparse_mla_merge. Otherwise
 * as pmqa_sparse_mla_decode; a row with no position in its slice gives out = 0
 * and lse = -inf.
 */
int pmqa_sparse_mla_decode_range(const pmqa_mla_problem *p, const int32_t *token_begin,
                                 const int32_t *token_end, void *out, float *lse, void *ws,
                                 size_t ws_bytes, pmqa_stream_t stream);

/*
 * Merge of `parts` partial decodes of the same rows (each over a disjoint part
 * of every row's listed positions, e.g. the slices of a context split):
 *   outs  bf16 [parts, rows, heads, 512]; lses fp32 [parts, rows, heads]
 *   out   bf16 [rows, heads, 512] = sum_g w_g outs[g] / sum_g w_g,
 *         w_g = exp(lses[g] - max_g lses[g]) (a part with lse -inf weighs 0)
 *   lse   fp32 [rows, heads] or NULL: max_g lses[g] + ln sum_g w_g
 * heads must be 16. No workspace; one kernel launch.
 */
int pmqa_sparse_mla_merge(const void *outs, const float *lses, int32_t parts, int32_t rows,
                          int32_t heads, void *out, float *lse, pmqa_stream_t stream);

/*
 * A paged K/V cache held in 8 bits, and four operators on it: append a step's
 * new tokens, attend to the cached ones, add up the attention weight that each
 * cached token received, and keep the tokens with the most of it in fewer
 * blocks. It serves the layers (or models) that keep ordinary keys and values
 * beside the indexed latent cache of the sparse layers; the source pages have no
 * counterpart.
 *
 *   k_cache, v_cache  fp8 e4m3fn [num_blocks, kv_heads, block_size, head_dim],
 *                 contiguous, 16-byte aligned: a block holds block_size
 *                 consecutive tokens of one request
 *   k_scale, v_scale  fp32 [num_blocks, kv_heads]: one scale per block and head;
 *                 a cached value is its code times its scale
 *   block_tables  int32 [bs, max_blocks_per_seq], row-major; only the first
 *                 ceil(ctx_i / block_size) entries of row i are read
 *   context_lens  int32 [bs]: ctx_i, tokens of request i, this call's new ones
 *                 included
 *   row_begin     int32 [bs + 1], not decreasing, within [0, rows]: request i
 *                 has the n_i = row_begin[i + 1] - row_begin[i] <= max_rows rows
 *                 from row_begin[i] on; its row j sits at slot
 *                 ctx_i - n_i + j and sees the slots t <= ctx_i - n_i + j.
 *                 Rows of no request are neither read nor written; max_rows is at
 *                 least 1. Unused by pmqa_cache_evict (as are rows and max_rows).
 * head_dim must be 64 or 128, block_size at most 1024, kv_heads at most 65535,
 * num_blocks * kv_heads * block_size < 2^32 - 1 (PMQA_ERR_UNSUPPORTED otherwise).
 * A context outside [0, block_size * max_blocks_per_seq] or above 2^31 - 2^16, or
 * rows that break the rules above, are clamped and set
 * PMQA_DEV_BAD_CONTEXT; a table entry outside [0, num_blocks) sets
 * PMQA_DEV_BAD_BLOCK_ID, and its tokens are left out (not written by append,
 * not attended to or weighed, zeros where evict would have moved them).
 *
 * Every call takes a workspace of pmqa_cache_workspace_bytes() bytes, 256-byte
 * aligned, its status word zero before the first use (pmqa_workspace_init). Outputs
 * overlap no input and no other output unless a call says so.
 */
typedef struct pmqa_cache_problem {
    void *k_cache;
    void *v_cache;
    float *k_scale;
    float *v_scale;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *row_begin;
    int32_t bs;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t block_size;
    int32_t max_blocks_per_seq;
    int32_t rows;
    int32_t max_rows;
    int64_t num_blocks;
} pmqa_cache_problem;

/* About 32 MB, whatever the problem. */
size_t pmqa_cache_workspace_bytes(void);

/*
 * Quantise a call's new tokens into their blocks. k, v: bf16 [rows, kv_heads,
 * head_dim], 16-byte aligned, already rotated where the model rotates. With
 * e(a) = 2^ceil(log2(a / 448)), at least 2^-100, the new scale of a touched
 * block and head (keys and values apart) is
 *   s' = max(s, e(a)) if the block holds earlier tokens of the request, else e(a),
 * a the largest finite |value| the call writes there; where s' != s the earlier
 * codes c become rne(c s / s'), and a new value x is stored as rne(x / s'),
 * saturated at 448 (NaN stays NaN). Slots behind ctx_i and blocks without a new
 * token are left as they were. A block that receives tokens must belong to one
 * request only. Lengths out of range drop rows and move none: row j's slot is
 * ctx_i - n_i + j from the lengths as given, and rows whose slot is negative or
 * behind the table's last, rows past the first max_rows and rows outside [0, rows) are
 * not written (PMQA_DEV_BAD_CONTEXT). One kernel launch.
 */
int pmqa_cache_append(const pmqa_cache_problem *p, const void *k, const void *v, void *ws,
                      size_t ws_bytes, pmqa_stream_t stream);

/*
 * Attention of every row to the slots that it sees, query head hq with kv head
 * h = hq / (heads / kv_heads):
 *   s_t = sm_scale * q . k_t,  out = sum_t softmax(s)_t v_t,  lse = ln sum_t exp(s_t)
 *   q    bf16 [rows, heads, head_dim], 16-byte aligned
 *   out  bf16 [rows, heads, head_dim], 16-byte aligned
 *   lse  fp32 [rows, heads] or NULL
 * heads must be a multiple of kv_heads, at most 128 times kv_heads, and
 * max_rows * heads < 2^31. A row that sees no slot gives out = 0 and lse = -inf.
 * sm_scale must be finite (times log2(e) too). A row of q with an infinite or NaN value
 * gives NaN. A NaN among a block's values (v) makes that column NaN
 * for every row of the request that the block's other tokens reach, rows that do
 * not see the NaN's token among them; a NaN key reaches only the rows that see it.
 * Requests of more than 32 rows n_i * heads / kv_heads take q as the sum of two 8-bit
 * terms, exact where a value is at least 2^-13 of its row's largest and off by at
 * most 2^-21 of that below (fewer rows: exact from 2^-31 on); weigh does the same.
 * They hold their values (code * scale) to 2^-31 of the largest block scale met so
 * far; by 2^-11 of themselves where two scales' quotient is no power of two. Fewer
 * rows hold the weight times the scale, to 2^-25 (2^-11 of itself above 2^-14) of the
 * largest scale among 32 tokens, or of one up to 32 times as large. Value scales
 * below 1e-36 count as 0.
 * One kernel launch where block_size * max_blocks_per_seq <= 640, else two, and
 * one or two more where max_rows * heads / kv_heads > 32 (those alone where
 * heads / kv_heads > 32).
 * Every sum is formed in one order: equal calls give equal bits.
 */
int pmqa_cache_attention(const pmqa_cache_problem *p, const void *q, int32_t heads, float sm_scale,
                         void *out, float *lse, void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * The weight each cached token received: for t < ctx_i (and t < mass_width)
 *   mass_out[i][h][t] = mass_in[i][h][t] + sum of exp(sm_scale * q_(j,hq) . k_t - lse[j][hq])
 * over request i's rows j that see t and the query heads hq of kv head h; other
 * entries are not written. q, heads and sm_scale as in the attention call whose
 * lse this is; v_cache and v_scale are not read and may be NULL.
 *   mass_in   fp32 [bs, kv_heads, mass_width] or NULL (zeros); may be mass_out, but
 *             must not overlap it otherwise
 *   mass_out  fp32 [bs, kv_heads, mass_width]
 * Every sum is formed in one order: equal calls give equal bits. One kernel
 * launch, two where max_rows * heads / kv_heads > 32.
 */
int pmqa_cache_weigh(const pmqa_cache_problem *p, const void *q, int32_t heads, float sm_scale,
                     const float *lse, const float *mass_in, float *mass_out, int64_t mass_width,
                     void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * Keep min(ctx_i, keep) tokens of every request and kv head, each head its own,
 * in new blocks. A request with ctx_i <= keep keeps all; otherwise its first
 * `sinks` and last `recent` tokens stay, and of those between, the
 * keep - sinks - recent with the largest mass (equal masses: the lower slot;
 * NaN lowest). Their order is kept, so token n of the new context is slot
 * kept[i][h][n] of the old one.
 *   mass        fp32 [bs, kv_heads, mass_width]; ctx_i must not exceed mass_width
 *   new_tables  int32 [bs, new_blocks_per_seq], new_blocks_per_seq * block_size >=
 *               keep: the blocks that receive the kept tokens, in the same pools;
 *               the first ceil(min(ctx_i, keep) / block_size) of row i are used.
 *               None of them may be in use by block_tables or listed twice
 *   kept        int32 [bs, kv_heads, keep]: old slots in rising order, then -1
 *   lens_out    int32 [bs]: min(ctx_i, keep); must not overlap context_lens
 *   mass_out    fp32 [bs, kv_heads, mass_width] or NULL: the kept tokens' masses,
 *               then zeros; must not overlap mass
 * A new block's scale is e(largest |code * scale| moved there) (see append), its
 * codes rounded to it; slots past the new length are left as they were. Masks by
 * slot keep their meaning after it: a request's last `recent` tokens are still
 * its last. sinks + recent <= keep. Two kernel launches.
 */
int pmqa_cache_evict(const pmqa_cache_problem *p, const float *mass, int64_t mass_width, int32_t keep,
                     int32_t sinks, int32_t recent, const int32_t *new_tables,
                     int32_t new_blocks_per_seq, int32_t *kept, int32_t *lens_out, float *mass_out,
                     void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * Around the sparse-MLA step: what rotates queries and keys, what writes the
 * indexer's cache and the latent cache with the step's queries beside them, what
 * gives cached indexer keys back, and the attention that reads all of a latent
 * cache. The source pages start from caches and queries that exist; these calls
 * make them from a model's projections (bf16).
 *
 * Rows of a step, and where their tokens lie in a paged cache of num_blocks
 * blocks of block_size tokens:
 *   block_tables  int32 [bs, max_blocks_per_seq], row-major
 *   context_lens  int32 [bs]: ctx_i, tokens of request i, this step's included
 *   row_begin     int32 [bs + 1], not decreasing, within [0, rows]: request i has
 *                 the n_i = row_begin[i + 1] - row_begin[i] <= max_rows rows from
 *                 row_begin[i] on; its row j is the token at slot ctx_i - n_i + j.
 *                 Rows of no request are neither read nor written
 * bs * max_blocks_per_seq < 2^31 and num_blocks * block_size < 2^32 - 1
 * (PMQA_ERR_UNSUPPORTED otherwise). Lengths that break the rules, and rows whose
 * slot is negative or behind the table's last, set PMQA_DEV_BAD_CONTEXT; a table
 * entry outside [0, num_blocks) sets PMQA_DEV_BAD_BLOCK_ID.
 */
typedef struct pmqa_paged_rows {
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *row_begin;
    int32_t bs;
    int32_t block_size;
    int32_t max_blocks_per_seq;
    int32_t rows;
    int32_t max_rows;
    int64_t num_blocks;
} pmqa_paged_rows;

/*
 * Rotary positions. Of each head the values begin .. begin + dim are rotated in
 * dim / 2 pairs: pair i is (x_i, x_{i + dim/2}), or (x_{2i}, x_{2i+1}) with
 * `interleaved`, and with theta = position * inv_freq[i]
 *   a' = scale * (a cos theta - b sin theta),  b' = scale * (b cos theta + a sin theta)
 * The angle is formed modulo a turn in 64-bit fixed point: no accuracy is lost at
 * far positions. Negative positions turn back.
 *   inv_freq   fp64 [dim / 2], device: radians per position (pmqa_rope_frequencies)
 *   positions  int32 [rows], or NULL where a call has slots: the row's slot
 * dim a multiple of 16 (0: nothing is rotated, the pointers are not used), begin a
 * multiple of 8, begin + dim at most the head's width, scale finite.
 */
typedef struct pmqa_rotary {
    const double *inv_freq;
    const int32_t *positions;
    int32_t dim;
    int32_t begin;
    int32_t interleaved;
    float scale;
} pmqa_rotary;

/*
 * Frequencies base^(-2 i / dim), i < dim / 2, for contexts `factor` (>= 1) times as
 * long as the `trained` positions, written to host memory, and the scale that
 * belongs to them:
 *   PMQA_ROPE_PLAIN   as they are (factor and trained unused); scale 1
 *   PMQA_ROPE_LINEAR  all divided by factor; scale 1
 *   PMQA_ROPE_PARTS   divided where a pair turns fewer than slow_turns times over the
 *                     trained positions, kept where more than fast_turns times, and
 *                     between the two weighted linearly in i (the ends rounded
 *                     outwards to whole i, within 0 to dim - 1); scale 0.1 ln(factor) + 1
 * A host function: no device work. dim even and positive, base > 1; for PARTS
 * trained >= 1 and 0 < slow_turns < fast_turns.
 */
enum { PMQA_ROPE_PLAIN = 0, PMQA_ROPE_LINEAR = 1, PMQA_ROPE_PARTS = 2 };
int pmqa_rope_frequencies(int32_t dim, double base, int kind, double factor, double trained,
                          double slow_turns, double fast_turns, double *inv_freq, float *scale);

/*
 * Heads of bf16 values to rotate: element d of head h of row r at
 * x + r * x_row + h * x_head + d (strides in elements, multiples of 8), the result
 * at out likewise; both 16-byte aligned. out may be x (with the same strides: the
 * values outside the rotated part are then not touched); their spans overlap
 * otherwise nowhere. Two results never share an element, nor does one tensor's result
 * with the other's input.
 */
typedef struct pmqa_heads {
    const void *x;
    void *out;
    int64_t x_row;
    int64_t x_head;
    int64_t out_row;
    int64_t out_head;
    int32_t heads;
    int32_t head_dim;
} pmqa_heads;

/*
 * Rotate the heads of a, and of b unless NULL (queries and keys of one step), at
 * rotary->positions; values outside the rotated part are copied. Products and
 * sums in fp32, one rounding to bf16. head_dim a multiple of 8, at most 1024, the
 * heads of a and b together at most 2^24 (PMQA_ERR_UNSUPPORTED otherwise). One
 * kernel launch.
 */
int pmqa_rope(const pmqa_rotary *rotary, int32_t rows, const pmqa_heads *a, const pmqa_heads *b,
              pmqa_stream_t stream);

/*
 * Normalisation of a row before it is rotated or quantised, in fp32:
 *   PMQA_NORM_LAYER  (x - mean) / sqrt(var + eps)     PMQA_NORM_RMS  x / sqrt(mean(x^2) + eps)
 * times weight, plus bias (fp32, 16-byte aligned, of the row's width, NULL for 1 and
 * 0; unused with PMQA_NORM_NONE). eps >= 0 and finite.
 */
enum { PMQA_NORM_NONE = 0, PMQA_NORM_LAYER = 1, PMQA_NORM_RMS = 2 };
typedef struct pmqa_norm {
    int32_t kind;
    float eps;
    const float *weight;
    const float *bias;
} pmqa_norm;

/*
 * The indexer's inputs of a step, from the projections.
 *   keys     k: bf16 [rows, 128], row r at k + r * k_row. Normalised (norm),
 *            rotated, and written to the row's slot of kv_cache (pmqa_problem) as 128
 *            codes rne(k' / s) and the fp32 scale s = max(a, 2^-100) / 448, a the
 *            largest finite |k'|; infinite values saturate, NaN stays NaN. (The
 *            quotient is k' times 448 / a, each in fp32: within 2^-21 of it)
 *   queries  q: bf16 [rows, heads, 128], head h of row r at q + r * q_row + h * q_head;
 *            rotated and quantised alike, each head with its own scale s, which goes
 *            into the head's weight:
 *              weights_out[r][h] = weights[r][h] * s * weight_scale
 *            so that q_out and weights_out are what pmqa_logits, pmqa_logits_topk and
 *            pmqa_mqa_logits take. weights: fp32 (bf16 with weights_bf16) [rows,
 *            heads], row r at weights + r * weights_row
 *   q_out    fp8 [rows, heads, 128], weights_out fp32 [rows, heads]
 * k or q may be NULL: then there is no key to write, or there are no queries (and
 * weights, q_out and weights_out are not used). k, q and their strides: 16-byte
 * aligned, multiples of 8 elements; q_out 8-byte aligned; heads at most 65535 and
 * rows * heads < 2^31 (PMQA_ERR_UNSUPPORTED otherwise). weights_out may be
 * weights (fp32, weights_row = heads); outputs overlap nothing else.
 */
typedef struct pmqa_index_rows {
    const void *k;
    const void *q;
    const void *weights;
    void *q_out;
    float *weights_out;
    int64_t k_row;
    int64_t q_row;
    int64_t q_head;
    int64_t weights_row;
    int32_t heads;
    int32_t weights_bf16;
    float weight_scale;
} pmqa_index_rows;

/*
 * kv_cache: uint8 [num_blocks, block_size, 132], 4-byte aligned. A slot that
 * receives a key belongs to one request only; other slots are left as they were.
 * Rows past their request's first max_rows are not processed; a row without a slot
 * writes no key. norm and rotary may be NULL (none). ws: any workspace of this
 * library (256 bytes are enough); only its status word is used. One kernel launch.
 */
int pmqa_index_append(const pmqa_paged_rows *p, void *kv_cache, const pmqa_index_rows *x,
                      const pmqa_norm *norm, const pmqa_rotary *rotary, void *ws, size_t ws_bytes,
                      pmqa_stream_t stream);

/*
 * Cached indexer keys as contiguous rows, the form that pmqa_mqa_logits takes: row
 * row_begin[i] + j is the token at slot start[i] + j of request i (start: int32
 * [bs], or NULL for zeros); p->context_lens and p->max_rows are not used, rows of no
 * request are left as they were, rows without a slot or with a bad table entry give
 * zeros (a code and a scale of 0).
 *   k        fp8 [rows, 128], 16-byte aligned
 *   k_scale  fp32 [rows]
 * One kernel launch; ws as for pmqa_index_append.
 */
int pmqa_index_read(const pmqa_paged_rows *p, const void *kv_cache, const int32_t *start, void *k,
                    float *k_scale, void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * The latent rows and queries of a step, in the form of pmqa_sparse_mla_decode and
 * pmqa_latent_attention: a row is 512 latent values and 64 rotary ones.
 *   keys     c: bf16 [rows, 512] (row r at c + r * c_row), normalised (norm), and k_pe:
 *            bf16 [rows, 64] (stride pe_row), rotated; written to the row's slot of
 *            the latent cache as rne(x / kv_scale), saturated at 448 (NaN stays NaN)
 *   queries  q_c: bf16 [rows, heads, 512] (the query carried into the latent space)
 *            and q_pe: bf16 [rows, heads, 64], rotated; q_out: fp8 [rows, heads, 576],
 *            rne(x / q_scale), saturated
 * (x / scale is x times the scale's fp32 reciprocal.) c or q_c may be NULL, as in
 * pmqa_index_append. Strides in elements, multiples of 8; inputs 16-byte, outputs
 * 8-byte aligned; the scales finite, with finite reciprocals; heads as there.
 */
typedef struct pmqa_latent_rows {
    const void *c;
    const void *k_pe;
    const void *q_c;
    const void *q_pe;
    void *q_out;
    int64_t c_row;
    int64_t pe_row;
    int64_t q_c_row;
    int64_t q_c_head;
    int64_t q_pe_row;
    int64_t q_pe_head;
    int32_t heads;
    float kv_scale;
    float q_scale;
} pmqa_latent_rows;

/* kv_cache: fp8 [num_blocks, block_size, 576], 8-byte aligned. The rest as for
   pmqa_index_append. */
int pmqa_latent_append(const pmqa_paged_rows *p, void *kv_cache, const pmqa_latent_rows *x,
                       const pmqa_norm *norm, const pmqa_rotary *rotary, void *ws, size_t ws_bytes,
                       pmqa_stream_t stream);

/* About 41 MB, whatever the problem. */
size_t pmqa_latent_workspace_bytes(void);

/*
 * Attention of every row to all the cached tokens that it sees, the slots t <=
 * ctx_i - n_i + j: the dense form of pmqa_sparse_mla_decode, for any number of
 * heads and for prompts.
 *   s_t = sm_scale * (q_scale * q_h) . (kv_scale * kv_t),  out = sum_t softmax(s)_t v_t,
 *   v_t = kv_scale * kv_t[0..511],  lse = ln sum_t exp(s_t)
 *   q         fp8 e4m3fn [rows, heads, 576], 16-byte aligned
 *   kv_cache  fp8 e4m3fn [num_blocks, block_size, 576], 16-byte aligned
 *   out       bf16 [rows, heads, 512], 16-byte aligned; lse fp32 [rows, heads] or NULL
 * heads 1 to 128, rows * heads < 2^31, |sm_scale * q_scale * kv_scale| * log2(e) at
 * most 1e20 (PMQA_ERR_UNSUPPORTED otherwise); all of them finite. A row that sees no
 * token gives out = 0 and lse = -inf; tokens behind a bad table entry are not attended
 * to. A NaN among a token's values makes the rows that see it NaN, and no other row.
 * A row whose largest score passes about 2^23 ln 2 (5.8 million) in magnitude sets
 * PMQA_DEV_SCORE_RANGE.
 * The weights enter the products as two fp8 terms, each to 2^-8 of itself where
 * min(rows, max_rows) * heads <= 32 and to 2^-7 otherwise. What is lost of small ones
 * beside that is, over all n tiles of 128 tokens that a row sees, at most 2^-7.6 (1 + ln n) of the
 * row's weight (light tokens behind a heavy one with 80 % of it: 1 % of theirs, measured
 * up to 128 k tokens). Their sum is formed in fp32 of the unrounded ones.
 * ws: pmqa_latent_workspace_bytes() bytes, 256-byte aligned, its status word zero
 * before the first use (pmqa_workspace_init). One kernel launch where block_size *
 * max_blocks_per_seq <= 512, else two. Every sum is formed in one order: equal
 * calls give equal bits.
 */
int pmqa_latent_attention(const pmqa_paged_rows *p, const void *q, const void *kv_cache,
                          int32_t heads, float q_scale, float kv_scale, float sm_scale, void *out,
                          float *lse, void *ws, size_t ws_bytes, pmqa_stream_t stream);

/*
 * Measurement aid beside the decode path (computes nothing of the method): reads
 * the rows rows[0..n) of a pool of fixed-pitch rows, each as its 16-byte aligned
 * window (144 bytes for row_pitch 132, the token row of the KV cache; 576 bytes
 * for row_pitch 576, the latent row of the MLA cache), to time how fast the GPU
 * gathers such rows. One launch, one CTA per SM.
 *   pool      device, 16-byte aligned, pool_bytes long; a window that would pass
 *             its end, and a negative row, is skipped (PMQA_DEV_BAD_CONTEXT in out[0])
 *   rows      device int32 [n]
 *   method    0: 16-byte loads into registers; 1: 16-byte cp.async into shared
 *             memory; 2: one bulk copy (cp.async.bulk) per window into shared memory
 *   out       device uint32 [2], zeroed by the caller: out[0] |= status bits
 *             (PMQA_DEV_TIMEOUT for a wait that ran out), out[1] ^= the XOR of
 *             every 32-bit word read (method 0) or of each window's first
 *             word (methods 1, 2)
 * Returns PMQA_ERR_UNSUPPORTED for another pitch, PMQA_ERR_INVALID_ARG for
 * n < 0, a method outside 0..2, a null or misaligned pointer (n = 0 launches
 * nothing and returns PMQA_OK).
 */
int pmqa_gather_probe(const void *pool, uint64_t pool_bytes, const int32_t *rows, int64_t n,
                      int32_t row_pitch, int32_t method, uint32_t *out, pmqa_stream_t stream);

/*
 * Synchronise the stream, return the device status bits recorded since the
 * last read (>= 0) and clear them, or a negative PMQA_ERR_* code.
 */
int pmqa_read_device_status(void *ws, pmqa_stream_t stream);

/* Static text for a return code. */
const char *pmqa_status_string(int code);

/* Library version, major * 10000 + minor * 100 + patch. */
int pmqa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PMQA_H */
