/*
 * qsaidx.h -- paged MQA-logits scoring and per-row top-k for a sparse-attention
 * (QSA-style) indexer, on AMD Instinct MI355X (gfx950).
 *
 * The library computes, for every query row r with H index heads of dimension
 * D, and every compressed key column c of the row's request:
 *
 *     logit[r, c] = sum_h w[r, h] * ReLU( q[r, h, :] . k[c, :] )      c <  ctx[r]
 *     logit[r, c] = -inf                                             ctx[r] <= c < width
 *
 * The ReLU is applied per head, before the heads are summed (ROCm/ATOM PR #2651,
 * "Changes"); zero-padded heads therefore add exactly 0 (sglang PR #48649,
 * "Accuracy Tests").  w is an f32 weight per (row, head), or 1 when absent
 * (ROCm/aiter PR #4221, "Motivation" and "Technical details").  For fp8 keys with
 * a per-key f32 scale s[c], k[c, :] is the dequantised key fp8(k8[c, :]) * s[c]
 * (same page).  Key column c of request b lives in pool block
 * block_table[b, c / B] at slot c % B (same page, block-flat commit; sglang
 * PR #48649 test body).  Columns past a row's visible count are -inf (ROCm/aiter
 * PR #4221, test gate: the -inf mask is compared exactly).
 *
 * qsa_topk then selects, per row, the k columns of [0, ctx[r]) with the largest
 * logits (vLLM PR #62589, "Details": top-k reads only [0, visible); sglang
 * PR #48649: rows that fit in k keep everything).
 *
 * Conventions shared by every entry point
 *  - Every pointer argument is DEVICE memory owned by the caller, unless stated.
 *    The library allocates nothing, keeps no pointer after returning, and has no
 *    global state other than a thread-local error message.
 *  - Compute calls are asynchronous on `stream` (a hipStream_t; NULL = the null
 *    stream).  They never synchronise the device or read device memory on the
 *    host, so they may be captured into a HIP graph.
 *  - Only host-visible scalars are validated; a failed validation returns a
 *    status with no launch.  Device values are preconditions, listed per call.
 *  - No call aborts or throws.  qsa_last_error() describes the last non-OK
 *    status of the calling thread.
 */
#ifndef QSAIDX_H
#define QSAIDX_H

#include <stdint.h>

#ifndef QSA_API
#define QSA_API __attribute__((visibility("default")))
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum qsa_status {
    QSA_OK = 0,
    QSA_E_INVALID = 1,     /* null pointer, negative or inconsistent size          */
    QSA_E_DTYPE = 2,       /* unknown dtype, or q and k dtypes differ               */
    QSA_E_UNSUPPORTED = 3, /* valid request outside the compiled set (see below)    */
    QSA_E_RANGE = 4,       /* a size or offset exceeds what the kernels address     */
    QSA_E_ALIGN = 5,       /* pointer or stride misaligned                          */
    QSA_E_HIP = 6          /* the HIP runtime rejected the launch                  */
} qsa_status;

typedef enum qsa_dtype {
    QSA_BF16 = 0,          /* bfloat16 q and keys                                   */
    QSA_FP8_E4M3FN = 1,    /* OCP fp8 E4M3 ("fn": no infinities, max 448) q and keys */
    QSA_FP16 = 2           /* IEEE binary16 q and keys (vLLM #62589, "Details": the  */
                           /* dot runs in fp16 for fp16 inputs, fp32 accumulation)   */
} qsa_dtype;

typedef enum qsa_kv_layout {
    /* kcache is [num_blocks][block_size][head_dim] elements; for fp8 an optional
     * separate kscale [num_blocks][block_size] f32.                             */
    QSA_KV_PAGED = 0,
    /* fp8 only, block-flat co-packed (ROCm/aiter PR #4221, block-flat commit):
     * each block is block_size*head_dim key bytes (key of slot s at byte
     * s*head_dim) followed by block_size little-endian f32 scales (slot s at
     * byte block_size*head_dim + 4*s); block stride block_size*(head_dim+4).  */
    QSA_KV_COPACKED = 1,
    /* fp8 only, co-packed with the keys preshuffled in 16x16-byte tiles
     * (ROCm/aiter PR #4221, preshuffle commit and the commit that unifies both
     * layouts as one coordinate space with two stride vectors): the scale tail
     * is as in QSA_KV_COPACKED; in the key section, byte d of slot s sits at
     * (s/16)*16*head_dim + (d/16)*256 + (s%16)*16 + d%16 (each group of 16
     * slots is stored as head_dim/16 chunks of 16 slots x 16 bytes).
     * block_size must be a multiple of 16.                                     */
    QSA_KV_COPACKED_SHUFFLED = 2
} qsa_kv_layout;

typedef struct qsa_logits_shape {
    int32_t num_rows;    /* R query rows                                           */
    int32_t num_heads;   /* H index heads per row, zero-padded heads included      */
    int32_t head_dim;    /* D                                                      */
    int32_t block_size;  /* B key COLUMNS per pool block                           */
    int32_t num_reqs;    /* rows of block_table                                    */
    int32_t max_blocks;  /* columns of block_table                                 */
    int32_t width;       /* W logits written per row                               */
    int32_t q_dtype;     /* qsa_dtype                                              */
    int32_t k_dtype;     /* qsa_dtype; must equal q_dtype                          */
    int32_t kv_layout;   /* qsa_kv_layout                                          */
    int64_t num_blocks;  /* blocks in the key pool                                 */
    int64_t out_stride;  /* floats between consecutive rows of out, >= width       */
} qsa_logits_shape;

/*
 * qsa_paged_logits -- the masked logits [R][W] (formula at the top of this file).
 *
 *   q           [R][H][D] elements of q_dtype, row-major; rows of one request may
 *               sit anywhere, but request-major order lets rows share key reads.
 *   w           [R][H] f32, or NULL for w = 1.
 *   kcache      key pool in kv_layout (see qsa_kv_layout).
 *   kscale      QSA_KV_PAGED + fp8: [num_blocks][B] f32 or NULL (scale 1).
 *               Must be NULL for bf16, fp16 and the co-packed layouts.
 *   block_table [num_reqs][max_blocks] int32 pool block indices.
 *   ctx_lens    [R] int32 visible columns per row.
 *   row_to_req  [R] int32 row -> block_table row.
 *   out         [R][out_stride] f32; columns [0, W) of every row are written,
 *               columns [W, out_stride) are not touched.
 *
 * Visible count: ctx_eff[r] = clamp(ctx_lens[r], 0, min(W, max_blocks*B)).
 * Device preconditions: 0 <= row_to_req[r] < num_reqs; the first
 * ceil(ctx_eff/B) table entries of each row's request index blocks of the pool;
 * fp8 scales are >= 0 (the scale is applied after the ReLU, which equals
 * applying it to the key only for non-negative scales).  Out-of-range indices are
 * never dereferenced: a row_to_req value outside [0, num_reqs) makes that row's
 * visible columns NaN, and a table entry outside [0, num_blocks) makes the
 * columns it would feed NaN (with B a multiple of 16: the 16 columns of every
 * 16-column tile it feeds).
 *
 * Compiled set (else QSA_E_UNSUPPORTED): D in {64, 128}; H in {1,2,4,8,16,32,64};
 * B in [1, 1024] (B = 1: one key per table entry, the per-token layout of
 * ROCm/aiter PR #4221 before its KVBlockSize >= 1 commit; B not a multiple of 16
 * takes a per-column gather); bf16 + PAGED, fp16 + PAGED, fp8 + PAGED,
 * fp8 + COPACKED, fp8 + COPACKED_SHUFFLED (B a multiple of 16).
 * Alignment (else QSA_E_ALIGN): q, kcache, out 16-byte aligned; out_stride % 4 == 0.
 * Range (else QSA_E_RANGE): W <= 1<<24; R*out_stride*4 and num_blocks*block
 * bytes below 2^62.
 */
QSA_API qsa_status qsa_paged_logits(const void *q, const float *w, const void *kcache,
                            const float *kscale, const int32_t *block_table,
                            const int32_t *ctx_lens, const int32_t *row_to_req, float *out,
                            const qsa_logits_shape *shape, void *stream);

/* qsa_paged_logits, with the kernel timed: start_event / stop_event (hipEvent_t
 * created by the caller, or NULL) are recorded by the dispatch itself at the
 * kernel's start and end, so hipEventElapsedTime gives the kernel's duration
 * without marker-packet overhead.  For measurement tools; otherwise identical.
 * When the call launches nothing (R = 0 or W = 0) the events are not touched. */
QSA_API qsa_status qsa_paged_logits_timed(const void *q, const float *w, const void *kcache,
                                          const float *kscale, const int32_t *block_table,
                                          const int32_t *ctx_lens, const int32_t *row_to_req,
                                          float *out, const qsa_logits_shape *shape, void *stream,
                                          void *start_event, void *stop_event);

/* Validation of qsa_paged_logits' host-visible arguments only: no HIP call, no
 * launch.  Returns what qsa_paged_logits would return before launching. */
QSA_API qsa_status qsa_paged_logits_check(const void *q, const float *w, const void *kcache,
                                  const float *kscale, const int32_t *block_table,
                                  const int32_t *ctx_lens, const int32_t *row_to_req,
                                  const float *out, const qsa_logits_shape *shape);

/*
 * qsa_topk -- per row r, the k columns of its candidate range with the largest
 * logits; equal logits (+0 and -0 are equal) are broken toward the lower
 * column.  Rows with n_r <= k keep their whole range.
 *
 * Candidate range (vLLM PR #62589, "Details": top-k reads only the visible
 * columns; sglang PR #48649, "Accuracy Tests": the top-k takes per-row starts
 * and context lengths, and rows that fit in k keep everything):
 *   s_r = clamp(row_starts[r], 0, width)  (0 when row_starts is NULL),
 *   n_r = clamp(ctx_lens[r], 0, width - s_r),
 * the columns [s_r, s_r + n_r) of row r.  An index is reported as the offset
 * of its column from s_r, in [0, n_r): a row's result does not depend on where
 * its range sits in the buffer.
 *
 *   logits     [num_rows][logits_stride] f32 (the buffer holds num_rows *
 *              logits_stride floats); only the candidate range decides the
 *              result (reads are widened to whole 16-byte groups inside the
 *              row's stride).
 *   ctx_lens   [num_rows] int32: candidate count per row.
 *   row_starts [num_rows] int32, or NULL: first candidate column per row.
 *              Starts that are multiples of 4 take the same paths as no
 *              starts; other starts are exact but use the slower full-row
 *              selection for rows longer than k.
 *   idx_out    [num_rows][k] int32: the selected offsets in ascending order,
 *              then -1 in slots [min(k, n_r), k).  The order is part of this
 *              implementation, not of the selection's definition (a set).
 *
 * Device precondition: no NaN inside a candidate range (a NaN ranks by its bit
 * pattern: above +inf when its sign is clear, below -inf when set).
 *
 *   workspace  device scratch owned by the caller, or NULL.  With NULL every
 *              row is selected by one workgroup.  Otherwise it must hold at
 *              least qsa_topk_workspace_bytes(num_rows, width, k) bytes (else
 *              QSA_E_INVALID) at a 16-byte aligned address (else QSA_E_ALIGN).
 *              When that size is non-zero (at most 128 rows, width > 4096,
 *              and fewer than 48 rows or width > 32768), each row is shared
 *              by several workgroups in two kernels that pass counts and
 *              candidates through the workspace.  Its contents need
 *              no initialisation and are not kept between calls; calls that
 *              share a workspace must be ordered (same stream).  The selection
 *              does not depend on which path runs.
 *
 * Compiled set (else QSA_E_UNSUPPORTED): 1 <= k <= 2048; width <= 69632.
 * Alignment (else QSA_E_ALIGN): logits 16-byte aligned, logits_stride % 4 == 0.
 */
QSA_API qsa_status qsa_topk(const float *logits, int64_t logits_stride, const int32_t *ctx_lens,
                            const int32_t *row_starts, int32_t num_rows, int32_t width, int32_t k,
                            int32_t *idx_out, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * qsa_paged_logits_topk -- qsa_paged_logits, then qsa_topk on the logits it wrote
 * (row stride shape->out_stride, candidates [0, clamp(ctx_lens[r], 0, width)),
 * no row starts), in one call: the logits in `out` and the indices in idx_out
 * are exactly those of the two calls.  The pages time the whole selection, not
 * the scoring alone (vLLM PR #62589, "Performance": score + top-k, CUDA events
 * around both); here, for shapes that the per-tile scorer takes with 4 or fewer
 * heads (decode batches), its epilogue also writes each row's 16 largest scores
 * of every 64-column chunk into the workspace, and one selection kernel works
 * from those lists (a quarter of the row) instead of a sampling kernel and a
 * resolve kernel over the whole row.  Other shapes run the scoring kernel and
 * the plain selection.
 *
 *   q .. shape   as qsa_paged_logits (out is both its output and the
 *                selection's input).
 *   k, idx_out   as qsa_topk ([num_rows][k] int32, ascending, -1 padded).
 *   workspace    device scratch owned by the caller of at least
 *                qsa_paged_logits_topk_workspace_bytes(shape, k) bytes, 16-byte
 *                aligned (else QSA_E_INVALID / QSA_E_ALIGN), or NULL: no fusion
 *                and one workgroup per row for the selection (the results do
 *                not change).  No initialisation needed, nothing kept between
 *                calls; calls sharing a workspace must be ordered.
 *
 * Errors: those of qsa_paged_logits and of qsa_topk.  Device preconditions: both
 * calls'.  Asynchronous on `stream`; graph-capturable.
 */
QSA_API qsa_status qsa_paged_logits_topk(const void *q, const float *w, const void *kcache, const float *kscale,
                                         const int32_t *block_table, const int32_t *ctx_lens,
                                         const int32_t *row_to_req, float *out, const qsa_logits_shape *shape,
                                         int32_t k, int32_t *idx_out, void *workspace, int64_t workspace_bytes,
                                         void *stream);

/* Bytes of workspace qsa_paged_logits_topk uses for this shape (0 when none);
 * host-only, no HIP call. */
QSA_API int64_t qsa_paged_logits_topk_workspace_bytes(const qsa_logits_shape *shape, int32_t k);

/* qsa_paged_logits_topk with dispatch-recorded events (as qsa_paged_logits_timed):
 * start_event at the scoring kernel's start, mid_event at its end, stop_event at
 * the end of the selection.  Events may be NULL. */
QSA_API qsa_status qsa_paged_logits_topk_timed(const void *q, const float *w, const void *kcache,
                                               const float *kscale, const int32_t *block_table,
                                               const int32_t *ctx_lens, const int32_t *row_to_req, float *out,
                                               const qsa_logits_shape *shape, int32_t k, int32_t *idx_out,
                                               void *workspace, int64_t workspace_bytes, void *stream,
                                               void *start_event, void *mid_event, void *stop_event);

/*
 * qsa_topk_noalloc -- qsa_topk for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same selection as qsa_topk with a workspace of
 * qsa_topk_workspace_bytes(num_rows, width, k) bytes, but the workspace is a
 * fixed 9 MiB device array held by the library (one per GPU, until the process
 * ends), so the call allocates nothing.  Every supported shape fits (the
 * largest needs 8,652,800 bytes); a shape that would not returns QSA_E_RANGE.
 * The array is that of the calling thread's current device, which must be the
 * device of `stream`.  Calls on one GPU share the array: calls that overlap
 * (concurrent streams, several threads) race; order them on one stream.
 * Arguments and other errors as qsa_topk.
 */
QSA_API qsa_status qsa_topk_noalloc(const float *logits, int64_t logits_stride, const int32_t *ctx_lens,
                                    const int32_t *row_starts, int32_t num_rows, int32_t width, int32_t k,
                                    int32_t *idx_out, void *stream);

/* Bytes of workspace qsa_topk uses for this shape; 0 when every row is selected
 * by one workgroup whatever the workspace.  Host-only, no HIP call; k does not
 * change the size in this version of the library. */
QSA_API int64_t qsa_topk_workspace_bytes(int32_t num_rows, int32_t width, int32_t k);

/* qsa_topk with its kernels timed by dispatch-recorded events (as
 * qsa_paged_logits_timed): start_event at the start of the first kernel,
 * stop_event at the end of the last. */
QSA_API qsa_status qsa_topk_timed(const float *logits, int64_t logits_stride, const int32_t *ctx_lens,
                                  const int32_t *row_starts, int32_t num_rows, int32_t width, int32_t k,
                                  int32_t *idx_out, void *workspace, int64_t workspace_bytes, void *stream,
                                  void *start_event, void *stop_event);

/* Validation of qsa_topk's host-visible arguments only: no HIP call, no launch. */
QSA_API qsa_status qsa_topk_check(const float *logits, int64_t logits_stride, const int32_t *ctx_lens,
                                  const int32_t *row_starts, int32_t num_rows, int32_t width, int32_t k,
                                  const int32_t *idx_out, const void *workspace, int64_t workspace_bytes);

/*
 * qsa_expand -- the step after the selection: each selected compressed column
 * becomes the key tokens it stands for.  The pages time a full selection as
 * "score + top-k + expand" with a compression ratio of 4 (vLLM PR #62589,
 * "Performance" and the MI355X comment) without defining the step; this is the
 * plain reading: compressed column c covers tokens [c * ratio, c * ratio + ratio).
 *
 *   idx         [num_rows][k] int32 selected columns (qsa_topk's output; -1 is
 *               padding).
 *   token_lens  [num_rows] int32 tokens per row, or NULL for no bound.
 *   tokens_out  [num_rows][k * ratio] int32: slot p * ratio + j holds
 *               idx[r][p] * ratio + j when idx[r][p] >= 0 and that token is below
 *               token_lens[r] (and fits in int32), else -1.  Ascending columns
 *               give ascending tokens.
 *
 * Errors: QSA_E_INVALID for null pointers with num_rows > 0, num_rows < 0,
 * k < 1 or ratio < 1; QSA_E_RANGE when k * ratio > 2^24.
 */
QSA_API qsa_status qsa_expand(const int32_t *idx, int32_t num_rows, int32_t k, int32_t ratio,
                              const int32_t *token_lens, int32_t *tokens_out, void *stream);

/*
 * The calls below stand around the scorer and the selection in a serving step:
 *
 *   qsa_plan_batch        request lengths -> block table, slot maps, visible counts
 *   qsa_write_kv          new keys and values into the paged caches
 *   qsa_write_keys        new index keys into the scorer's cache
 *   qsa_norm_rope         head norms and rotary positions, keys and values to the caches
 *   qsa_paged_attention   attention over all visible tokens
 *   qsa_window_attention  attention over the newest tokens and the first ones
 *   qsa_sparse_attention  attention over the tokens of the selected columns
 *   qsa_verify_drafts     drafted tokens against the target's probabilities
 */

typedef struct qsa_plan_shape {
    int32_t num_reqs;     /* n requests                                            */
    int32_t max_blocks;   /* columns of block_table                                */
    int32_t block_size;   /* B tokens per block                                    */
    int32_t ratio;        /* tokens per compressed index column; divides B         */
    int32_t num_rows;     /* R: entries of the per-row outputs                     */
    int32_t num_free;     /* entries of free_blocks                                */
    int64_t num_blocks;   /* blocks in the pool                                    */
} qsa_plan_shape;

/*
 * qsa_plan_batch -- the metadata of one step, from request lengths.
 *
 * Request i holds past_lens[i] cached tokens (clamped to [0, max_blocks * B]) and
 * brings new_lens[i] new ones (negative: none).  Its rows are
 * [q_starts[i], q_starts[i + 1]), the row of its j-th new token stands for token
 * t = past + j.  Rows behind num_rows do not exist: the requests that would hold
 * them bring fewer tokens, down to none.
 *
 *   past_lens, new_lens [n] int32.
 *   free_blocks  [num_free] int32 pool blocks to take from, in order.
 *   block_table  [n][max_blocks] int32, updated: entries
 *                [ceil(past / B), ceil((past + new) / B)) of request i (up to
 *                max_blocks) take the next free blocks, request by request; -1
 *                once the list is used up.  Other entries are left alone.
 *   q_starts     [n + 1] int32.
 *   row_to_req   [R] int32.
 *   ctx_lens     [R] int32 visible tokens, t + 1 (at most max_blocks * B).
 *   slots        [R] int64 block_table[i][t / B] * B + t % B, or -1 where the
 *                table has no place for the token (t past its end, or an entry
 *                outside [0, num_blocks)).
 *   col_lens     [R] int32 whole compressed columns visible, ctx_lens / ratio, or
 *                NULL: qsa_paged_logits' ctx_lens over a cache with the same
 *                block table and B / ratio columns per block.
 *   col_slots    [R] int64 slot of the column that the row's token completes
 *                ((t + 1) % ratio == 0), block * (B / ratio) + (t % B) / ratio,
 *                else -1; or NULL.
 *   blocks_used  [1] int32 blocks asked of the free list (more than num_free:
 *                that many were missing), or NULL.
 *
 * Rows behind the last request's get request 0, no visible token and no slots,
 * so a batch padded for a captured graph passes through the other calls.  The
 * call does not change its own inputs but for block_table's new entries: called
 * again it gives the same answer.
 *
 * Device precondition: free_blocks are distinct blocks of the pool that no entry
 * holds.  Compiled set: n <= 4096.  Range: max_blocks * B <= 2^30, R <= 2^30.
 */
QSA_API qsa_status qsa_plan_batch(const int32_t *past_lens, const int32_t *new_lens, const int32_t *free_blocks,
                                  int32_t *block_table, int32_t *q_starts, int32_t *row_to_req, int32_t *ctx_lens,
                                  int64_t *slots, int32_t *col_lens, int64_t *col_slots, int32_t *blocks_used,
                                  const qsa_plan_shape *shape, void *stream);

/* Validation of qsa_plan_batch's host-visible arguments only: no HIP call. */
QSA_API qsa_status qsa_plan_batch_check(const int32_t *past_lens, const int32_t *new_lens,
                                        const int32_t *free_blocks, const int32_t *block_table,
                                        const int32_t *q_starts, const int32_t *row_to_req, const int32_t *ctx_lens,
                                        const int64_t *slots, const qsa_plan_shape *shape);

typedef struct qsa_kv_shape {
    int32_t num_rows;          /* R rows to write                                  */
    int32_t num_kv_heads;
    int32_t head_dim;          /* 64 or 128                                        */
    int32_t block_size;        /* B tokens per block                               */
    int32_t dtype;             /* QSA_BF16 or QSA_FP16, sources and caches         */
    int32_t reserved;
    int64_t num_blocks;
    /* strides in elements (the last dimension is contiguous): of k and v, and
     * of kcache and vcache                                                      */
    int64_t src_row_stride, src_head_stride;
    int64_t kv_block_stride, kv_slot_stride, kv_head_stride;
} qsa_kv_shape;

/*
 * qsa_write_kv -- k and v [R][num_kv_heads][head_dim] into the paged caches, row r
 * at slot slots[r] (block slots[r] / B, place slots[r] % B).  Rows whose slot is
 * outside [0, num_blocks * B) write nothing.
 *
 * Device precondition: the slots written are distinct (two rows for one slot
 * leave a mixture of both).  Alignment: pointers 16 bytes, strides multiples of 8
 * elements.  kcache and vcache have the same strides.
 */
QSA_API qsa_status qsa_write_kv(const void *k, const void *v, const int64_t *slots, void *kcache, void *vcache,
                                const qsa_kv_shape *shape, void *stream);
QSA_API qsa_status qsa_write_kv_check(const void *k, const void *v, const int64_t *slots, const void *kcache,
                                      const void *vcache, const qsa_kv_shape *shape);

typedef struct qsa_keys_shape {
    int32_t num_rows;          /* R keys to write                                  */
    int32_t head_dim;          /* D: 64 or 128                                     */
    int32_t block_size;        /* B key columns per block                          */
    int32_t src_dtype;         /* QSA_BF16 or QSA_FP16                             */
    int32_t k_dtype;           /* src_dtype, or QSA_FP8_E4M3FN                     */
    int32_t kv_layout;         /* qsa_kv_layout                                    */
    int64_t num_blocks;
    int64_t src_stride;        /* elements between keys, >= D                      */
} qsa_keys_shape;

/*
 * qsa_write_keys -- index keys [R][D] into qsa_paged_logits' key cache, key r at
 * slot slots[r] (rows whose slot is outside [0, num_blocks * B) write nothing).
 * 16-bit keys are copied.  For an fp8 cache each key x is stored as codes
 * rne(x / s) with s = max|x| / 448, or 1 for a key of zeros, in the layout's
 * place for its scale; a paged fp8 cache without kscale holds rne(x), saturated
 * to +-448.  A key with an infinity or a NaN spoils its own slot only.
 *
 * Device precondition: the slots written are distinct.  Alignment: keys and kcache
 * 16 bytes, src_stride a multiple of 8 elements.
 */
QSA_API qsa_status qsa_write_keys(const void *keys, const int64_t *slots, void *kcache, float *kscale,
                                  const qsa_keys_shape *shape, void *stream);
QSA_API qsa_status qsa_write_keys_check(const void *keys, const int64_t *slots, const void *kcache,
                                        const float *kscale, const qsa_keys_shape *shape);

typedef enum qsa_rope_layout {
    QSA_ROPE_HALF = 0,         /* pair i: elements i and i + rot_dim / 2           */
    QSA_ROPE_INTERLEAVED = 1   /* pair i: elements 2 i and 2 i + 1                 */
} qsa_rope_layout;

typedef struct qsa_rope_shape {
    int32_t num_rows;          /* R rows                                           */
    int32_t num_heads;         /* Hq query heads, 0: no queries                    */
    int32_t num_kv_heads;      /* Hk key heads, 0: no keys                         */
    int32_t head_dim;          /* D: 64 or 128                                     */
    int32_t rot_dim;           /* rotated elements of a head, a multiple of 16     */
    int32_t rot_offset;        /* the first of them, a multiple of 8               */
    int32_t layout;            /* qsa_rope_layout                                  */
    int32_t dtype;             /* QSA_BF16 or QSA_FP16: all heads and the caches   */
    int32_t position_offset;   /* added to positions                               */
    int32_t block_size;        /* B tokens per block (with caches)                 */
    float eps;                 /* of the norms, >= 0                               */
    float factor;              /* on cosines and sines, 1 where nothing is scaled  */
    int64_t num_blocks;        /* (with caches)                                    */
    /* strides in elements (the last dimension is contiguous)                    */
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    int64_t q_out_row_stride, q_out_head_stride, k_out_row_stride, k_out_head_stride;
    int64_t kv_block_stride, kv_slot_stride, kv_head_stride;
} qsa_rope_shape;

/*
 * qsa_norm_rope -- query and key heads normed and rotated by their positions, keys and
 * values into the paged caches, in one pass:
 *
 *     y = x w / sqrt(mean(x^2) + eps)          over a head's D elements, where it has a weight
 *     (a, b) -> factor (a cos t - b sin t, b cos t + a sin t),   t = position inv_freq[i]
 *
 * for the pairs i of elements [rot_offset, rot_offset + rot_dim), the others unchanged.
 * position = positions[r] + position_offset: qsa_plan_batch's ctx_lens with an offset of
 * -1 are the rows' positions.  A row whose position is negative (one behind the last
 * request's) writes nothing.
 *
 *   q, q_out   [R][Hq][D]; both NULL with Hq = 0.  q_out may be q.
 *   k, k_out   [R][Hk][D]; both NULL with Hk = 0.  k_out may be k, or NULL where kcache
 *              takes the keys.
 *   v          [R][Hk][D], stored as they are; with vcache.
 *   q_weight, k_weight [D] f32, or NULL: no norm.
 *   positions  [R] int32.
 *   inv_freq   [rot_dim / 2] f64, radians per position (any scaling for long contexts is in
 *              them and in factor); NULL with rot_dim = 0.
 *   slots      [R] int64 with the caches, as qsa_write_kv's (rows outside
 *              [0, num_blocks * B) write q_out and k_out only).
 *   kcache, vcache  NULL, or k's and v's; vcache only with kcache.  Both have the same
 *              strides.
 *
 * Norms, angles' reduction and products are 32-bit or more with one rounding at the end;
 * the angle itself is a 64-bit product.  A head's sum of squares has to stay below 2^127 (heads
 * of larger values come out 0 or NaN); with eps below 2^-118 it has to be 2^-118 at least (smaller
 * bf16 heads are off or NaN, as is a head of zeros with eps = 0).  An infinity or a NaN spoils its
 * own head only.
 *
 * Device precondition: the slots written are distinct.  Outputs must not overlap inputs
 * but for q_out = q and k_out = k with their strides.  Compiled set: D in {64, 128};
 * Hq <= 8192, Hk <= 1024.  Range: R <= 2^21.  Alignment: q, k, v, their outputs and the
 * caches 16 bytes, strides multiples of 8 elements.
 */
QSA_API qsa_status qsa_norm_rope(const void *q, const void *k, const void *v, const float *q_weight,
                                 const float *k_weight, const int32_t *positions, const double *inv_freq,
                                 const int64_t *slots, void *q_out, void *k_out, void *kcache, void *vcache,
                                 const qsa_rope_shape *shape, void *stream);
QSA_API qsa_status qsa_norm_rope_check(const void *q, const void *k, const void *v, const int32_t *positions,
                                       const double *inv_freq, const int64_t *slots, const void *q_out,
                                       const void *k_out, const void *kcache, const void *vcache,
                                       const qsa_rope_shape *shape);

typedef struct qsa_attn_shape {
    int32_t num_rows;          /* R query rows of q and out                        */
    int32_t num_heads;         /* Hq query heads                                   */
    int32_t num_kv_heads;      /* Hk; query head h reads kv head h / (Hq / Hk)     */
    int32_t head_dim;          /* D: 64 or 128                                     */
    int32_t block_size;        /* B tokens per block                               */
    int32_t num_reqs;          /* rows of block_table                              */
    int32_t max_blocks;        /* columns of block_table                           */
    int32_t dtype;             /* QSA_BF16 or QSA_FP16: q, caches and out          */
    float scale;               /* of the scores, in (0, 1e38]                      */
    int32_t reserved;
    int64_t num_blocks;
    /* strides in elements (the last dimension is contiguous)                    */
    int64_t q_row_stride, q_head_stride;
    int64_t out_row_stride, out_head_stride;
    int64_t kv_block_stride, kv_slot_stride, kv_head_stride;
} qsa_attn_shape;

/*
 * qsa_paged_attention -- attention of new tokens over the paged cache:
 *
 *     out[r, h, :] = sum_c p_c v[c],  p = softmax_c(scale * q[r, h, :] . k[c])
 *     lse[r, h]    = log sum_c exp(scale * q[r, h, :] . k[c])
 *
 * over the columns c < ctx_lens[r] of the row's request (clamped to
 * [0, max_blocks * B]); a chunk of new tokens is causal when ctx_lens are
 * qsa_plan_batch's.  Token c lies in pool block block_table[i][c / B] at place
 * c % B.  A row that sees nothing has out 0 and lse -inf.
 *
 *   q         [R][Hq][D], rows of one request together.
 *   ctx_lens  [R] int32; any counts, not only causal ones.
 *   q_starts  [num_reqs + 1] int32, non-decreasing: request i's rows are
 *             [q_starts[i], q_starts[i + 1]) (values are clamped to [0, R]).
 *             Rows outside all requests are left as they were in out and lse.
 *   lse       [R][Hq] f32 contiguous, or NULL.
 *   workspace qsa_paged_attention_workspace_bytes(shape) bytes (0 also for shapes
 *             that the call refuses), 16-byte aligned, or NULL: then few rows over
 *             long contexts are not spread over the chip.  No initialisation; calls
 *             that share it must be ordered.
 *
 * Keys and values of columns that no row of the request sees are not used, and
 * what only other rows see does not change a row, infinities and NaN included; an
 * infinite value that a row sees is infinite in its output.
 * A table entry outside [0, num_blocks) is not dereferenced: rows that see its
 * columns are NaN.  Weights are rounded to dtype before the second product (fp16:
 * those below 2^-27 of a row's largest to multiples of 2^-37 of it, or finer); sums,
 * maxima and lse are 32-bit.  Weighted values are summed before the division: with bf16
 * the magnitudes of a row's values in one element have to add up to less than 2^119.
 *
 * Compiled set: Hq / Hk <= 128, Hq <= 8192, B <= 1024.  Range: max_blocks * B <=
 * 2^30, R and num_reqs <= 2^21, and (R * Hq / (256 Hk) + num_reqs) * Hk tiles <= 2^22.
 * Alignment: pointers 16 bytes, strides multiples of 8 elements.  out and lse must
 * not overlap the inputs.
 */
QSA_API qsa_status qsa_paged_attention(const void *q, const void *kcache, const void *vcache,
                                       const int32_t *block_table, const int32_t *ctx_lens,
                                       const int32_t *q_starts, void *out, float *lse, const qsa_attn_shape *shape,
                                       void *workspace, int64_t workspace_bytes, void *stream);
QSA_API qsa_status qsa_paged_attention_check(const void *q, const void *kcache, const void *vcache,
                                             const int32_t *block_table, const int32_t *ctx_lens,
                                             const int32_t *q_starts, const void *out, const qsa_attn_shape *shape,
                                             const void *workspace, int64_t workspace_bytes);
QSA_API int64_t qsa_paged_attention_workspace_bytes(const qsa_attn_shape *shape);

/*
 * qsa_window_attention -- qsa_paged_attention over a sliding window and the first tokens:
 * row r sees the newest `window` of its ctx_lens[r] tokens and the first `sinks`, that is
 * the columns c < ctx_lens[r] with c >= ctx_lens[r] - window or c < sinks, each once.
 *
 * Table entries and tokens that no row of a request sees are not used when its rows'
 * visible counts are neighbours (qsa_plan_batch's are): the blocks between the first
 * tokens and the oldest row's window may have been freed, their entries be anything.  (With
 * other counts, rows far apart in one request, entries between their windows are read
 * too: those outside [0, num_blocks) cost time, nothing else.)
 *
 *   window    >= 1.  sinks >= 0.
 *   workspace as above, qsa_window_attention_workspace_bytes(shape, window, sinks).
 *
 * The other arguments, errors and limits are qsa_paged_attention's.
 */
QSA_API qsa_status qsa_window_attention(const void *q, const void *kcache, const void *vcache,
                                        const int32_t *block_table, const int32_t *ctx_lens,
                                        const int32_t *q_starts, int32_t window, int32_t sinks, void *out, float *lse,
                                        const qsa_attn_shape *shape, void *workspace, int64_t workspace_bytes,
                                        void *stream);
QSA_API qsa_status qsa_window_attention_check(const void *q, const void *kcache, const void *vcache,
                                              const int32_t *block_table, const int32_t *ctx_lens,
                                              const int32_t *q_starts, int32_t window, int32_t sinks, const void *out,
                                              const qsa_attn_shape *shape, const void *workspace,
                                              int64_t workspace_bytes);
QSA_API int64_t qsa_window_attention_workspace_bytes(const qsa_attn_shape *shape, int32_t window, int32_t sinks);

/*
 * qsa_sparse_attention -- qsa_paged_attention over selected tokens: row r attends to tokens
 * idx[r][p] * ratio + j, j < ratio, for its non-negative idx (qsa_topk's output,
 * or with ratio 1 qsa_expand's); tokens at or behind token_lens[r] are left out.
 * The order of a row's indices does not matter; an index given twice counts
 * twice.  A row without tokens has out 0 and lse -inf.
 *
 * qsa_topk over qsa_plan_batch's col_lens selects whole columns.  A row's newest
 * ctx_lens % ratio tokens, its own among them, are in none of those: a caller that
 * wants them gives column ctx_lens / ratio as one index more per row, which
 * token_lens = ctx_lens cuts behind the row's own token.
 *
 *   row_to_req [R] int32; a value outside [0, num_reqs) makes the row's outputs
 *              NaN (if it selects anything).
 *   idx        [R][k] int32, negative entries are padding, anywhere.
 *   token_lens [R] int32 or NULL (the table's max_blocks * B).
 *   workspace  as above, qsa_sparse_attention_workspace_bytes(shape, k, ratio).
 *
 * The other arguments, errors and limits are qsa_paged_attention's; k * ratio <=
 * 2^24.
 */
QSA_API qsa_status qsa_sparse_attention(const void *q, const void *kcache, const void *vcache,
                                        const int32_t *block_table, const int32_t *row_to_req, const int32_t *idx,
                                        int32_t k, int32_t ratio, const int32_t *token_lens, void *out, float *lse,
                                        const qsa_attn_shape *shape, void *workspace, int64_t workspace_bytes,
                                        void *stream);
QSA_API qsa_status qsa_sparse_attention_check(const void *q, const void *kcache, const void *vcache,
                                              const int32_t *block_table, const int32_t *row_to_req,
                                              const int32_t *idx, int32_t k, int32_t ratio, const void *out,
                                              const qsa_attn_shape *shape, const void *workspace,
                                              int64_t workspace_bytes);
QSA_API int64_t qsa_sparse_attention_workspace_bytes(const qsa_attn_shape *shape, int32_t k, int32_t ratio);

typedef struct qsa_verify_shape {
    int32_t num_rows;          /* R rows of probs                                  */
    int32_t num_reqs;          /* n requests                                       */
    int32_t vocab;             /* V                                                */
    int32_t max_tokens;        /* columns of out_tokens, >= 1                      */
    int64_t prob_stride;       /* floats between rows of probs, >= V               */
    int64_t draft_stride;      /* the same of draft_probs                          */
} qsa_verify_shape;

/*
 * qsa_verify_drafts -- the end of a verify step: which drafted tokens are kept, and the
 * token after them, so that the tokens are distributed as the target's.
 *
 * Request i's rows are [q_starts[i], q_starts[i + 1]) (values are clamped to [0, R]); of
 * more than max_tokens rows only the first max_tokens count.  Row s + j's input is
 * tokens[s + j]: the last token so far at j = 0, then the drafts, so that draft j is
 * x = tokens[s + j + 1] and p = probs[s + j] is the target's distribution for its place.
 *
 *     draft j is kept      iff all before it are and uniforms[s + j] * q(x) < p(x)
 *     the token after them ~ max(p - q, 0) of the first row whose draft is not kept, or
 *                            p of the last row where all are
 *
 * with q = draft_probs[s + j], or the certainty of x without draft_probs.  The token is
 * the lowest index whose cumulative weight passes sample_uniforms[i] times the weights'
 * sum (the last index with weight where none does): sums and products in 64 bits, a
 * difference p - q rounded once to 32; a row's own sum need not be 1.  Entries that are not positive numbers have no weight.  Where
 * p is nowhere above q the token is taken from p, and it is -1 where p has no weight either.
 * A draft outside [0, V) is not kept.
 *
 *   probs, draft_probs [R][V] f32 (draft_probs or NULL; a request's last row of it is not
 *                   read).  Of rows that decide nothing at most the entries of their drafts
 *                   are read.
 *   tokens          [R] int32.
 *   uniforms        [R] f32 in [0, 1), one per draft (a request's last is not used).
 *   sample_uniforms [n] f32 in [0, 1).
 *   out_tokens      [n][max_tokens] int32: the drafts kept, the token after them, then -1.
 *   num_tokens      [n] int32: drafts kept + 1, what qsa_plan_batch's past_lens grow by; 0 for
 *                   a request without rows.
 *   workspace       qsa_verify_drafts_workspace_bytes(shape) bytes (0: none is used), 16-byte
 *                   aligned, or NULL: then few requests are not spread over the chip (the
 *                   tokens do not change, unless a cumulative weight and the number it has
 *                   to pass are alike to 2^-40 without being equal sums of exact terms).  No
 *                   initialisation; calls that share it must be ordered.
 *
 * Device precondition: the outputs overlap neither the inputs nor each other.
 * Compiled set: V <= 2^20.  Range: R <= 2^24, n <= 2^22, n * max_tokens <= 2^30.
 */
QSA_API qsa_status qsa_verify_drafts(const float *probs, const float *draft_probs, const int32_t *tokens,
                                     const int32_t *q_starts, const float *uniforms, const float *sample_uniforms,
                                     int32_t *out_tokens, int32_t *num_tokens, const qsa_verify_shape *shape,
                                     void *workspace, int64_t workspace_bytes, void *stream);
QSA_API qsa_status qsa_verify_drafts_check(const float *probs, const float *draft_probs, const int32_t *tokens,
                                           const int32_t *q_starts, const float *uniforms,
                                           const float *sample_uniforms, const int32_t *out_tokens,
                                           const int32_t *num_tokens, const qsa_verify_shape *shape,
                                           const void *workspace, int64_t workspace_bytes);
QSA_API int64_t qsa_verify_drafts_workspace_bytes(const qsa_verify_shape *shape);

/* Message for the calling thread's last non-OK status ("" if none). Owned by the
 * library; valid until the thread's next call. */
QSA_API const char *qsa_last_error(void);

/* Library version string, e.g. "qsaidx 0.1.0 gfx950". */
QSA_API const char *qsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QSAIDX_H */
