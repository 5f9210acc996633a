/*
 * dsrows: one decode step of DeepSeek-style sparse attention over up to eight
 * independent rows (requests), each with its own caches and its own length,
 * on one NVIDIA GB300 (sm_103a).
 *
 * The operations follow the DeepSeek-V4 joint-decode kernels of the mlx-native
 * crate: `src/shaders/deepseek_rows.metal` (sections "Lightning indexer score
 * and deterministic top-512" and "Sparse attention (selected shared-KV rows
 * with learned sinks)") and their dispatch in `src/ops/deepseek_rows.rs`
 * (`dispatch_deepseek_indexer_rows`, `dispatch_deepseek_sparse_attention_rows`,
 * row structs `DeepSeekIndexerRow` / `DeepSeekSparseAttentionRow`).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers, owned by the caller, which also
 *   guarantees their sizes (stated per argument). The library allocates no
 *   memory and never synchronises the host; every entry point only enqueues
 *   work on `stream` (a cudaStream_t; NULL is the legacy default stream).
 * - bf16 tensors are passed as `ds_bf16` (uint16_t bit patterns).
 * - Arguments are validated on the host before anything is enqueued. On a
 *   bad argument the call enqueues nothing, returns a negative `DS_E*` code
 *   and sets a message readable with ds_rows_last_error() (per host thread).
 *   A CUDA launch failure returns DS_ECUDA.
 * - Bad DATA (NaN/Inf inputs, an out-of-range index) is not a call error: it
 *   zeroes the affected attention heads ("fail closed") and is reported in
 *   the optional `invalid` output.
 * - Row `r` of a joint call is bitwise equal to a call with only row `r`: all
 *   tiling, split counts and reduction orders depend on that row's kv_len and
 *   width alone (except ds_rows_prefix_attn, which says what it keeps).
 * - Calls that share a workspace or an output must not overlap in time
 *   (order them on one stream).
 * - A call's kernels are chained with programmatic dependent launch. Its first
 *   kernel may become resident while the stream's previous kernel still runs,
 *   but it waits for that kernel to complete before it reads or writes
 *   anything. Its last kernel lets the stream's next kernel launch early: a
 *   kernel the caller launches next with programmatic stream serialization
 *   must wait (griddepcontrol.wait, cudaGridDependencySynchronize) before it
 *   touches this call's outputs. Ordinary launches need nothing.
 */
#ifndef DSROWS_H
#define DSROWS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DS_ROWS_MAX 8     /* rows per call (binding slots per cache family) */
#define DS_INDEX_HEADS 64 /* indexer query heads */
#define DS_INDEX_DIM 128  /* indexer key / query width */
#define DS_INDEX_VROWS_MAX 64 /* rows x queries of one multi-query indexer call */
#define DS_TOPK 512       /* most selected KV rows per row */
#define DS_HEADS 64       /* attention heads */
#define DS_DIM 512        /* shared-KV row width (K and V) */
#define DS_PREFIX_ROWS_MAX 64 /* rows of a shared-prefix attention call */

/* Status codes. */
#define DS_OK 0
#define DS_EINVAL (-1) /* a bad argument (message says which) */
#define DS_ESIZE (-2)  /* workspace too small, or a size overflows 32 bits */
#define DS_EALIGN (-3) /* a pointer is not aligned as required */
#define DS_ECUDA (-4)  /* a CUDA call failed while enqueueing */

typedef uint16_t ds_bf16;

/*
 * One row of a call (`DeepSeekSparseAttentionRow` plus the indexer's fields).
 *   kv_len       keys / KV rows in the row's caches (> 0).
 *   width        selected slots of the row: 1 <= width <= min(512, kv_len).
 *                The top-k stage and the decode step select exactly
 *                min(512, kv_len) (DS_EINVAL otherwise) and write that many
 *                indices, -1 in slots past the row's finite scores; the
 *                attention stage takes any width in that range (the caller's
 *                index list).
 *   index_offset element offset of the row's `width` int32 indices in the
 *                indices buffer.
 *   q_row        row of the [*, 64, 128] / [*, 64, 512] queries, the [*, 64]
 *                head weights, per-row sinks, outputs and invalid flags.
 */
typedef struct {
    uint32_t kv_len;
    uint32_t width;
    uint32_t index_offset;
    uint32_t q_row;
} ds_row_t;

/*
 * The rows of a call: `rows` entries of `table` (host memory), and per entry
 * a device pointer to its caches (host arrays of `rows` pointers):
 *   index_keys[e]  bf16 [kv_len, 128] row-major indexer keys   (16-B aligned)
 *   kv[e]          bf16 [kv_len, 512] row-major shared K/V rows (16-B aligned)
 * A call reads only the cache family it needs; the other may be NULL.
 */
typedef struct {
    int rows;
    const ds_row_t* table;
    const ds_bf16* const* index_keys;
    const ds_bf16* const* kv;
} ds_row_set_t;

/*
 * Device status. The first 4 bytes of a workspace hold a uint32 status word.
 * Every call that takes a workspace zeroes it when it starts, and its kernels
 * OR these bits into it:
 *   DS_STATUS_WAIT_TIMEOUT  a bounded device-side wait (2 s of %globaltimer)
 *                           gave up; the kernel unwound without finishing and
 *                           the call's outputs are not valid.
 *   DS_STATUS_OVERFLOW      an internal consistency check of the selection
 *                           failed (candidate counts disagreed); its indices
 *                           may be incomplete. Not expected in any input.
 * Read the word once the call has completed (for example a 4-byte
 * cudaMemcpyAsync on the same stream); the next call on the workspace clears
 * it. 0: neither happened. ds_rows_topk_static keeps its word in the
 * library (ds_rows_topk_static_status reads it).
 */
#define DS_STATUS_WAIT_TIMEOUT 1u
#define DS_STATUS_OVERFLOW 2u

/*
 * Workspace bytes that every entry point below needs for this row table
 * (the largest need over the entry points). 0 when the table is invalid
 * (see ds_rows_last_error). The workspace must be 256-byte aligned; its
 * contents need no initialisation and are scratch between calls.
 */
size_t ds_rows_workspace_bytes(int rows, const ds_row_t* table);

/*
 * (1) Lightning-indexer score (`deepseek_indexer_score_mma_rows_bf16`):
 *   scores[e * score_stride + j] =
 *       sum_{h<64} w_index[q_row, h] * max(0, sum_{d<128} q_index[q_row, h, d] * K_e[j, d])
 * for j < kv_len of entry e; a non-finite score is stored as -inf. Every key
 * is valid (no causal cut).
 *   q_index     bf16 [Q, 64, 128]                              (16-B aligned)
 *   w_index     fp32 [Q, 64]
 *   scores      fp32, entry e at e * score_stride; score_stride >= max kv_len.
 *               Elements j >= kv_len of a row are not written.
 */
int ds_rows_indexer_score(const ds_row_set_t* set, const ds_bf16* q_index, const float* w_index,
                          float* scores, size_t score_stride, void* stream);

/*
 * (2) Deterministic top-k (`deepseek_indexer_topk_block/merge/finalize_rows_i32`):
 * for each entry e, the first `width` indices j < kv_len ordered best first by
 * (score descending, then lower index), over the finite scores only; slots past
 * the number of finite scores hold -1. -0.0 and +0.0 tie.
 *   scores      fp32, entry e at e * score_stride (as ds_rows_indexer_score).
 *   indices     int32, entry e writes [index_offset, index_offset + width);
 *               these ranges must not overlap.
 *   workspace   at least ds_rows_workspace_bytes(...) bytes.
 */
int ds_rows_topk(const ds_row_set_t* set, const float* scores, size_t score_stride,
                 int32_t* indices, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Top-k without a workspace. There is no counterpart on the prior-art pages:
 * this entry point exists for callers that cannot allocate device memory when
 * they run the top-k stage, for example code running under a CUDA graph or a
 * real-time loop that forbids allocation, or an embedding whose device
 * allocator is not reachable from the calling code. It computes exactly what
 * ds_rows_topk computes (same arguments, bitwise the same indices) but keeps
 * its scratch in one fixed array inside the library instead of a
 * caller-provided workspace, and allocates nothing.
 *   - Size: the array holds DS_TOPK_STATIC_SCRATCH_BYTES bytes (about 64 KiB),
 *     enough for DS_ROWS_MAX rows of any kv_len; every GPU that loads the
 *     library keeps it until the process exits. A table needing more is
 *     rejected with DS_ESIZE (more than DS_ROWS_MAX rows is DS_EINVAL).
 *   - Set-up: the first call on each device looks up the array's device
 *     address (with that device current). Make that first call before any
 *     stream capture.
 *   - Sharing: every call on a device uses the same array, which keeps the
 *     previous call's contents; each call clears what must start at zero.
 *     Calls that overlap on the GPU (different streams, no ordering between
 *     them) race on the array and give wrong results: order them.
 */
#define DS_TOPK_STATIC_SCRATCH_BYTES 65792
int ds_rows_topk_static(const ds_row_set_t* set, const float* scores, size_t score_stride,
                        int32_t* indices, void* stream);

/*
 * The status word of ds_rows_topk_static on the current device (DS_STATUS_*
 * bits, as in a workspace's first word; each ds_rows_topk_static call clears
 * it when it starts). Enqueues a 4-byte copy of the word on `stream` into
 * `status` (device or page-locked host memory, 4-byte aligned); read it once
 * the stream has passed this point. Allocates nothing; like the top-k call it
 * shares the library's array, so a call on another stream that overlaps it
 * races. DS_EINVAL for a NULL `status`, DS_ECUDA when the copy cannot be
 * enqueued.
 */
int ds_rows_topk_static_status(uint32_t* status, void* stream);

/*
 * (3)+(4) Gather and sink-softmax sparse attention
 * (`deepseek_sparse_attention_score_rows_bf16` + `..._reduce_rows_bf16`):
 * for each entry e and head h, over the slots t < width with index
 * i_t = indices[index_offset + t]:
 *   i_t == -1 is skipped; i_t < -1 or i_t >= kv_len zeroes every head of e;
 *   l_t = scale * q_attn[q_row, h, :] . KV_e[i_t, :]
 *   m = max(sink_h, max_t l_t), den = exp(sink_h - m) + sum_t exp(l_t - m)
 *   out[q_row, h, :] = bf16( sum_t exp(l_t - m) * KV_e[i_t, :] / den )
 * The sink has no value row. A non-finite sink, q element or selected KV
 * element, an overflowed logit or den <= 0 zeroes the head (fail closed).
 * The sums run over the row's valid indices in ascending order (duplicates
 * kept), so the result does not depend on the order of the indices within
 * [index_offset, index_offset + width): it is a function of their multiset.
 *   q_attn      bf16 [Q, 64, 512]                              (16-B aligned)
 *   sinks       fp32; head h of entry e at sinks[q_row * sinks_row_stride + h];
 *               sinks_row_stride 0 shares one [64] vector, else >= 64.
 *   indices     int32 (as written by ds_rows_topk).
 *   scale       finite and > 0 (1/sqrt(512) for the DeepSeek shapes).
 *   out         bf16 [Q, 64, 512]; q_row must be unique across the entries.
 *   invalid     optional uint32 [Q, 64]: 1 where the head was zeroed, else 0.
 *   workspace   at least ds_rows_workspace_bytes(...) bytes.
 */
int ds_rows_sparse_attn(const ds_row_set_t* set, const ds_bf16* q_attn, const float* sinks,
                        size_t sinks_row_stride, const int32_t* indices, float scale,
                        ds_bf16* out, uint32_t* invalid, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * The whole decode step: (1) indexer score -> (2) top-`width` -> (3)+(4)
 * gather and sink attention, on one stream. Scores and the selection stay in
 * the workspace. Arguments as in the stages above; `indices` is optional
 * (NULL: the selection is not written out) and, when given, receives the
 * selected indices best first at each entry's index_offset (ranges must not
 * overlap). The attention sums over the selected rows in ascending index
 * order, as ds_rows_sparse_attn does, so `out` is bitwise what
 * ds_rows_sparse_attn gives on those indices.
 */
int ds_rows_decode(const ds_row_set_t* set, const ds_bf16* q_index, const float* w_index,
                   const ds_bf16* q_attn, const float* sinks, size_t sinks_row_stride,
                   float scale, ds_bf16* out, int32_t* indices, uint32_t* invalid,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes for ds_rows_decode_host: the decode workspace plus device
 * staging for the step's inputs and outputs; 0 when the table is invalid. */
size_t ds_rows_decode_host_workspace_bytes(int rows, const ds_row_t* table, size_t sinks_row_stride);

/*
 * ds_rows_decode with the step's inputs and outputs in HOST memory. The
 * caches stay on the device (`set`). Everything is ordered on `stream`, and
 * the call returns before the step completes: synchronise `stream` before
 * reading h_out. Results are bitwise those of ds_rows_decode.
 *   - h_q_index and h_w_index are copied into device staging inside the
 *     workspace (the indexer's query is a tensor-core operand); when pinned,
 *     by the workspace-clear kernel itself.
 *   - A pinned h_q_attn is copied into staging by the indexer while it waits
 *     for its first scores; the attention reads h_sinks, and writes h_out,
 *     h_indices and h_invalid, in place when they are pinned (page-locked)
 *     host memory. Any other host memory goes through staging, with
 *     cudaMemcpyAsync before and after the kernels.
 * The call may be captured in a CUDA graph.
 *   h_q_index   bf16 [Q, 64, 128] (16-B aligned); h_w_index fp32 [Q, 64]
 *   h_q_attn    bf16 [Q, 64, 512] (16-B aligned); h_sinks as for ds_rows_decode
 *   h_out       bf16 [Q, 64, 512] (16-B aligned): the entries' q_rows are
 *               written, no others.
 *   h_indices   optional int32 (as ds_rows_decode's indices).
 *   h_invalid   optional uint32 [Q, 64]: the entries' q_rows are written.
 *   Q = max q_row + 1. When the entries use every q_row 0..Q-1, a staged array
 *   travels as one copy, else one copy per entry.
 *   workspace   at least ds_rows_decode_host_workspace_bytes(...) bytes.
 * Errors as ds_rows_decode, plus DS_EINVAL for a NULL host array.
 */
int ds_rows_decode_host(const ds_row_set_t* set, const ds_bf16* h_q_index, const float* h_w_index,
                        const ds_bf16* h_q_attn, const float* h_sinks, size_t sinks_row_stride, float scale,
                        ds_bf16* h_out, int32_t* h_indices, uint32_t* h_invalid, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * One row of a positioned indexer call (`DeepSeekIndexerRow`; compression
 * ratio 4, one query per row):
 *   kv_len        compressed keys in the row's indexer cache (> 0).
 *   start_pos     the query's absolute position. The row's valid keys are
 *                 j < valid_count = (start_pos + 1) / 4; kv_len must be at
 *                 least valid_count (start_pos < 2^32 - 1).
 *   offset        added to every emitted index: >= 0, and
 *                 offset + valid_count - 1 must fit int32 (-1 is the sentinel).
 *   q_row         row of the [*, 64, 128] queries and [*, 64] head weights.
 *   output_offset element offset of the row's 512 output indices; the ranges
 *                 [output_offset, output_offset + 512) must not overlap.
 */
typedef struct {
    uint32_t kv_len;
    uint32_t start_pos;
    int32_t offset;
    uint32_t q_row;
    uint32_t output_offset;
} ds_indexer_row_t;

/* Workspace bytes for ds_rows_indexer_topk with this table; 0 when the table
 * is invalid (see ds_rows_last_error). 256-byte aligned, scratch between calls. */
size_t ds_rows_indexer_topk_workspace_bytes(int rows, const ds_indexer_row_t* table);

/*
 * (1)+(2) Positioned indexer and causal top-512 (`dispatch_deepseek_indexer_rows`:
 * `deepseek_indexer_score_mma_rows_bf16` with its valid_count, then
 * `deepseek_indexer_topk_block/merge/finalize_rows_i32`). For each entry e, with
 * valid_count = min(kv_len, (start_pos + 1) / 4):
 *   s[j] = sum_{h<64} w_index[q_row, h] * max(0, q_index[q_row, h, :] . K_e[j, :])
 * for j < valid_count (keys at or past valid_count take no part), and
 *   indices[output_offset + t], t < 512 = the t-th best j (score descending,
 *   then lower index, finite scores only) plus offset, for t < valid_count when
 *   such a j exists; every other slot is -1.
 *   index_keys  host array of `rows` device pointers: bf16 [kv_len, 128] (16-B aligned).
 *   q_index     bf16 [Q, 64, 128] (16-B aligned); w_index fp32 [Q, 64].
 *   indices     int32, 512 per entry at output_offset.
 *   workspace   at least ds_rows_indexer_topk_workspace_bytes(...) bytes.
 */
int ds_rows_indexer_topk(int rows, const ds_indexer_row_t* table, const ds_bf16* const* index_keys,
                         const ds_bf16* q_index, const float* w_index, int32_t* indices,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes for ds_rows_indexer_topk_queries; 0 when the arguments are
 * invalid. ds_rows_indexer_topk_workspace_bytes(r, t) equals this with
 * query_len 1. */
size_t ds_rows_indexer_topk_queries_workspace_bytes(int rows, const ds_indexer_row_t* table, uint32_t query_len);

/*
 * (1)+(2) with query_len consecutive queries per entry (the query loop of
 * `deepseek_indexer_score_mma_rows_bf16`, whose query j sits at position
 * start_pos + j; its valid_count = min(kv_len, (start_pos + j + 1) / 4)). For
 * each entry e and query j < query_len, exactly ds_rows_indexer_topk of the
 * entry with start_pos + j, q_row + j and output_offset + 512 j. (The pages'
 * top-k kernels take the first query only; each query's own list is the
 * reading taken here.)
 *   query_len   1 .. 64 with rows * query_len <= DS_INDEX_VROWS_MAX.
 *   table       as for ds_rows_indexer_topk, except: kv_len must be at least
 *               the last query's count (start_pos + query_len) / 4,
 *               start_pos + query_len must fit u32, offset + that count - 1
 *               must fit int32, q_row .. q_row + query_len - 1 are the
 *               entry's query rows, and the output ranges are
 *               [output_offset, output_offset + 512 query_len).
 *   indices     int32, 512 per (entry, query) at output_offset + 512 j.
 *   workspace   at least ds_rows_indexer_topk_queries_workspace_bytes(...) bytes.
 * Up to four queries of an entry share each key tile on the tensor cores, so
 * the keys are read once for them. Errors as ds_rows_indexer_topk.
 */
int ds_rows_indexer_topk_queries(int rows, const ds_indexer_row_t* table, uint32_t query_len,
                                 const ds_bf16* const* index_keys, const ds_bf16* q_index, const float* w_index,
                                 int32_t* indices, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One row of a KV compressor call (`DeepSeekCompressorRow`): the row's
 * recurrent window (device fp32, updated in place) and its token's position.
 *   kv_state     fp32 [coff * ratio, coff * head_dim]     (16-B aligned)
 *   score_state  fp32, same shape                          (16-B aligned)
 *   start_pos    the decode token's absolute position, 1 .. 2^32 - 2.
 * coff is 2 for ratio 4 (overlapping windows) and 1 for ratio 128. The state
 * buffers of a call must not overlap.
 */
typedef struct {
    float* kv_state;
    float* score_state;
    uint32_t start_pos;
} ds_compressor_row_t;

/*
 * (5) Learned KV compressor, one decode token per row
 * (`deepseek_compressor_rows_bf16`, `dispatch_deepseek_compressor_rows`), for
 * (ratio, head_dim) in {(4, 128), (4, 512), (128, 512)}. With P = coff * head_dim:
 *   1. the token (t = start_pos mod ratio) is written to state row
 *      (ratio if coff == 2 else 0) + t: kv (0 where not finite) and
 *      score + ape[t] (NaN where either is not finite);
 *   2. when start_pos + 1 is a multiple of ratio, each feature f softmax-pools
 *      the window's values with its scores (coff * ratio rows; with coff == 2
 *      the first ratio rows read feature f, the others head_dim + f), rounds
 *      to bf16 (c) and writes out = bf16(c * norm / sqrt(mean(c^2) + epsilon)),
 *      or zeros when a score is NaN or +inf, or a value, pooled value, norm,
 *      sum or result is not finite; with coff == 2 the window then shifts the
 *      current block into the previous rows. Otherwise out is zero.
 *   kv, score  fp32 [rows, P]; ape fp32 [ratio, P]; norm fp32 [head_dim]
 *              (all 16-B aligned); epsilon finite and > 0.
 *   out        bf16 [rows, head_dim]                       (16-B aligned)
 */
int ds_rows_compress_kv(int rows, const ds_compressor_row_t* table, const float* kv, const float* score,
                        const float* ape, const float* norm, uint32_t ratio, uint32_t head_dim,
                        float epsilon, ds_bf16* out, void* stream);

/* ---------------------------------------------------------------------------
 * Positions and paged caches
 *
 * A decode step over paged caches is ds_rows_rope on the queries,
 * ds_rows_append on the new keys and KV rows, ds_rows_indexer_score_paged,
 * ds_rows_topk on its scores, ds_rows_sparse_attn_paged, and ds_rows_rope with
 * `inverse` on the output where the model asks for it.
 * ------------------------------------------------------------------------- */

/* Element types of ds_rows_rope, ds_rows_append and ds_rows_fetch. */
#define DS_BF16 0
#define DS_F16 1
#define DS_F32 2

/* Which elements of a rotated range [first, first + rot_dim) form pair i. */
#define DS_ROPE_INTERLEAVED 0 /* first + 2 i and first + 2 i + 1 */
#define DS_ROPE_HALF 1        /* first + i and first + rot_dim / 2 + i */

/*
 * A rotation: pair (a, b) = pair i of a row at position t becomes
 *   m (a cos x - b sin x), m (a sin x + b cos x),  x = t theta_i.
 *   turns      device uint64 [rot_dim / 2] (8-B aligned): theta_i / (2 pi) as the
 *              nearest 64-bit fraction of a turn, from ds_rows_rope_turns.
 *              t * turns[i] modulo 2^64 is the reduced angle, off by t half steps
 *              of 2^-64 of a turn: 4e-10 at the last position.
 *   first      first rotated element of a row (even when interleaved)
 *   rot_dim    rotated elements: even, 2 .. 512
 *   layout     DS_ROPE_INTERLEAVED or DS_ROPE_HALF
 *   magnitude  m: finite and > 0 (1, or a long-context attention factor)
 */
typedef struct {
    const uint64_t* turns;
    uint32_t first;
    uint32_t rot_dim;
    int layout;
    float magnitude;
} ds_rope_t;

/*
 * The turns of a rotation, written to HOST memory [rot_dim / 2] (no GPU is
 * used; copy them to the device once), each the nearest to its formula's value
 * (taken with 100 bits; YaRN's low and high, whole numbers, in 64-bit floating
 * point). theta_i = base^(-2 i / rot_dim), then
 *   factor 1:                      as it is;
 *   factor > 1, original_len 0:    theta_i / factor (linear interpolation);
 *   factor > 1, original_len > 0:  YaRN: theta_i (1 - r_i) + theta_i / factor r_i,
 *     r_i = clamp((i - low) / max(high - low, 0.001), 0, 1),
 *     low = max(floor(c(beta_fast)), 0), high = min(ceil(c(beta_slow)), rot_dim - 1),
 *     c(b) = rot_dim ln(original_len / (2 pi b)) / (2 ln base).
 *   base > 1, factor >= 1, beta_fast >= beta_slow > 0, all finite (the betas are
 *   used with original_len only).
 */
int ds_rows_rope_turns(uint32_t rot_dim, double base, double factor, uint32_t original_len, double beta_fast,
                       double beta_slow, uint64_t* turns);

/*
 * Rotary positions of x [tokens, heads, dim], one position a token:
 *   x, out     device, element type `dtype`; element strides *_token_stride and
 *              *_head_stride, the dim elements of a head contiguous. `out` may be
 *              `x` with the same strides (in place: only the rotated elements
 *              are touched); otherwise the two must not share memory, and the
 *              elements outside the rotated range are copied. The rows of `out`
 *              must not overlap; those of x may (stride 0 broadcasts).
 *   tokens     0 enqueues nothing; heads 1 .. 65536; tokens * heads < 2^31
 *   dim        1 .. 1024; first + rot_dim <= dim. Strides are at most 2^31
 *              (the stride of a side of one is not looked at).
 *   positions  device int32 [tokens]; a negative position marks padding: its
 *              rows of `out` are left as they are.
 *   inverse    nonzero: the angles are negated. This is the transpose of the
 *              rotation, so it maps the gradient of `out` to the gradient of x
 *              (m is the same factor, not its reciprocal).
 * The angle is reduced in 64-bit integers, sine and cosine are taken and the
 * products are summed in 32 bits, and the result is rounded once to `dtype`. Pointers need
 * the type's alignment; with 16-byte aligned rows and ranges the call is fastest.
 */
int ds_rows_rope(const ds_rope_t* rope, const void* x, uint64_t x_token_stride, uint64_t x_head_stride, void* out,
                 uint64_t out_token_stride, uint64_t out_head_stride, int dtype, uint64_t tokens, uint32_t heads,
                 uint32_t dim, const int32_t* positions, int inverse, void* stream);

/* Types of a paged cache. */
#define DS_CACHE_BF16 0
#define DS_CACHE_INT4 1
#define DS_CACHE_FP8 3 /* 2 is not in use */

/*
 * A paged cache of `dim`-wide rows (128: indexer keys, 512: shared K/V rows).
 * Entry e's row j lies in page id = page_table[e * table_stride + j / page_size],
 * at place j mod page_size. Entries may share pages.
 *   pages       device, num_pages pages one after another (16-B aligned), each of
 *               ds_rows_page_bytes(page_size, dim, format) bytes:
 *     DS_CACHE_BF16  bf16 [page_size][dim].
 *     DS_CACHE_INT4  a row is dim / 16 groups of 16 values n s: s an e4m3 scale,
 *                    n an integer in -7 .. 7 held as n + 8 in 4 bits. A 32-bit
 *                    word holds 8 values, value i at bits 4 (i / 2) + 16 (i mod 2);
 *                    a scale byte above 0x7E (NaN, or a sign) makes its group NaN.
 *                    dim 512: [page_size][256 bytes of values, 32 scales].
 *                    dim 128: 4 planes [page_size][16 bytes], plane c with values
 *                    32 c .. 32 c + 31 of each row, then [page_size][8 scales]
 *                    (a plane is read by consecutive threads without bank conflicts).
 *     DS_CACHE_FP8   a row is dim / 128 blocks of 128 values v 2^e: v an e4m3 byte, e =
 *                    -100 .. 7 held as the byte e + 127 (any other byte makes its block
 *                    NaN; the e4m3 bytes 0x7F and 0xFF are never written, and read as 480 and
 *                    -480). Every value is exact in bf16.
 *                    dim 512: [page_size][512 bytes of values], then [page_size][4 exponents].
 *                    dim 128: 8 planes [page_size][16 bytes], plane c with values
 *                    16 c .. 16 c + 15 of each row, then [page_size] exponents.
 *   page_table  device int32 [entries, table_stride] (4-B aligned)
 *   page_size   rows of a page: 16, 32, 64, 128 or 256
 *   num_pages   pages of the pool; num_pages * page_size < 2^31
 */
typedef struct {
    void* pages;
    const int32_t* page_table;
    uint32_t entries;
    uint32_t table_stride;
    uint32_t page_size;
    uint32_t num_pages;
    uint32_t dim;
    int format;
} ds_paged_cache_t;

/* Bytes of one page; 0 when the arguments are invalid (see ds_rows_last_error). */
size_t ds_rows_page_bytes(uint32_t page_size, uint32_t dim, int format);

/*
 * Append rows to a paged cache, rotated on the way: row i of x [tokens, dim]
 * becomes row slot[i] of entry seq[i].
 *   x          device, element type `dtype`, rows x_stride elements apart (the
 *              elements of a row contiguous); must not share memory with the pages or `values`
 *   tokens     below 2^31; 0 enqueues nothing. x_stride is at most 2^31 (of a lone row: not looked at).
 *   seq, slot  device int32 [tokens]. seq -1 marks padding: the row is skipped.
 *              The (seq, slot) pairs of a call, and the places they map to, must
 *              be distinct: of two rows for one place, any mix may remain.
 *   rope       NULL: no rotation; else rotates as ds_rows_rope with
 *   positions  device int32 [tokens]: the rotation's position, >= 0 (not the slot:
 *              a compressed row stands for several tokens); unused without rope
 *   values     optional bf16 [tokens, dim] (16-B aligned): the row as the cache
 *              now holds it (what later reads will see); skipped rows are left
 *   invalid    optional uint32 [tokens]: 1 where the row was not written because
 *              seq, slot, its page id or its position is out of range, else 0
 * The rotated row is kept in 32 bits and rounded once. DS_CACHE_BF16: to nearest
 * even. DS_CACHE_INT4, per group of 16 values y: s = e4m3(min(max|y| / 7, 448)) to
 * nearest even, n = y / s to the nearest integer (even on ties) within -7 .. 7
 * (s = 0: n = 0); a group with a non-finite value is stored as NaN. n s is exact
 * in bf16 and in fp16. DS_CACHE_FP8, per block of 128 values y: e = the least of -100 .. 7
 * with max|y| <= 448 2^e (7 if there is none), v = y 2^-e to the nearest e4m3 (even on
 * ties, saturating at 448); a block with a non-finite value is stored as NaN (exponent byte 255, its values
 * zeros).
 */
int ds_rows_append(const ds_paged_cache_t* cache, const void* x, uint64_t x_stride, int dtype, uint64_t tokens,
                   const int32_t* seq, const int32_t* slot, const ds_rope_t* rope, const int32_t* positions,
                   ds_bf16* values, uint32_t* invalid, void* stream);

/*
 * Rows read back from a paged cache: row i of out [tokens, dim] becomes row slot[i] of
 * entry seq[i], as ds_rows_append's `values` gave it: widened exactly, rounded once to
 * `dtype` (only DS_F16 can round: to nearest even, to infinity past 65504).
 *   seq, slot  device int32 [tokens]. seq -1 marks padding: the row of out is left as it
 *              is. The same (seq, slot) may come up again.
 *   out        device, element type `dtype`, rows out_stride elements apart (the elements of
 *              a row contiguous; out_stride >= dim, at most 2^31; of a lone row: not looked
 *              at); must not share memory with the pages. 32-byte aligned rows are fastest.
 *   tokens     below 2^31; 0 enqueues nothing
 *   invalid    optional uint32 [tokens]: 1 where seq, slot or its page id is out of range
 *              (the row of out is NaN), else 0
 */
int ds_rows_fetch(const ds_paged_cache_t* cache, const int32_t* seq, const int32_t* slot, void* out,
                  uint64_t out_stride, int dtype, uint64_t tokens, uint32_t* invalid, void* stream);

/*
 * ds_rows_indexer_score with the keys in a paged cache (dim 128): entry e of the
 * table reads entry e of the cache. 8- and 4-bit keys are widened exactly, and the scores
 * are bitwise those of the bf16 keys that the cache stands for. A key whose page id is
 * not in [0, num_pages), or with a NaN scale, scores -inf. DS_EINVAL when the
 * cache has fewer entries than rows, or a table row cannot reach kv_len; kv_len
 * is below 2^31; w_index and scores are 4-B aligned (DS_EALIGN). There is no status word: keys that a bounded device-side wait
 * gave up on (see DS_STATUS_WAIT_TIMEOUT) score -inf.
 */
int ds_rows_indexer_score_paged(int rows, const ds_row_t* table, const ds_paged_cache_t* keys,
                                const ds_bf16* q_index, const float* w_index, float* scores, size_t score_stride,
                                void* stream);

/*
 * ds_rows_sparse_attn with the KV rows in a paged cache (dim 512): entry e of the
 * table reads entry e of the cache. 8- and 4-bit rows are widened to bf16 exactly, so
 * the output is bitwise that of ds_rows_sparse_attn on the bf16 rows that the
 * cache stands for. A selected row whose page id is not in [0, num_pages) zeroes
 * every head of its entry, as an index out of range does; a NaN scale zeroes the
 * heads as a non-finite KV element does. The workspace (256-byte aligned, at least
 * DS_PAGED_WORKSPACE_BYTES; any other workspace of this library will do) holds the
 * call's status word only. sinks, indices and invalid are 4-B aligned (DS_EALIGN).
 */
#define DS_PAGED_WORKSPACE_BYTES 256
int ds_rows_sparse_attn_paged(int rows, const ds_row_t* table, const ds_paged_cache_t* kv, const ds_bf16* q_attn,
                              const float* sinks, size_t sinks_row_stride, const int32_t* indices, float scale,
                              ds_bf16* out, uint32_t* invalid, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes for ds_rows_prefix_attn over a cache of `format` (-1: of any); 0 when the
 * arguments are invalid (see ds_rows_last_error). 256-byte aligned, scratch between calls.
 * For DS_CACHE_FP8 and DS_CACHE_INT4 it holds the attended rows as bf16 (1 KB each) where
 * enough entries share them to widen them once beforehand; with DS_CACHE_BF16's
 * bytes the call works as well, and widens them as they are used. DS_CACHE_BF16's are below 46 MB for any call;
 * the others' are at most 128 KB more for each 128 rows, begun ones too, of the prefix and of each entry's own. */
size_t ds_rows_prefix_attn_workspace_bytes(int rows, const ds_row_t* table, uint32_t prefix_len, int format);

/*
 * Sink-softmax attention over EVERY cached row, for rows that share a prefix (samples of
 * one prompt; also layers that attend to all their compressed rows): for each entry e and head h,
 * over the slots j < kv_len of e,
 *   l_j = scale * q_attn[q_row, h, :] . g_j
 *   m = max(sink_h, max_j l_j), den = exp(sink_h - m) + sum_j exp(l_j - m)
 *   out[q_row, h, :] = bf16( sum_j exp(l_j - m) g_j / den )
 * where g_j is row j of entry 0 of the cache for j < prefix_len, else row j of entry e.
 * The prefix is read once for every two entries, and its products with the
 * queries are taken for them together.
 *   rows        1 .. DS_PREFIX_ROWS_MAX
 *   table       kv_len (1 .. 2^31 - 1, at least prefix_len) and q_row (unique) of each entry;
 *               width and index_offset are not looked at
 *   prefix_len  shared rows: 0 (nothing is shared) to the shortest kv_len. It may end
 *               inside a page: behind it each entry reads its own page.
 *   kv          dim 512, any format, with at least `rows` entries that reach kv_len
 *   q_attn      bf16 [Q, 64, 512], 16-B aligned; sinks, sinks_row_stride, scale, out and invalid
 *               as for ds_rows_sparse_attn (sinks and invalid 4-B aligned); out may be q_attn
 *   workspace   at least ds_rows_prefix_attn_workspace_bytes(..., DS_CACHE_BF16) bytes, 256-byte
 *               aligned
 * A page id out of range under one of an entry's rows zeroes every head of it (under the prefix:
 * of every entry). A head is zeroed where a q element, the sink, an element of one of
 * the entry's rows or a logit (in units of ln 2) is not finite. Memory behind kv_len, and rows of
 * an entry's own pages before prefix_len, are not read. Weights exp(l_j - m) are rounded to bf16 for
 * the product with g_j; maxima, sums and outputs are kept in 32 bits (by the tensor cores for at most 65536 slots at a
 * time). An element whose sum, with weights of up to 2^8, passes 32 bits is zero. How the slots are split over the GPU
 * depends on the whole call, and with it the last bits of a row: the same call gives the same bits, a
 * call with other rows beside it may not. Status bits as DS_STATUS_* in the workspace's
 * first word; after a wait that gave up every head of the call is zeros.
 */
int ds_rows_prefix_attn(int rows, const ds_row_t* table, uint32_t prefix_len, const ds_paged_cache_t* kv,
                        const ds_bf16* q_attn, const float* sinks, size_t sinks_row_stride, float scale, ds_bf16* out,
                        uint32_t* invalid, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Self-test of the device-side failure detection, on the current device. One
 * CTA runs the library's bounded mbarrier wait twice on a shared-memory
 * barrier: on a phase that completes, and on a phase that nothing completes,
 * each with a budget of `budget_ns` nanoseconds of %globaltimer (1,000 to
 * 10,000,000,000). It writes result[0] = 1 if the first wait succeeded and
 * result[1] = 1 if the second gave up, and ORs DS_STATUS_WAIT_TIMEOUT into
 * *status when it gives up, as the library's kernels do. Nothing faults and
 * the device stays usable. Takes about budget_ns on the GPU.
 *   status   device uint32 (zeroed by the caller beforehand)
 *   result   device uint32 [2]
 */
int ds_rows_selftest_bounded_wait(uint32_t* status, uint32_t* result, uint64_t budget_ns, void* stream);

/* Message of the last failed call on this host thread ("" if none). */
const char* ds_rows_last_error(void);

/* Library version string. */
const char* ds_rows_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSROWS_H */
