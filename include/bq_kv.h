/*
 * bq_kv.h -- C ABI of the quantised KV cache's operators for B200 (sm_100a):
 * writing new keys and values into a preallocated cache, reading them back,
 * and decode attention over a 4-bit cache.
 *
 * Beside bq_attn_decode_q8 (bq.h), which reads a Q8 cache.  The conventions of
 * bq.h hold for every call here: the caller owns every buffer, nothing is
 * allocated, calls are asynchronous on `stream` (launched with the
 * programmatic-dependent-launch attribute, so they read and write no memory
 * before the previous kernel on the stream has completed), a call whose return
 * code is not BQ_OK launched nothing, what the device detects is OR-ed into
 * *dev_status as 1 << code, and the device never traps.  Every call can be
 * captured into a CUDA graph.  Results are deterministic for a given device
 * and arguments.
 *
 * In a decode step the calls follow each other on one stream:
 *
 *   q|k|v projection (bq_gemv_*) -> bq_kv_append_* -> attention -> o projection
 *
 * and lens[b] of the attention is start[b] + count[b] of the append.
 */
#ifndef BQ_KV_H
#define BQ_KV_H

#include "bq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further status code of this header's calls (bq_status_string knows it).
 * device: a row's position is outside [0, Tmax), or a count outside [0, T]. */
enum { BQ_ERR_POSITION = 10 };

/* Element types of rows and outputs. */
enum { BQ_F32 = 0, BQ_F16 = 1, BQ_BF16 = 2 };

/* A preallocated 4-bit KV cache of Tmax positions per (sequence, KV head):
 * keys and values quantised in the Q4 format of the weights (32-element
 * blocks along the head dimension, fp16 scale = fp16(absmax / 7), 4-bit code
 * q, value = scale * (q - 8); byte i of a block holds element i in its low
 * nibble and element i + 16 in its high nibble).  Keys and values have the
 * same position-major layout: a position's row is what bq_quantize_q4 makes of
 * a D-column matrix row, with its D/32 scales not padded.
 *   k_codes, v_codes    uint8 [B][Hkv][Tmax][D/2]
 *   k_scales, v_scales  fp16 bits [B][Hkv][Tmax][D/32]
 * Device pointers, 16-byte aligned, caller-owned.  D is 64 or 128, Tmax a
 * multiple of 32, B * Hkv * Tmax < 2^31.  144 bytes a position and KV head at
 * D = 128, against 272 for the Q8 cache and 512 in fp16.  The planes need no
 * initialisation: no call reads a position past the valid ones into a result. */
typedef struct bq_kv_cache_q4 {
    uint8_t *k_codes;
    uint16_t *k_scales;
    uint8_t *v_codes;
    uint16_t *v_scales;
    int32_t D, Tmax;
} bq_kv_cache_q4;

/* Dense key and value rows: T tokens of each of B sequences, Hkv heads of D
 * elements.  Row (b, i, h) starts at k + b * k_batch + i * k_token + h * k_head
 * elements (v likewise) and its D elements are contiguous, so k and v may be
 * column ranges of one q|k|v projection output.  Base addresses and strides
 * are multiples of 16 bytes; a source's strides may be 0 (a broadcast row),
 * a destination's rows must not overlap. */
typedef struct bq_kv_rows {
    void *k;
    void *v;
    int64_t k_batch, k_token, k_head;    /* strides in elements */
    int64_t v_batch, v_token, v_head;
    int32_t dtype;                       /* BQ_F32, BQ_F16 or BQ_BF16: both k and v */
    int32_t T;                           /* tokens a sequence, 1 .. min(Tmax, 2^30) */
} bq_kv_rows;

/* Quantise new keys and values as they are written to the cache: row i of
 * sequence b (i < count[b]) goes to position start[b] + i, for every head.
 * Codes and scales are bit for bit those of bq_quantize_q4 / bq_quantize_q8 on
 * the fp32 values of the row.  Nothing else of the cache is touched.
 *   kv      the cache (its planes are written); q8: the cache of
 *           bq_attn_decode_q8 (D = 128, Tmax a multiple of 128; the const of
 *           its fields is the reader's view)
 *   rows    source rows (read only)
 *   B, Hkv  sequences and KV heads of the cache and of the rows; Hkv <= 65535
 *   start   device int32 [B]: first position written
 *   count   device int32 [B], or NULL: every sequence writes T rows.  Rows from
 *           count[b] on are not read, nor are those past the cache's end
 * Device status: BQ_ERR_POSITION for rows whose position is outside [0, Tmax)
 * (those are not written) and for counts outside [0, T] (taken as the nearer
 * end); BQ_ERR_RANGE for a 32-block that is not finite or whose scale overflows
 * fp16 (it is stored as zeros).
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (D, Tmax, Hkv, T, dtype, cache size),
 * BQ_ERR_BATCH (B < 1), BQ_ERR_ALIGN, BQ_ERR_CUDA. */
BQ_API int32_t bq_kv_append_q4(const bq_kv_cache_q4 *kv, const bq_kv_rows *rows, int32_t B,
                               int32_t Hkv, const int32_t *start, const int32_t *count,
                               int32_t *dev_status, void *stream);
BQ_API int32_t bq_kv_append_q8(const bq_kv_cache *kv, const bq_kv_rows *rows, int32_t B,
                               int32_t Hkv, const int32_t *start, const int32_t *count,
                               int32_t *dev_status, void *stream);

/* Read cached positions back: position start[b] + i of sequence b (i <
 * count[b]) becomes row i, for every head; value = scale * code, exact in fp32
 * and rounded once (to nearest even) to fp16 or bf16.  A magnitude above
 * fp16's range becomes infinite.  Rows from count[b] on, and rows of positions
 * outside [0, Tmax), are left as they were.
 *   rows    destination; k or v (not both) may be NULL and is then skipped; k
 *           and v at one address are refused (BQ_ERR_SHAPE)
 * Other arguments, device status (BQ_ERR_POSITION) and errors as
 * bq_kv_append_*. */
BQ_API int32_t bq_kv_read_q4(const bq_kv_cache_q4 *kv, const bq_kv_rows *rows, int32_t B,
                             int32_t Hkv, const int32_t *start, const int32_t *count,
                             int32_t *dev_status, void *stream);
BQ_API int32_t bq_kv_read_q8(const bq_kv_cache *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
                             const int32_t *start, const int32_t *count, int32_t *dev_status,
                             void *stream);

/* Bytes of workspace bq_attn_decode_q4 needs: arrival counters and CTA
 * partials, independent of B, Hkv and Tmax.  0 on a bad shape. */
BQ_API size_t bq_attn_q4_workspace_bytes(int32_t D, int32_t Tq, int32_t G);

/* Decode attention over a Q4 cache: for sequence b, query token i and query
 * head j (KV head h = j / G),
 *   s_t = scale * sum_d q[b][i][j][d] K[t][d]
 *   p   = softmax of s over t < lens[b] - (Tq - 1 - i)
 *   o[b][i][j][d] = sum_t p_t V[t][d].
 * With Tq = 1 this is a decode step; with Tq > 1 the Tq newest positions of a
 * sequence are its query tokens' own (the drafted tokens of a verification
 * step), each seeing the positions up to its own.
 *   kv      the cache (read only)
 *   q       device fp16 bits [B][Tq][Hkv*G][D]
 *   lens    device int32 [B]: valid positions of sequence b, the query tokens'
 *           included (clamped to [0, Tmax]).  A query token that sees no
 *           position gets o = 0.  Nothing that a query token does not see is
 *           read into its result, whatever the cache holds there.  (A value
 *           scale that is not finite makes NaN of its block's 32 elements for
 *           the tokens that see it; a NaN key scale, of whole rows.)
 *   Tq      query tokens a sequence, 1..32
 *   G       query heads per KV head, 1..16
 *   scale   softmax scale, |scale| <= 1e18 (any sign; below 1e-28 as 1e-28)
 *   o       device [B][Tq][Hkv*G][D], overwritten; o_dtype BQ_F32 or BQ_F16
 *           (the input type of the next bq_gemv); must not overlap q (at q's
 *           address: BQ_ERR_SHAPE)
 *   ws      device workspace >= bq_attn_q4_workspace_bytes(D, Tq, G),
 *           zero-filled before first use, left zero-filled by every call that
 *           completes; not shared with calls that may run at the same time
 *   dev_status  as the other calls'; there is nothing this one reports, and it
 *           may be NULL
 * Rounding: scores, softmax sums and outputs accumulate in fp32 and the codes
 * enter the tensor cores exactly.  Weights are made from differences of unscaled
 * scores, so scores may be of any size.  Each softmax weight times its value scale
 * enters as two fp16 terms: off by 2^-21 of it or, where that is more, by 2^-35
 * of the largest finite value scale (2^-14 at least) below lens[b].  BQ_F16 output is
 * the BQ_F32 output rounded once.
 * Errors: BQ_ERR_NULL, BQ_ERR_SHAPE (D, Tmax, Hkv, G, Tq, scale, o_dtype, cache
 * size; also B * Hkv * Tmax * passes >= 2^35, which Tq * G <= 256 never
 * reaches), BQ_ERR_BATCH (B < 1), BQ_ERR_ALIGN, BQ_ERR_WORKSPACE, BQ_ERR_CUDA. */
BQ_API int32_t bq_attn_decode_q4(const bq_kv_cache_q4 *kv, const uint16_t *q, const int32_t *lens,
                                 int32_t B, int32_t Tq, int32_t Hkv, int32_t G, float scale,
                                 void *o, int32_t o_dtype, void *ws, size_t ws_bytes,
                                 int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* BQ_KV_H */
