/*
 * libkdloss, the layers on the model's side of the output head: what makes
 * the hidden states H that the losses take, and what passes their gradient dH
 * on.
 *
 *  - token embeddings, from a table or from the columns of the head itself
 *    (tied weights), and their gradient;
 *  - layer norm, forward and backward, with the gradients of its weight and
 *    bias;
 *  - rows held in 8 bits: activations kept for a backward pass in half the
 *    memory, and the operands of the next;
 *  - the product of 8-bit integers with a scale for each token and channel: a
 *    frozen head, or a frozen layer, in half its bytes.
 *
 * Conventions (layouts, ownership, streams, status codes, error text) are
 * those of kdloss.h: dense row-major arrays, caller-allocated buffers and
 * workspace, every argument checked on the host before anything is enqueued,
 * no synchronisation, no state between calls, the same bits for the same
 * call.  Element types are KD_F32, KD_BF16 and KD_F16.  Arrays need no more
 * alignment than their elements' except where a call says so, and rows may
 * have any length: whole rows of 16-byte pieces are only the fastest.
 * Masks are uint8 [T], 1 = valid, NULL = all valid; what masked rows hold is
 * never read.  Values on the device are not checked; what each call does with
 * values outside their range is said there, and no value leads to a read or
 * write outside the arrays.  An output may not overlap an input or another
 * output, except where a call says so.  T, V and d must be below 2^30, 2^30
 * and 2^24 (KD_ERR_UNSUPPORTED).
 */
#ifndef KDLAYERS_H
#define KDLAYERS_H

#include "kdpolicy.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- token embeddings
 * out[t] = scale E[tokens[t]], rounded once to the table's type dt.  The table
 * is E [V,d] (tied = 0), or the head W [d,V] of the losses (tied = 1), token
 * v's embedding then being its column v.  Masked rows get zeros.  A valid
 * token outside [0, V) gets a row of NaN.  A vocabulary shard [v0, v0 + Vs)
 * takes tokens - v0 and a mask of the rows whose tokens are its own; the shards'
 * outputs add up to the whole head's, and the backward call needs the same two.
 * tokens [T] int32; out [T,d] of type dt. */
kd_status kd_embedding_fwd(const int32_t* tokens, const void* table, const uint8_t* mask, float scale, int64_t T,
                           int64_t V, int64_t d, kd_dtype dt, int32_t tied, void* out, void* stream);
/* Workspace bytes for kd_embedding_bwd: the sorted tokens (16 bytes a token), 4
 * bytes for each of the V tokens, float32 partial sums (up to d / 2 bytes a token) and, if tied, a float32 row
 * of sums for each token (in slabs of columns of 1 GiB at most, or of 64
 * columns). */
kd_status kd_embedding_workspace_size(int64_t T, int64_t V, int64_t d, int32_t tied, size_t* bytes);
/* dE_v = scale sum of grad[t] over the valid t with tokens[t] = v, added up in
 * float32 in an order that T and the tokens decide (no atomics), rounded once
 * to grad_dt.
 * grad [T,d] of type dt; grad_table of type grad_dt, laid out as the table.
 * accumulate = 0: all of grad_table is written.  accumulate = 1: dE_v is added
 * to what it holds (the sum rounded once) at the tokens that occur, and the
 * rest is neither read nor written: with tied = 1 the head's own gradient dW
 * takes the embedding's share.  Valid tokens outside [0, V) add nothing.
 * T = 0 writes zeros, or nothing with accumulate. */
kd_status kd_embedding_bwd(const void* grad, const int32_t* tokens, const uint8_t* mask, float scale, int64_t T,
                           int64_t V, int64_t d, kd_dtype dt, kd_dtype grad_dt, int32_t tied, int32_t accumulate,
                           void* grad_table, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- rows in 8 bits
 * A row of d values in groups of `group` consecutive ones (32, 64, 128, 256 or
 * 512; the last group of a row may be shorter; 0: the whole row is one group)
 * is held as q [T,d], one byte a value, and scale [T, ceil(d / group)]
 * float32:
 *   KD_ROWS_INT8   scale = max |x| / 127, q = x / scale to the nearest integer
 *   KD_ROWS_E4M3   scale = max |x| / 448, q = x / scale to the nearest value
 *                  of the 8-bit format with 4 exponent and 3 significand bits
 *                  (largest 448, no infinities)
 * The scale is rounded to float32, ties to even, also below its normal range;
 * q is the nearest to the exact quotient of x and that scale, ties to even, but
 * no larger than 127 or 448 (where such a scale was rounded down).  A group of zeros, or one whose scale rounds
 * to 0, has scale 0 and q 0.  A group with an infinity or a NaN has scale NaN
 * and q 0: it comes back as NaN. */
typedef enum kd_rows_kind { KD_ROWS_NONE = 0, KD_ROWS_INT8 = 1, KD_ROWS_E4M3 = 2, KD_ROWS_KIND_MAX_ENUM = 0x7fffffff } kd_rows_kind;
kd_status kd_rows_quantize(const void* x, int64_t T, int64_t d, kd_dtype dt, kd_rows_kind kind, int64_t group, void* q,
                           float* scale, void* stream);
/* out [T,d] of type dt = q scale, the product in float32, rounded to dt. */
kd_status kd_rows_dequantize(const void* q, const float* scale, int64_t T, int64_t d, kd_rows_kind kind, int64_t group,
                             kd_dtype dt, void* out, void* stream);

/* ---------------------------------------------------------------- layer norm
 * Per valid row of x [T,d], in float32:
 *   mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
 *   y = (x - mean) rstd weight + bias, rounded once
 * weight and bias [d] of type wdt (that of x, or KD_F32); either may be NULL
 * (1 and 0).  Masked rows get y = mean = rstd = 0.  mean, rstd [T] float32 are
 * kept for the backward call (both may be NULL where there is none).
 * kind: KD_ROWS_NONE, or the form in which the call also leaves x for the
 * backward call, in q [T,d] and scale as kd_rows_quantize gives them (masked
 * rows: 0). */
kd_status kd_layer_norm_fwd(const void* x, const void* weight, const void* bias, const uint8_t* mask, double eps,
                            int64_t T, int64_t d, kd_dtype dt, kd_dtype wdt, void* y, float* mean, float* rstd,
                            kd_rows_kind kind, int64_t group, void* q, float* scale, void* stream);
/* Workspace bytes for kd_layer_norm_bwd: float32 partial sums. */
kd_status kd_layer_norm_workspace_size(int64_t T, int64_t d, size_t* bytes);
/* For the upstream gradient grad [T,d] (of x's type dt), with
 * h = (x - mean) rstd and g = grad weight:
 *   dx = rstd (g - mean_d(g) - h mean_d(g h))   [T,d] of type dt, 0 on masked rows
 *   dweight = sum_t grad h, dbias = sum_t grad  [d] of type wdt, added up in float32
 * Each of the three may be NULL where it is not wanted, not all.
 * x, or with kind != KD_ROWS_NONE (then x is NULL) q and scale, the forward's:
 * x then is what they stand for, mean and rstd are still those of the x that
 * the forward call saw.  T = 0 sets dweight and dbias to zero. */
kd_status kd_layer_norm_bwd(const void* grad, const void* x, const void* weight, const uint8_t* mask,
                            const float* mean, const float* rstd, int64_t T, int64_t d, kd_dtype dt, kd_dtype wdt,
                            kd_rows_kind kind, int64_t group, const void* q, const float* scale, void* dx,
                            void* dweight, void* dbias, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- product of 8-bit integers
 * out[t,v] = x_scale[t] w_scale[v] sum_k x[t,k] w[v,k], the sum exact in 32-bit
 * integers, the two products in float32, rounded to out_dt.
 * x [T,d] int8 and w [V,d] int8 (one row a channel: the transposed head),
 * 16-byte aligned, d a multiple of 16 below 2^17; x_scale [T], w_scale [V]
 * float32; out [T,V].  kd_rows_quantize with KD_ROWS_INT8 and group 0 gives
 * such operands. */
kd_status kd_int8_matmul_workspace_size(int64_t T, int64_t d, int64_t V, size_t* bytes);
kd_status kd_int8_matmul(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale, int64_t T,
                         int64_t d, int64_t V, kd_dtype out_dt, void* out, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* KDLAYERS_H */
