/*
 * maxsim_embed.h -- C ABI of the embedding head: the operators between an
 * encoder's hidden states and the token embeddings that maxsim.h scores.
 *
 *   serving:  hidden states -> maxsim_quantize_tok -> maxsim_embed_i8
 *             -> maxsim_fwd_i8_tok (codes) or maxsim_fwd (floats)
 *   training: maxsim_dropout_fwd -> projection -> maxsim_normalize_fwd
 *             -> maxsim_fwd, maxsim_bwd -> maxsim_normalize_bwd
 *             -> the projection's gradients -> maxsim_dropout_bwd
 *
 * The conventions of maxsim.h hold here too (device pointers, C-contiguous
 * rows, asynchronous on `stream`, no allocation, all checks on the host before
 * anything is enqueued, outputs alias neither inputs nor each other, results
 * bitwise reproducible run to run), with these additions:
 *   - A "row" is one token. T rows are processed independently of each other,
 *     so NaN or Inf in one row reaches no other row.
 *   - mask [T] uint8 0/1 or NULL: rows with mask 0 (padding) are not looked
 *     at, whatever they hold (NaN included); their outputs are written with
 *     the values each entry point names.
 *   - Float row tensors X, Y, E, dY, dX and int8 row tensors A, W, codes must
 *     be 16-byte aligned, every other array aligned to its element type. Rows
 *     whose byte length is not a multiple of 16 run more slowly.
 *   - T == 0 enqueues nothing. Row offsets are 64-bit inside the kernels.
 *   - Sums, norms and statistics are held in 32-bit floats or more (the
 *     products of 8-bit integers in exact int32); each float output is rounded
 *     once, when it is written.
 *   - A row whose largest magnitude is below 2^-110 counts as a row of zeros
 *     where a row is divided by its norm or its largest magnitude.
 */
#ifndef MAXSIM_EMBED_H
#define MAXSIM_EMBED_H

#include "maxsim.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row of these entry points: 131071 * 128^2 < 2^31, so an int32 sum of
 * products of any int8 values cannot overflow. */
#define MAXSIM_EMBED_MAX_WIDTH 131071
/* Widest embedding of maxsim_embed_i8 (the widest that maxsim.h scores). */
#define MAXSIM_EMBED_MAX_DIM 1024

/*
 * Rows of floats to 8-bit codes with one symmetric scale per token, the form
 * that maxsim_fwd_i8_tok and maxsim_linear_i8 take:
 *   m_t = max_k |X[t,k]|,  codes[t,k] = the integer nearest 127 X[t,k] / m_t
 *   (ties to even; decided exactly, as if in unlimited precision)
 *   scale[t] = m_t / 127, so that codes * scale is X, or with normalize != 0
 *   scale[t] = 1 / ||127 X[t] / m_t||, so that codes * scale is X[t] / ||X[t]||
 * Rows of zeros and masked rows get codes 0 and scale 1 (a scale is always
 * positive).
 *   X [T, d] of `dtype` (F16, BF16, F32); mask [T] or NULL
 *   codes int8 [T, d] in [-127, 127], scale float32 [T]: fully overwritten
 * A row that holds a NaN or an infinity (and is not masked) gets scale NaN and
 * unspecified codes, so that whatever is computed from it is NaN.
 * Errors: SHAPE (negative sizes), UNSUPPORTED (d outside 1..131071, dtype,
 * alignment), NULL, OVERFLOW (T >= 2^31).
 */
maxsim_status_t maxsim_quantize_tok(maxsim_dtype_t dtype, const void* X, int64_t T, int64_t d,
                                    const uint8_t* mask, int normalize, int8_t* codes,
                                    float* scale, maxsim_stream_t stream);

/*
 * Matrix product of 8-bit integers with a scale for each token and for each
 * output channel (the layout of a linear layer):
 *   Y[t,n] = a_scale[t] * w_scale[n] * sum_k A[t,k] W[n,k] + bias[n]
 * The sum is exact (int32); it is converted to float32, multiplied by the
 * float32 product of the two scales, the bias is added, and the result is
 * rounded to `dtype`.
 *   A int8 [T, K], a_scale float32 [T]; W int8 [N, K], w_scale float32 [N];
 *   bias float32 [N] or NULL; Y [T, N] of `dtype` (F16, BF16, F32). Any int8
 *   value is allowed, -128 included; scales may have any sign.
 * Errors: SHAPE (negative sizes), UNSUPPORTED (K outside 1..131071, N < 1,
 * dtype, alignment), NULL, OVERFLOW (T >= 2^31 or N > 2^26).
 */
maxsim_status_t maxsim_linear_i8(maxsim_dtype_t dtype, const int8_t* A, const float* a_scale,
                                 const int8_t* W, const float* w_scale, const float* bias,
                                 int64_t T, int64_t N, int64_t K, void* Y,
                                 maxsim_stream_t stream);

/*
 * maxsim_linear_i8 with each row divided by its Euclidean norm, in one pass:
 * the projection from hidden states to token embeddings.
 *   y[t] as in maxsim_linear_i8 with N = d,  E[t] = y[t] / ||y[t]||
 * dtype F16, BF16 or F32: E [T, d] of that type, e_scale unused (NULL).
 *   Rows of zeros and masked rows give zeros.
 * dtype I8: E int8 [T, d] codes of y[t] and e_scale float32 [T], as
 *   maxsim_quantize_tok with normalize makes them of y: y is the exact sum
 *   times the exact product of the scales plus the bias, rounded once to
 *   float64, and its codes are decided exactly, ties to even. Rows of zeros
 *   and masked rows give codes 0, scale 1.
 * A row whose y holds a NaN or an infinity gives NaN: as floats in every
 * channel, as codes (unspecified) through scale NaN.
 * E holds scratch until it is written.
 *   mask [T] uint8 or NULL; a mask needs no care for what A and a_scale hold
 *   in the rows it drops.
 * Errors: as maxsim_linear_i8; UNSUPPORTED also for d outside 1..1024; NULL
 * also for a missing e_scale with I8.
 */
maxsim_status_t maxsim_embed_i8(maxsim_dtype_t dtype, const int8_t* A, const float* a_scale,
                                const int8_t* W, const float* w_scale, const float* bias,
                                const uint8_t* mask, int64_t T, int64_t d, int64_t K, void* E,
                                float* e_scale, maxsim_stream_t stream);

/*
 * Rows divided by their Euclidean norm:
 *   Y[t] = X[t] / ||X[t]||,  rnorm[t] = 1 / ||X[t]||
 * Rows of zeros and masked rows give Y = 0 and rnorm = 0.
 *   X [T, d] of x_dtype, Y [T, d] of y_dtype (F16, BF16, F32 each),
 *   rnorm float32 [T]: what the backward needs beside X
 * Norms above 2^126 make rnorm subnormal, with fewer bits. Errors as
 * maxsim_quantize_tok.
 */
maxsim_status_t maxsim_normalize_fwd(maxsim_dtype_t x_dtype, const void* X, int64_t T, int64_t d,
                                     const uint8_t* mask, maxsim_dtype_t y_dtype, void* Y,
                                     float* rnorm, maxsim_stream_t stream);

/*
 * Gradient of maxsim_normalize_fwd through the unrounded Y:
 *   u = X[t] rnorm[t],  dX[t] = rnorm[t] (dY[t] - u <u, dY[t]>)
 * Rows with rnorm 0 (zeros, masked) give dX = 0 and are not looked at.
 *   X [T, d] of x_dtype and rnorm [T] as in the forward; dY [T, d] float32
 *   (the dQ or dD of maxsim_bwd); dX [T, d] of dx_dtype
 * Errors as maxsim_quantize_tok.
 */
maxsim_status_t maxsim_normalize_bwd(maxsim_dtype_t x_dtype, const void* X, const float* rnorm,
                                     const float* dY, int64_t T, int64_t d,
                                     maxsim_dtype_t dx_dtype, void* dX, maxsim_stream_t stream);

/*
 * Dropout with a counter-based generator: whether element i is dropped is a
 * function of (seed, step, i), computed where it is needed, so no mask is
 * stored and the backward repeats the forward's.
 *   q = floor(65536 p + 1/2)  (p is rounded to a multiple of 2^-16)
 *   element i is dropped where its 16 bits are below q: bits 16 (i mod 2) ..
 *   of word (i mod 8) / 2 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
 *   SC 2011) at counter (floor(i / 8), s), key seed, each 64-bit value as two
 *   32-bit words, low first
 *   s = step + *step_dev (modulo 2^64; step_dev NULL counts as 0). A captured
 *   graph that advances the step in device memory draws a new mask at every
 *   replay.
 *   Y[i] = 0 where dropped (whatever X[i] holds), else X[i] * 65536/(65536 - q)
 * in float32, rounded to `dtype`; p = 0 copies X, p = 1 gives zeros. The
 * scale is that of the rounded p, so the expectation of Y is X.
 *   X, Y [n] of `dtype` (F16, BF16, F32); one (seed, step) pair for each
 *   tensor that is dropped from
 * maxsim_dropout_bwd: dX[i] = 0 where dropped, else dY[i] * 65536/(65536 - q),
 * for the forward's p, seed and step.
 * n == 0 enqueues nothing. Errors: SHAPE (n < 0), UNSUPPORTED (p not in
 * [0, 1], dtype, alignment), NULL, OVERFLOW (n >= 2^43).
 */
maxsim_status_t maxsim_dropout_fwd(maxsim_dtype_t dtype, const void* X, int64_t n, double p,
                                   uint64_t seed, uint64_t step, const uint64_t* step_dev, void* Y,
                                   maxsim_stream_t stream);
maxsim_status_t maxsim_dropout_bwd(maxsim_dtype_t dtype, const void* dY, int64_t n, double p,
                                   uint64_t seed, uint64_t step, const uint64_t* step_dev, void* dX,
                                   maxsim_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAXSIM_EMBED_H */
