/*
 * maxsim_mx4.h -- C ABI of 4-bit embeddings: token embeddings (and the hidden
 * states and weights that make them) as microscaled 4-bit floats, the format
 * "MXFP4" of the OCP Microscaling Formats specification v1.0: elements E2M1 in
 * blocks of 32 along a row, one power of two (E8M0) for each block. A token of
 * 128 channels takes 68 bytes.
 *
 *   index:   embeddings -> maxsim_quantize_mx4 -> maxsim_fwd_mx4 (the scan)
 *            -> maxsim_topk -> maxsim_fwd_pairs (exact rescoring)
 *   serving: hidden states -> maxsim_quantize_mx4 -> maxsim_linear_mx4
 *            -> maxsim_quantize_mx4 with normalize -> maxsim_fwd_mx4
 *
 * The conventions of maxsim.h hold here too (device pointers, C-contiguous
 * rows, asynchronous on `stream`, no allocation, all checks on the host before
 * anything is enqueued, outputs alias neither inputs nor each other, results
 * bitwise reproducible run to run), with these additions:
 *   - A row of d values has B = ceil(d / 32) blocks: `codes` uint8 [T, 16 B],
 *     two codes in a byte, the first in the low half, and `scale` uint8 [T, B].
 *     The codes of the last block behind value d must be 0 or 8 (zeros);
 *     maxsim_quantize_mx4 writes zeros there.
 *   - Code c stands for (c & 8 ? -1 : 1) * {0, 0.5, 1, 1.5, 2, 3, 4, 6}[c & 7]
 *     and scale byte s for 2^(s - 127); s = 255 makes the whole block NaN.
 *   - Code arrays and float row tensors must be 16-byte aligned, bias aligned
 *     to 4 bytes; scale and mask arrays may be at any address.
 *   - Rows are independent of each other. T == 0 enqueues nothing. Row offsets
 *     are 64-bit inside the kernels.
 *   - Products of two blocks are exact; they are added in 32-bit floats, and
 *     each float output is rounded once, when it is written. A product of two
 *     blocks beyond the range of a float32 overflows to an infinity.
 */
#ifndef MAXSIM_MX4_H
#define MAXSIM_MX4_H

#include "maxsim.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row of these entry points, as in maxsim_embed.h. */
#define MAXSIM_MX4_MAX_WIDTH 131071

/*
 * Rows of floats to 4-bit codes. With v = X[t], or with normalize != 0
 * v = X[t] / ||X[t]||, and m the largest magnitude of a block of v:
 *   scale = 127 + e,  e = floor(log2 m) - 2 within [-127, 127]
 *   code  = that of the level nearest to v[k] / 2^e, the even code on a tie,
 *           magnitudes above 6 to 6 (decided exactly, as if in unlimited
 *           precision, with normalize up to the rounding of a float64 norm)
 * Blocks of zeros and masked rows (which are not looked at) get codes 0 (a
 * negative zero keeps its sign) and scale 127. With normalize, a row whose
 * largest magnitude is below 2^-110 counts as zeros.
 *   X [T, d] of `dtype` (F16, BF16, F32); mask [T] uint8 0/1 or NULL
 *   codes [T, 16 B], scale [T, B]: fully overwritten
 * A block that holds a NaN or an infinity gets scale 255 (with normalize,
 * every block of its row) and unspecified codes.
 * Errors: SHAPE (negative sizes), UNSUPPORTED (d outside 1..131071, dtype,
 * alignment), NULL, OVERFLOW (T >= 2^31).
 */
maxsim_status_t maxsim_quantize_mx4(maxsim_dtype_t dtype, const void* X, int64_t T, int64_t d,
                                    const uint8_t* mask, int normalize, uint8_t* codes,
                                    uint8_t* scale, maxsim_stream_t stream);

/*
 * The values that codes stand for, Y[t,k] = level(code) * 2^(scale - 127),
 * rounded to `dtype` (exact in F32 and BF16 up to 2^128, from where they are
 * infinities, as they are from 65520 on in F16).
 *   Y [T, d] of `dtype` (F16, BF16, F32). Errors as maxsim_quantize_mx4.
 */
maxsim_status_t maxsim_dequantize_mx4(const uint8_t* codes, const uint8_t* scale, int64_t T,
                                      int64_t d, maxsim_dtype_t dtype, void* Y,
                                      maxsim_stream_t stream);

/*
 * Matrix product of 4-bit rows with 4-bit weights (the layout of a linear
 * layer), on the matrix cores' own block-scaled form:
 *   Y[t,n] = sum_k A[t,k] W[n,k] + bias[n]
 *   A [T, K] and W [N, K] as codes and scales; bias float32 [N] or NULL;
 *   Y [T, N] of `dtype` (F16, BF16, F32)
 * A row of A or W that holds a NaN block gives NaN in its row or channel.
 * Errors: SHAPE (negative sizes), UNSUPPORTED (K outside 1..131071, N < 1,
 * dtype, alignment), NULL, OVERFLOW (T >= 2^31 or N > 2^26).
 */
maxsim_status_t maxsim_linear_mx4(maxsim_dtype_t dtype, const uint8_t* A, const uint8_t* a_scale,
                                  const uint8_t* W, const uint8_t* w_scale, const float* bias,
                                  int64_t T, int64_t N, int64_t K, void* Y,
                                  maxsim_stream_t stream);

/*
 * Cross-product MaxSim of 4-bit queries and documents: maxsim_fwd on the
 * values that the codes stand for.
 *   Q [Nq, Lq, d] and D [Nd, Ld, d] as codes and scales, 1 <= d <= 1024
 *   masks, scores [Nq, Nd] and argmax [Nq, Nd, Lq] (or NULL) as in maxsim_fwd
 * Similarities are sums in float32, as in the other forwards, so the argmax is
 * that of the rounded ones; ties among equal maxima go to the lowest index (of the
 * tokens that count, where all of them are at -Inf by products that overflow).
 * Masked tokens and rows are not looked at, whatever they hold. If a token that
 * counts holds a NaN block, the scores that it enters are NaN, and the argmax
 * is unspecified (in [0, Ld)).
 * Errors as maxsim_fwd; OVERFLOW also for Nq, Lq or Ld >= 2^31 - 64 or
 * Nd >= 2^31.
 */
maxsim_status_t maxsim_fwd_mx4(const uint8_t* Q, const uint8_t* q_scale, const uint8_t* D,
                               const uint8_t* d_scale, int64_t Nq, int64_t Nd, int64_t Lq,
                               int64_t Ld, int64_t d, const uint8_t* q_mask,
                               const uint8_t* d_mask, float* scores, int32_t* argmax,
                               maxsim_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAXSIM_MX4_H */
