/*
 * maxsim_loss.h -- C ABI of what follows the scores: the log probabilities of
 * given columns of a score matrix under the softmax of their row, with their
 * ranks, the row's entropy and its best columns, and the gradient of those
 * probabilities and of the entropy.
 *
 *   training:  maxsim_fwd -> maxsim_logprob_fwd -> loss on logp (contrastive:
 *              one right document a row; distillation: the taught documents,
 *              weighted) -> maxsim_logprob_bwd -> maxsim_bwd as grad_scores
 *   retrieval: scores of a scan -> ranks of the judged documents, hard
 *              negatives (the best columns), how sure a query is (the entropy)
 *
 * The conventions of maxsim.h hold here too (device pointers, C-contiguous
 * rows, asynchronous on `stream`, no allocation, all checks on the host before
 * anything is enqueued, outputs alias neither inputs nor each other, results
 * bitwise reproducible run to run), with these additions:
 *   - Row i of X [Nq, Nd] holds scores; scale, from 2^-64 to 2^64, multiplies
 *     them (the inverse temperature). mask [Nq, Nd] uint8 0/1 or NULL: columns with mask 0 are not
 *     looked at. A column is a candidate if its mask is not 0 and its score is
 *     not -Inf. Scores of the type's lowest value are candidates like others.
 *   - targets [Nq, P] int32: columns; a column may be named more than once. An
 *     entry outside [0, Nd) names none.
 *   - With m the largest candidate of a row, z = scale (x - m) and
 *     L = log sum exp(z) over the candidates: log p = z - L. Sums are held in
 *     float64, each float output is rounded once.
 *   - Rows are independent of each other. A row that holds a NaN or +Inf among
 *     its candidates gives NaN in every float output; its ranks and best columns
 *     are unspecified, in [-1, Nd).
 *   - Every array is aligned to its element type, the workspace to 16 bytes.
 */
#ifndef MAXSIM_LOSS_H
#define MAXSIM_LOSS_H

#include "maxsim.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAXSIM_LOGPROB_MAX_K 1024 /* most best columns of a row */

/* Bytes of workspace that maxsim_logprob_fwd needs for these sizes, 0 for rows of
 * up to 4096 columns; -1 for sizes that it refuses. The workspace holds nothing
 * between calls; calls that may run at the same time need one each. */
int64_t maxsim_logprob_workspace(int64_t Nq, int64_t Nd, int64_t P, int64_t K);

/*
 *   logp [Nq, P] float32: log p of the targets; -Inf of a target that is no
 *        candidate, 0 where an entry names none
 *   rank [Nq, P] int32 or NULL: how many candidates come before the target in
 *        decreasing order of scores, equal ones in increasing column order; -1
 *        where the target is no candidate or none is named
 *   norm [Nq, 2] float32: m and L, what the backward needs (a row without
 *        candidates: -Inf and -Inf)
 *   entropy [Nq] float32 or NULL: -sum p log p (a row without candidates: 0)
 *   top_idx [Nq, K] int32, top_logp [Nq, K] float32: the K best candidates in the
 *        order of the ranks; -1 and -Inf where there are fewer. Not used with K = 0.
 *   X [Nq, Nd] of `dtype` (F16, BF16, F32)
 * Nq == 0 enqueues nothing. Errors: SHAPE (negative sizes, a workspace that is too
 * small), UNSUPPORTED (dtype, K > 1024, a scale outside its range, alignment),
 * NULL, OVERFLOW (Nq, Nd or P >= 2^31 - 4096, Nq * ceil(Nd / 4096) or
 * Nq * P >= 2^31).
 */
maxsim_status_t maxsim_logprob_fwd(maxsim_dtype_t dtype, const void* X, int64_t Nq, int64_t Nd,
                                   float scale, const uint8_t* mask, const int32_t* targets,
                                   int64_t P, int64_t K, float* logp, int32_t* rank, float* norm,
                                   float* entropy, int32_t* top_idx, float* top_logp,
                                   void* workspace, int64_t workspace_bytes,
                                   maxsim_stream_t stream);

/*
 * Gradient of sum grad_logp * logp + sum grad_entropy * entropy:
 *   dX[i,c] = scale (sum of grad_logp[i,p] over targets p that name c
 *                    - p_c (G + grad_entropy[i] (log p_c + entropy[i])))
 * with G the sum of grad_logp over the row's targets that are candidates; columns
 * that are no candidates get 0. (The best columns' log probabilities are
 * differentiated by passing them as targets.)
 *   X, scale, mask, targets, norm, entropy as in the forward and from it;
 *   grad_logp [Nq, P] float32; grad_entropy [Nq] float32, with entropy, or both
 *   NULL; dX [Nq, Nd] of `dx_dtype` (F16, BF16, F32): fully overwritten
 * Gradients of targets that are named more than once are added in the order of p
 * (for a column of probability above 0.6 in another order, a fixed one too). Such a
 * column's dX is formed from 1 - p_c, which L holds to 32 bits beside a 2^-47 of the
 * float64 sums, so that it does not lose the digits of a p_c next to 1.
 * Errors: SHAPE (negative sizes), UNSUPPORTED (dtypes, scale, alignment), NULL
 * (also one of entropy and grad_entropy without the other), OVERFLOW as above.
 */
maxsim_status_t maxsim_logprob_bwd(maxsim_dtype_t dtype, const void* X, int64_t Nq, int64_t Nd,
                                   float scale, const uint8_t* mask, const int32_t* targets,
                                   int64_t P, const float* norm, const float* entropy,
                                   const float* grad_logp, const float* grad_entropy,
                                   maxsim_dtype_t dx_dtype, void* dX, maxsim_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAXSIM_LOSS_H */
