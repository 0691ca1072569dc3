/*
 * ds_logprob.h -- C ABI of what is read off a row of logits: the log
 * probability of a given token, the entropy and the likeliest alternatives,
 * and the gradient of all of them.  Part of libds_topk.so; status codes,
 * dtypes and error texts are those of ds_topk.h.
 *
 * With z = scale * logits of a row:
 *   lse      = log sum_i exp z_i
 *   logprob  = z_t - lse of the row's given token t
 *   entropy  = lse - sum_i p_i z_i,  p_i = exp(z_i - lse)
 *   top      = z - lse of the k first tokens by (logit descending, index
 *              ascending), NaN above +inf and -0 = +0 as in ds_topk
 * A row's logits of -inf are tokens that cannot come: p = 0, and they add
 * nothing to the entropy or its gradient.  A row of nothing else has
 * lse = -inf, logprob and top -inf, entropy 0 and gradient 0.  A row with a NaN
 * or +inf has lse, logprob, entropy and top NaN (idx is by the order), and so
 * has its gradient.  A given token outside [0, vocab) (padding) has logprob 0
 * and takes no part in the gradient.
 * Sums, maxima and results are held in 32 bits.
 *
 * Asynchrony: both functions only enqueue work on `stream`, allocate nothing
 * and keep nothing from call to call.  Argument errors are reported before
 * anything is enqueued.
 */
#ifndef DS_LOGPROB_H
#define DS_LOGPROB_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Largest k of ds_token_logprobs, and vocab is below DS_LOGPROB_MAX_VOCAB. */
#define DS_LOGPROB_MAX_K 32
#define DS_LOGPROB_MAX_VOCAB 0x7fffffc0

/*
 * ds_token_logprobs
 *   logits    device, row r at r * row_stride elements of `dtype` (DS_FP32,
 *             DS_BF16 or DS_FP16), vocab of them side by side; any alignment
 *             to elements (rows of 16-bit types are read 16 bytes at a time
 *             wherever they start)
 *   rows      >= 0 (0 is a no-op)
 *   row_stride  >= vocab (any where rows < 2)
 *   tokens    device int32[rows]
 *   k         0 <= k <= min(vocab, DS_LOGPROB_MAX_K)
 *   scale     finite, above 0
 *   logprob, entropy, lse  device float[rows]
 *   idx, top  device int32 / float [rows][k]; ignored when k is 0
 */
int ds_token_logprobs(const void *logits, int dtype, int64_t rows, int64_t vocab,
                      int64_t row_stride, const int32_t *tokens, int k, float scale,
                      float *logprob, float *entropy, float *lse, int32_t *idx, float *top,
                      void *stream);

/*
 * ds_token_logprobs_backward -- gradient by the logits of
 *     sum grad_logprob logprob + grad_entropy entropy + grad_lse lse
 *       + sum_j grad_top[.][j] top[.][j]
 * with lse, entropy and idx as the forward call gave them; a gradient that is
 * NULL is 0 (idx is needed with grad_top).  An idx outside [0, vocab) takes no
 * part, one that is listed twice counts twice.  Results are rounded to `dtype`
 * once; the order of sums is fixed.
 *   grad      device, row r at r * grad_stride; may be logits itself, with the
 *             same stride, and overlaps it in no other way
 */
int ds_token_logprobs_backward(const void *logits, int dtype, int64_t rows, int64_t vocab,
                               int64_t row_stride, const int32_t *tokens, int k,
                               const int32_t *idx, float scale, const float *lse,
                               const float *entropy, const float *grad_logprob,
                               const float *grad_entropy, const float *grad_lse,
                               const float *grad_top, void *grad, int64_t grad_stride,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DS_LOGPROB_H */
