/*
 * wc_logprob.h — C ABI of libwc, what a step makes of its logits: the log
 * probabilities of given tokens, every row's entropy and its top alternatives.
 *
 *   lse        = log sum_i exp x[i]
 *   logprob    = x[token] - lse
 *   entropy    = - sum_i p[i] log p[i],  p[i] = exp(x[i] - lse)   (p = 0: no term)
 *   top        the `top` largest x, largest first, ties to the lower index, with
 *              x - lse.  Logits of -inf are no alternatives: a row with fewer
 *              others gets id -1 and -inf in the places that remain.
 * A row of -inf alone gets logprob -inf and entropy 0.  A token outside 0 ..
 * vocab - 1 gets logprob NaN.  A row that holds a NaN or +inf gets NaN for
 * logprob, entropy and the alternatives' log probabilities; NaN comes before
 * every number among its alternatives.
 *
 * Exponentials and sums are fp32, in an order that the shape fixes: the same call
 * gives the same bits.
 *
 * Conventions as in wc.h.  d_logits is aligned to its elements (2 or 4 bytes),
 * d_tokens 8-byte, d_work 16-byte, the outputs 4-byte.
 */
#ifndef WC_LOGPROB_H
#define WC_LOGPROB_H

#include "wc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WC_LOGITS_BF16 0u
#define WC_LOGITS_F32 1u
#define WC_LOGPROB_MAX_TOP 32u

typedef struct wc_logprob_shape {
  uint64_t stride; /* elements from one row to the next, at least vocab, below 2^40 */
  uint32_t rows;   /* below 2^24, else WC_E_SIZE */
  uint32_t vocab;  /* 1 .. 2^31 - 1 */
  uint32_t kind;   /* WC_LOGITS_BF16 or WC_LOGITS_F32 */
  uint32_t top;    /* 0 .. WC_LOGPROB_MAX_TOP, else WC_E_UNSUPPORTED */
} wc_logprob_shape;

/* Device scratch of a call of that shape (0: none is needed, or the call refuses the
 * shape).  Host only; asks the current device for its size. */
size_t wc_token_logprobs_workspace_bytes(const wc_logprob_shape *shape);

/*
 * d_logits [rows][stride]; d_tokens int64 [rows]; d_logprobs and d_entropy fp32
 * [rows], d_top_ids int32 and d_top_logprobs fp32 [rows][top] (not used where top
 * is 0).
 */
int wc_token_logprobs(const wc_logprob_shape *shape, const void *d_logits, const int64_t *d_tokens,
                      float *d_logprobs, float *d_entropy, int32_t *d_top_ids, float *d_top_logprobs,
                      void *d_work, size_t work_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* WC_LOGPROB_H */
