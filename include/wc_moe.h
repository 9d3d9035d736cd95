/*
 * wc_moe.h — C ABI of libwc, a whole mixture-of-experts layer for a few
 * tokens (a decode batch): router, choice of the experts, their gated products
 * and the weighted sum, with the experts' matrices in BF16 or in the 4-bit
 * form of wc_fp4.h.
 *
 *   logit[t][e] = sum_h x[t][h] router[e][h]
 *   score       = softmax over e, or 1 / (1 + exp(-logit))
 *   choice      the top_k experts by logit, or by score + bias[e] when there
 *               is a bias; ties go to the lower e, a NaN comes before every
 *               number.  A bias of -inf takes the expert out: tokens with
 *               fewer than top_k experts left get id -1 and weight 0 in the
 *               places that remain.
 *   weight      score of the chosen experts; with WC_MOE_RENORM divided by
 *               their sum (all 0 where that sum is 0); times scale
 *   y[t]        = sum over the chosen e of weight *
 *                 down[e] (silu(gate[e] x[t]) * (up[e] x[t]))
 * silu(a) = a / (1 + exp(-a)).  A token with no expert at all gets y = 0.
 *
 * Sums, scores and score + bias are fp32.  So sigmoid scores of logits above
 * about 17 are all 1 (with a bias, such experts are chosen by bias and index),
 * and those of logits below about -88 are 0 (a token with no others gets y = 0,
 * with WC_MOE_RENORM too).
 * weight * silu(gate) * up goes into the second product as the sum of two BF16
 * numbers: 16 bits of it, of fp32's 24.  At 64 tokens and 8 experts of 1024 that
 * is 2.4e-6 of y's norm before y's rounding (fp32 activations: 3.9e-7), and
 * y, rounded to BF16 once at the end, differs by one step in 0.3% of its
 * numbers; where the sum cancels, what is left is off by up to 2^-16 of its
 * terms.  The sums' order is fixed by the shape and the choice: the same call
 * gives the same bits.
 *
 * Conventions as in wc.h.  d_router, the weights' d_data and d_work are 16-byte
 * aligned, d_x too when hidden is a multiple of 8 and 2-byte otherwise, d_y
 * 2-byte, d_bias, d_ids and d_weights 4-byte.
 */
#ifndef WC_MOE_H
#define WC_MOE_H

#include "wc_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WC_MOE_SOFTMAX 0u
#define WC_MOE_SIGMOID 1u
#define WC_MOE_RENORM 1u /* flags: weights of a token's experts sum to scale */

#define WC_MOE_BF16 0u /* kind of a stack of matrices: BF16 [experts][rows][cols] */
#define WC_MOE_FP4 1u  /* codes and scales of experts * rows rows (wc_fp4.h) */

#define WC_MOE_MAX_TOKENS 64u
#define WC_MOE_MAX_EXPERTS 512u
#define WC_MOE_MAX_TOP_K 16u
#define WC_MOE_MAX_DIM 65536u /* hidden and inter */

typedef struct wc_moe_shape {
  uint32_t tokens;  /* 1..WC_MOE_MAX_TOKENS, else WC_E_UNSUPPORTED */
  uint32_t hidden;  /* length of x and y rows, 1..WC_MOE_MAX_DIM */
  uint32_t inter;   /* rows of gate and of up, 1..WC_MOE_MAX_DIM */
  uint32_t experts; /* 1..WC_MOE_MAX_EXPERTS */
  uint32_t top_k;   /* 1..min(experts, WC_MOE_MAX_TOP_K) */
  uint32_t scoring; /* WC_MOE_SOFTMAX or WC_MOE_SIGMOID */
  uint32_t flags;   /* WC_MOE_RENORM or 0 */
  float scale;      /* factor of every weight */
} wc_moe_shape;

typedef struct wc_moe_experts {
  uint32_t kind;           /* WC_MOE_BF16 or WC_MOE_FP4 */
  const void *d_data;      /* BF16 values, or codes */
  const uint8_t *d_scales; /* WC_MOE_FP4: the scales; WC_MOE_BF16: ignored */
} wc_moe_experts;

/* Device scratch that a call with this shape needs; 0 for a shape that
 * wc_moe refuses.  Host only. */
size_t wc_moe_workspace_bytes(const wc_moe_shape *shape);

/*
 * d_x BF16 [tokens][hidden]; d_router BF16 [experts][hidden]; d_bias fp32
 * [experts] or NULL; gate_up: stack of [2 inter][hidden] (the gate's rows, then
 * the up rows); down: stack of [hidden][inter]; d_y BF16 [tokens][hidden];
 * d_ids int32 and d_weights fp32 [tokens][top_k], best first, either may be
 * NULL.  d_work: wc_moe_workspace_bytes(shape) bytes, contents ignored and
 * overwritten.
 */
int wc_moe(const wc_moe_shape *shape, const uint16_t *d_x, const uint16_t *d_router,
           const float *d_bias, const wc_moe_experts *gate_up, const wc_moe_experts *down,
           uint16_t *d_y, int32_t *d_ids, float *d_weights, void *d_work, size_t work_bytes,
           void *stream);

#ifdef __cplusplus
}
#endif
#endif /* WC_MOE_H */
