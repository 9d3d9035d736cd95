/*
 * wc_fp4.h — C ABI of libwc, the 4-bit tier: BF16 matrices as 4-bit codes
 * with one power-of-two scale per 32 columns, exact read-back of what the
 * codes stand for, and matrix-vector products on them.  Unlike the coding of
 * wc.h this one loses precision: it is for tensors that 12 bits per weight
 * leave too large (4.25 bits per weight here).
 *
 * Format of a matrix W[rows][cols] (a stack of matrices is rows on rows):
 *   groups           G = ceil(cols / 32) per row, the last one possibly short
 *   scales           u8 [rows][G]: e stands for the scale 2^(e - 127); 255
 *                    makes every value of the group NaN
 *   codes            u8 [rows][16 G]: column c in byte c / 2 of its row, the
 *                    low nibble when c is even; nibbles past cols are 0.
 *                    Bit 3 is the sign, bits 2..0 select
 *                    0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   value            +-magnitude * scale, as the BF16 of that value: exact
 *                    for every e <= 252, infinite where it passes BF16's range
 * Every row of codes starts at a 16-byte boundary when the array does.
 *
 * Conventions as in wc.h: caller-owned device memory, work enqueued on
 * `stream` in order without waiting, WC_OK or a negative WC_E_* code, nothing
 * enqueued when an argument check fails, no abort and no exception.
 * d_w, d_out and d_codes must be 16-byte aligned, d_x too when cols is a
 * multiple of 8 and 2-byte otherwise, d_y 4-byte; d_scales may have any
 * alignment.
 */
#ifndef WC_FP4_H
#define WC_FP4_H

#include "wc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WC_FP4_GROUP 32u
#define WC_FP4_GROUPS(cols) (((uint64_t)(cols) + 31u) / 32u)
#define WC_FP4_CODE_BYTES(rows, cols) ((uint64_t)(rows) * 16u * WC_FP4_GROUPS(cols))
#define WC_FP4_SCALE_BYTES(rows, cols) ((uint64_t)(rows) * WC_FP4_GROUPS(cols))
#define WC_FP4_MAX_COLS (1u << 24) /* columns of one row */

/*
 * Codes W.  A group's scale is the smallest 2^(e - 127), e >= 1, that keeps
 * every |w| of the group within 7 scales: 6 is the largest magnitude and 2 the
 * largest step, so no weight moves by more than half of the largest step.
 * Weights round to the nearest value, ties to the even code; a value past
 * BF16's range is not taken (the next smaller one is).  A group that holds an
 * infinity or a NaN gets e = 255 and zero codes.  rows or cols 0: nothing to do.
 */
int wc_fp4_encode(const uint16_t *d_w, uint64_t rows, uint64_t cols, uint8_t *d_codes,
                  uint8_t *d_scales, void *stream);

/* The BF16 values that codes and scales stand for, into d_out[rows][cols]. */
int wc_fp4_decode(const uint8_t *d_codes, const uint8_t *d_scales, uint64_t rows, uint64_t cols,
                  uint16_t *d_out, void *stream);

/*
 * y[b][r] = sum_c W[r][c] x[b][c], with W's values rebuilt in registers:
 * d_x BF16 [batch][cols], d_y fp32 [batch][rows].  Products are exact, sums
 * fp32 in a fixed order (the same call gives the same bits).  batch in
 * 1..WC_MAX_BATCH, else WC_E_UNSUPPORTED.
 */
int wc_fp4_gemv(const uint8_t *d_codes, const uint8_t *d_scales, uint64_t rows, uint64_t cols,
                const uint16_t *d_x, uint32_t batch, float *d_y, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* WC_FP4_H */
