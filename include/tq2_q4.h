/*
 * tq2_q4.h -- C ABI of libtq2's 4-bit matrix-vector products with group scales.
 *
 *     out[m, n] = residual[m, n] + sum_g d[n, g] * sum_{k in group g} x[m, k] * (c[n, k] - 8)
 *
 * The projections a mixed-precision checkpoint keeps at 4 bits beside the
 * ternary ones of tq2.h.  The conventions of tq2.h hold: device pointers of the
 * caller, nothing allocated or synchronised, work only enqueued on `stream`,
 * negative tq2_status values for errors and nothing enqueued with them.
 *
 * Weight of [n, k]: two plain row-major arrays that need no conversion.
 *   codes   uint8 [n, k / 2]: weight 2j of a row in the low nibble of its byte
 *           j, weight 2j + 1 in the high nibble, each 0 .. 15;
 *   scales  binary16 [n, k / group]: d of each `group` consecutive weights.
 * The weight's value is (code - 8) * d.
 */
#ifndef TQ2_Q4_H
#define TQ2_Q4_H

#include "tq2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most rows of x that one call takes. */
#define TQ2_Q4_MAX_M 16

/* out[m, n] as above, for 1 <= m <= TQ2_Q4_MAX_M rows of x (the tokens of a
 * decode batch).
 * x: f32 [m, k] row-major; residual: f32 [m, n] or NULL; out: f32 [m, n], may
 * be the same pointer as residual and must overlap nothing else.
 * group: 32, 64 or 128; k a multiple of 128 (and at most 2^21).
 * codes: 16-byte aligned; scales: 16-byte aligned (rows of k / group
 * binary16), readable up to a multiple of 4 bytes: with an odd number of them
 * the two bytes after the last are loaded with it, whatever they hold; x,
 * residual, out: 16-byte aligned.
 * Accuracy: weights and scales exact, x split into two binary16 parts under a
 * power of two per row and 128 columns, f32 sums: within 1e-5 * (sum_k |x w| +
 * |residual|) + 2^-38 * sum_k X_k |w|, with X_k the largest |x| of k's 128
 * columns (128 j .. 128 j + 127).  The second term counts where a column far
 * above the others, by 2^16 and more, meets weights of almost zero.  Below 1e-33
 * there is 2^-151 * sum_k |w| besides, and the steps of subnormal results.  A row of x with a non-finite value gives non-finite or NaN
 * outputs for that row alone.
 * m == 0 or n == 0 is a no-op.  Errors: INVALID (null pointer, size out of
 * range, m > TQ2_Q4_MAX_M, another group), SHAPE (k not a multiple of 128),
 * ALIGN, ALIAS, DEVICE, LAUNCH. */
int tq2_q4_gemv(const void* codes, const void* scales, const float* x, const float* residual,
                float* out, int64_t m, int64_t n, int64_t k, int group, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ2_Q4_H */
