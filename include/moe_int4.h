/* 4-bit weights with group scales and the matrix-vector products of routed tokens
 * that read them, for MI355X (gfx950): few tokens, straight from the router's ids.
 *
 * Format ("int4 rows").  A row of K weights is padded with zeros to Kp = ceil(K /
 * 128) * 128 columns and cut into groups of `group` (32, 64 or 128) columns.
 *
 *   weight = scale * (code - 8),  code 0 .. 15, scale of the group in BF16 or FP16
 *
 * codes are packed two to a byte, the even column in the low half:
 * codes [rows, Kp / 2], scales [rows, Kp / group], both row-major and contiguous.
 */
#ifndef MOE_INT4_H_
#define MOE_INT4_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_int4_quantize -- rows of FP32, BF16 or FP16 weights to int4 rows.
 *
 * With a a group's largest magnitude, scale = FP32 quotient a / 7 rounded to the
 * scales' type; code = 8 + the FP32 quotient w / scale rounded to the nearest
 * integer, ties to even, at most 7 in magnitude (code 8 where the scale is zero).
 * A group that holds an infinity or a NaN, or whose scale is no finite number,
 * gets the scale NaN and codes 8.
 *
 *   w           [rows, K], consecutive columns, row r at w + r * row_stride
 *               elements (row_stride >= K), aligned to its element size
 *   rows        >= 0, rows * Kp / 8 at most 2^38 (else MRS_ERR_OVERFLOW);  K  1 .. 262144;
 *               group  32, 64 or 128
 *   scale_dtype MRS_DTYPE_BF16 or MRS_DTYPE_F16
 *   codes       [rows, Kp / 2] (written), 4-byte aligned
 *   scales      [rows, Kp / group] (written), 2-byte aligned
 * Asynchronous on `stream`; one launch for up to 2^31 groups of eight columns, one
 * more for each further 2^31; allocates nothing.  Returns MRS_OK or a negative
 * MRS_ERR_* code before any launch.
 */
int moe_int4_quantize(const void* w, int dtype, int64_t rows, int K, int64_t row_stride, int group, int scale_dtype,
                      uint8_t* codes, void* scales, void* stream);

/* What a product's results become. */
enum {
  MRS_INT4_PLAIN = 0, /* y [M, k, N]: the products                                  */
  MRS_INT4_GATED = 1, /* y [M, k, N / 2]: g sigmoid(g) u of columns i and N / 2 + i */
  MRS_INT4_SUM = 2    /* y [M, N]: sum over the picks, times weights[t, j]          */
};

/*
 * moe_int4_matvec -- for every token t and pick j with e = ids[t, j],
 *
 *     p[t, j, n] = sum_c x[t or (t, j), c] * w[e, n, c]
 *
 * and y as the mode says; a pick whose e lies outside [0, E) has p = 0 (and y = 0).
 * Sums and the mode's arithmetic are held in FP32 and rounded once to y's type.
 * The weights' bytes bound it: each pick reads its expert's matrix, so tokens that
 * share experts read them again.  The grouped products, which read an expert once for
 * many tokens, take 16-bit (moe_experts.h) or 4-bit microscaled weights
 * (moe_mxfp4.h), not these.
 *
 *   x         [M, K] (per_slot 0) or [M, k, K] (per_slot 1), dtype MRS_DTYPE_BF16 or
 *             MRS_DTYPE_F16, 2-byte aligned; |x| below 2^96 (an infinity or a NaN
 *             makes the results that it takes part in NaN)
 *   codes     int4 rows [E, N] of K columns, 16-byte aligned; scales of x's dtype
 *   ids       [M, k] int32
 *   weights   [M, k] FP32 (MRS_INT4_SUM only, else NULL; not looked at where M is 0)
 *   M         >= 0;  k  1 .. 64;  E  1 .. 4096;  K  1 .. 262144, any with the codes' Kp
 *   N         1 .. 2^20, even for MRS_INT4_GATED; N * Kp / 2 below 2^31 bytes and
 *             M * k * ceil(N / 32) below 2^24 (else MRS_ERR_OVERFLOW)
 *   y         of x's dtype, 2-byte aligned
 * Asynchronous on `stream`; one launch; allocates nothing.  Returns MRS_OK or a
 * negative MRS_ERR_* code before any launch.
 */
int moe_int4_matvec(const void* x, int dtype, const uint8_t* codes, const void* scales, const int32_t* ids,
                    const float* weights, int M, int k, int E, int K, int N, int group, int per_slot, int mode,
                    void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT4_H_ */
