/* 4-bit microscaled rows and the grouped product over the route-sort metadata
 * that reads them, for MI355X (gfx950).
 *
 * Format ("4-bit rows").  A row of K values is padded with zeros to
 * Kp = ceil(K / 128) * 128 columns and cut into blocks of 32.  Block c of the
 * row holds one scale byte X and 32 four-bit codes:
 *
 *   value = (-1)^sign * level * 2^(X - 127),  X = 255: the whole block is NaN
 *   level of the low three bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 is the sign
 *
 * codes are packed two to a byte, the even column in the low half:
 * codes [rows, Kp / 2], scales [rows, Kp / 32], both row-major and contiguous.
 */
#ifndef MOE_MXFP4_H_
#define MOE_MXFP4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Types of values beside MRS_DTYPE_F32 and MRS_DTYPE_BF16 (moe_route_sort.h). */
enum { MRS_DTYPE_F16 = 2 };

/*
 * moe_mxfp4_quantize -- rows of FP32, BF16 or FP16 values to 4-bit rows.
 *
 * For each block with largest magnitude a: X = max(floor(log2 a) - 2 + 127, 0)
 * (0 for a block of zeros); each value divided by 2^(X - 127) is rounded to
 * the nearest level, ties to the even code, magnitudes above 6 to 6; the sign
 * is kept.  A block that holds an infinity or a NaN gets X = 255 and zero codes.
 *
 *   x           [rows, K], consecutive columns, row r at x + r * row_stride
 *               elements (row_stride >= K), aligned to its element size
 *   rows        >= 0
 *   K           1 <= K <= 262144
 *   codes       [rows, Kp / 2] (written), 4-byte aligned
 *   scales      [rows, Kp / 32] (written)
 *   values      NULL, or [rows, K] contiguous of x's type (written): the values
 *               that codes and scales stand for (all exact in x's type); NaN in
 *               a block with X = 255
 * Asynchronous on `stream`; one launch for up to 2^31 groups of eight columns
 * (rows * Kp / 8; none for rows == 0), one more for each further 2^31; allocates
 * nothing.  Returns MRS_OK or a negative MRS_ERR_* code before any launch;
 * MRS_ERR_OVERFLOW when rows * Kp / 8 exceeds 2^38.
 */
int moe_mxfp4_quantize(const void* x, int dtype, int64_t rows, int K, int64_t row_stride, uint8_t* codes,
                       uint8_t* scales, void* values, void* stream);

/* Which row of x a sorted row r with slot s = sorted_ids[r] reads. */
enum {
  MRS_X_TOKENS = 0, /* row s / k: x holds the tokens' rows (first product of the experts)         */
  MRS_X_SORTED = 1  /* row r: x holds rows in sorted order (a later product, on earlier results)  */
};

/*
 * moe_grouped_gemm_mxfp4 -- for every sorted row r < *num_post_pad with
 * s = sorted_ids[r] and e = expert_of_block[r / block],
 *
 *     y[r, n] = sum_k x[row(r), k] * w[e, n, k]    if 0 <= s < M*k
 *     y[r, n] = 0                                  otherwise (padding row)
 *
 * on 4-bit rows, accumulated in FP32 and rounded once to y's type.
 *
 *   x_codes, x_scales   4-bit rows of K columns: M of them (MRS_X_TOKENS) or
 *                       moe_route_sort_max_rows(M, E, k, block) (MRS_X_SORTED)
 *   w_codes, w_scales   4-bit rows [E, N] of K columns (expert e's output n)
 *   sorted_ids, expert_of_block, num_post_pad
 *                       metadata of moe_route_sort or moe_sort_from_ids for the
 *                       same M, E, k and block
 *   K                   padded columns, K > 0 and K % 128 == 0
 *   N                   >= 1
 *   block               block >= 16 and block % 16 == 0
 *   y_dtype             MRS_DTYPE_BF16 or MRS_DTYPE_F32
 *   y                   [moe_route_sort_max_rows(M, E, k, block), N] (rows below
 *                       *num_post_pad are written, nothing else is)
 * codes 16-byte aligned, scales, metadata and y 4-byte aligned.  A NaN block
 * reaches every result that it takes part in and no padding row.  Rows of a
 * block whose expert id lies outside [0, E) are not written.
 * Asynchronous on `stream`; one launch; allocates nothing; num_post_pad is read
 * on the device.  Returns MRS_OK or a negative MRS_ERR_* code before any launch;
 * MRS_ERR_OVERFLOW where the rows pass 32 bits, or the tiles of a launch 2^24
 * (16 to 128 rows x 256 columns: 2^28 rows or more of blocks of 16, N <= 256).
 */
int moe_grouped_gemm_mxfp4(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                           const uint8_t* w_scales, const int32_t* sorted_ids, const int32_t* expert_of_block,
                           const int32_t* num_post_pad, int M, int k, int E, int K, int N, int block, int x_rows,
                           int y_dtype, void* y, void* stream);

/* Kernels of the product, for tests and tuning; each computes the same rows of y
 * (sums in another order). */
enum {
  MRS_PRODUCT_BY_RULE = 0, /* as moe_grouped_gemm_mxfp4 chooses by the sizes   */
  MRS_PRODUCT_ROWS_16 = 1, /* tiles of 16 rows x 16 columns                    */
  MRS_PRODUCT_ROWS_32 = 2, /* tiles of 16 rows x 32 columns                    */
  MRS_PRODUCT_TILE_16 = 3, /* tiles of 16 rows x 256 columns, and so on; the   */
  MRS_PRODUCT_TILE_32 = 4, /* rows have to divide block                        */
  MRS_PRODUCT_TILE_64 = 5,
  MRS_PRODUCT_TILE_128 = 6
};

/* moe_grouped_gemm_mxfp4 by a kernel that the caller names
 * (MRS_ERR_INVALID_ARG where its rows do not divide block). */
int moe_grouped_gemm_mxfp4_ex(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                              const uint8_t* w_scales, const int32_t* sorted_ids, const int32_t* expert_of_block,
                              const int32_t* num_post_pad, int M, int k, int E, int K, int N, int block, int x_rows,
                              int y_dtype, void* y, void* stream, int kernel);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MXFP4_H_ */
