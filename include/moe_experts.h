/* The experts of a routed layer in 16 bits, forward and backward, over the
 * route-sort metadata, for MI355X (gfx950): products grouped by expert, the gated
 * activation between two of them, and the mix of the experts' outputs.
 *
 * Throughout, r is a row of the sorted metadata (r < *num_post_pad), s =
 * sorted_ids[r] its slot, t = s / k the slot's token and e = expert_of_block[r /
 * block] its expert.  A row whose s lies outside [0, M*k) is a padding row.  Sums
 * are held in FP32 and rounded once to the type of the output, to nearest even.
 * dtype is MRS_DTYPE_BF16 or MRS_DTYPE_F16 (moe_mxfp4.h); an output type is that
 * one or MRS_DTYPE_F32.
 *
 * Every call is asynchronous on `stream`, allocates nothing, reads num_post_pad on
 * the device, and returns MRS_OK or a negative MRS_ERR_* code before any launch.
 * Sizes that would take 2^32 threads or more in a launch are MRS_ERR_OVERFLOW.  None of
 * a product are with R * ceil(J / 256) below 2^27, for R = max_rows and J columns of y or
 * dx, and none of the weights' gradient with E * ceil(N / 128) * ceil(K / 128) below
 * 2^22; the other calls state theirs.
 * Matrices are row-major and contiguous; every pointer is aligned to its element
 * size (products of matrices at multiples of 16 bytes whose rows are as well take a
 * faster path).
 */
#ifndef MOE_EXPERTS_H_
#define MOE_EXPERTS_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_grouped_gemm -- y[r, n] = sum_c x[row(r), c] * w[e, n, c]; zeros in padding rows.
 *
 *   x         rows of K columns: M of them, row(r) = t (MRS_X_TOKENS), or
 *             moe_route_sort_max_rows(M, E, k, block), row(r) = r (MRS_X_SORTED)
 *   w         [E, N, K]
 *   sorted_ids, expert_of_block, num_post_pad
 *             metadata of moe_route_sort or moe_sort_from_ids for the same M, E, k
 *             and block
 *   K, N      1 .. 2^20
 *   block     block >= 16 and block % 16 == 0
 *   y         [moe_route_sort_max_rows(M, E, k, block), N] (rows below
 *             *num_post_pad are written, nothing else is)
 * Rows of a block whose expert id lies outside [0, E) are not written.  What a
 * padding row of x holds is not used.  One launch.
 */
int moe_grouped_gemm(const void* x, const void* w, int dtype, const int32_t* sorted_ids,
                     const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K, int N,
                     int block, int x_rows, int y_dtype, void* y, void* stream);

/*
 * moe_grouped_gemm_dx -- the gradient of moe_grouped_gemm's x, in sorted rows:
 * dx[r, c] = sum_n dy[r, n] * w[e, n, c]; zeros in padding rows.
 *
 *   dy        [max_rows, N] (what padding rows hold is not used)
 *   dx        [max_rows, K] (rows below *num_post_pad are written)
 * A token's gradient is the sum of its slots' rows (moe_combine without weights).
 */
int moe_grouped_gemm_dx(const void* dy, const void* w, int dtype, const int32_t* sorted_ids,
                        const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K, int N,
                        int block, int dx_dtype, void* dx, void* stream);

/* The two products above by tiles of `tile` rows (16, 32, 64 or 128, dividing block; 0
 * for the choice by sizes), the first three of them also with fewer columns (or'ed with
 * MRS_TILE_NARROW), for tests and tuning: the same results. */
enum { MRS_TILE_NARROW = 1 << 16 };
int moe_grouped_gemm_ex(const void* x, const void* w, int dtype, const int32_t* sorted_ids,
                        const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K, int N,
                        int block, int x_rows, int y_dtype, void* y, void* stream, int tile);
int moe_grouped_gemm_dx_ex(const void* dy, const void* w, int dtype, const int32_t* sorted_ids,
                           const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K,
                           int N, int block, int dx_dtype, void* dx, void* stream, int tile);

/*
 * moe_grouped_gemm_dw -- the gradient of moe_grouped_gemm's w:
 * dw[e, n, c] = sum of dy[r, n] * x[row(r), c] over e's rows that are no padding
 * rows; zeros for an expert without any.  expert_of_block has to be ascending
 * below *num_post_pad / block, as the metadata calls write it.
 *
 *   dw        [E, N, K] (written whole)
 * The order of the sums is fixed: equal inputs give equal bits.
 */
int moe_grouped_gemm_dw(const void* dy, const void* x, int dtype, const int32_t* sorted_ids,
                        const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K, int N,
                        int block, int x_rows, int dw_dtype, void* dw, void* stream);

/*
 * moe_swiglu -- h[r, i] = g * sigmoid(g) * u with g = a[r, i], u = a[r, I + i].
 *
 *   a         [rows, 2 I]
 *   num_post_pad  NULL (every row), or the rows to take: r < min(rows, *num_post_pad)
 *   rows      0 .. 2^31 - 1, rows * ceil(I / 8) at most 2^31;  I  1 .. 262144
 *   h         [rows, I], of a's type (other rows are left as they were)
 */
int moe_swiglu(const void* a, int dtype, const int32_t* num_post_pad, int64_t rows, int I, void* h, void* stream);

/* moe_swiglu_backward -- da of dh [rows, I]: da[r, i] = dh u sigmoid(g) (1 + g (1 -
 * sigmoid(g))), da[r, I + i] = dh g sigmoid(g).  da may be a itself. */
int moe_swiglu_backward(const void* a, const void* dh, int dtype, const int32_t* num_post_pad, int64_t rows, int I,
                        void* da, void* stream);

/*
 * moe_slot_rows -- rows[s] = the row r < *num_post_pad with sorted_ids[r] = s, -1
 * for a slot that has none (a dropped route).  One or two launches, by the sizes.
 *   sorted_ids  `capacity` entries;  rows  [M, k] int32 (written whole)
 *   capacity and M * k at most 2^31 - 257, k 1 .. 64
 */
int moe_slot_rows(const int32_t* sorted_ids, const int32_t* num_post_pad, int64_t capacity, int M, int k,
                  int32_t* rows, void* stream);

/*
 * moe_combine -- out[t, n] = sum_j weights[t, j] * y[rows[t, j], n]; a slot whose
 * row lies outside [0, capacity) adds nothing.
 *
 *   y         [capacity, N]
 *   rows      [M, k] int32, or NULL: rows[t, j] = t k + j (y in slot order)
 *   weights   [M, k] FP32, or NULL for ones
 *   N         1 .. 2^20;  k  1 .. 64;  capacity and M * k below 2^31;
 *             M * ceil(N / 512) at most 2^26 - 4
 *   out       [M, N] of y's type or FP32
 */
int moe_combine(const void* y, int dtype, const int32_t* rows, const float* weights, int64_t capacity, int M, int k,
                int N, int out_dtype, void* out, void* stream);

/*
 * moe_combine_backward -- dy[r] = weights[s] * dout[t], zeros in padding rows, and
 * dweights[t, j] = sum_n dout[t, n] * y[rows[t, j], n] (0 for a slot without a row).
 *
 *   dout      [M, N] of y's type
 *   rows      moe_slot_rows of this metadata; a row named twice is undefined
 *   sorted_ids, num_post_pad  the metadata, `capacity` rows
 *   weights   [M, k] FP32 or NULL for ones
 *   y, dweights  both given, or both NULL (no gradient of the weights is wanted); not
 *             looked at where M is 0
 *   dy        [capacity, N] (rows below *num_post_pad are written)
 *   N, k      as for moe_combine;  M * k + capacity / 64 at most 2^26 - 12
 */
int moe_combine_backward(const void* dout, const void* y, int dtype, const int32_t* rows, const int32_t* sorted_ids,
                         const int32_t* num_post_pad, const float* weights, int64_t capacity, int M, int k, int N,
                         void* dy, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H_ */
