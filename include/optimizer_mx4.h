/*
 * optimizer_mx4.h -- C ABI of the microscaled 4-bit operators of the MI355X
 * (gfx950) optimizer library: quantisation of weights, activations and
 * gradients to 4-bit floats with one power-of-two scale per 32 values, the
 * way back, products of quantised matrices, and products grouped by expert
 * over ragged row ranges.
 *
 * It stands next to optimizer_update.h (statuses and dtypes are those of
 * that header) and keeps its manner: plain pointers and sizes, the caller
 * owns every buffer, nothing is allocated, arguments are checked before
 * anything is launched, on an error nothing is launched or written, calls
 * enqueue on `stream` (hipStream_t, NULL = the default stream) and return
 * without synchronising, and all of them may be captured into a graph.
 * Sizes that pass what one launch can hold (some 2^30 rows or columns) are
 * OU_EINVAL.
 * The library is liboptimizer_mx4.so.
 *
 * Format.  A block is 32 neighbouring values along the contracted axis,
 * starting at a multiple of 32.  With e the biased binary32 exponent of the
 * block's largest magnitude (a subnormal number and zero have e = 0):
 *   scale code s = max(0, e - 2); 255 if the block holds a NaN or an infinity
 *   code of x    = the 4-bit float (sign, 2 exponent bits, 1 mantissa bit;
 *                  magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 as codes 0..7, sign
 *                  in bit 3) nearest to x / 2^(s - 127), ties to the even
 *                  code, magnitudes above 6 give 6; 0 where s = 255
 *   value        = magnitude(code) * 2^(s - 127); NaN where s = 255
 *
 * Held matrix of R rows and K columns.  codes: R rows of P / 2 bytes, the
 * even column in the low four bits; scales: R rows of P / 32 bytes;
 * P = ou_mx4_columns(K) = K rounded up to 128, what lies behind K being
 * zero codes (with the scale code of the block they are in, or 0).  codes
 * must be 16-byte aligned, scales 4-byte.  A batch of matrices is held one
 * after the other.
 */
#ifndef OPTIMIZER_MX4_H
#define OPTIMIZER_MX4_H

#include <stdint.h>

#include "optimizer_update.h"

#ifdef __cplusplus
extern "C" {
#endif

/* K rounded up to 128: the columns of a held matrix (-1 for K < 0). */
int64_t ou_mx4_columns(int64_t k);

/* Quantises x, `batch` matrices of rows x cols values of `dtype` (element
 * (b, r, c) at x[b * batch_stride + r * row_stride + c]; row_stride >= cols),
 * along its columns into codes/scales (a held matrix of `rows` rows) and
 * along its rows into codes_t/scales_t (x transposed: a held matrix of
 * `cols` rows and `rows` columns).  Either pair may be NULL, not both; with
 * both, x is read once. */
int ou_mx4_quantize(int dtype, const void* x, int64_t batch, int64_t rows, int64_t cols,
                    int64_t row_stride, int64_t batch_stride, uint8_t* codes, uint8_t* scales,
                    uint8_t* codes_t, uint8_t* scales_t, void* stream);

/* Columns of the transposed form by groups: an upper bound of the sum over
 * the groups of their rows rounded up to 128, ((rows + 127 groups) / 128)
 * * 128 (-1 for arguments below 0). */
int64_t ou_mx4_grouped_columns(int64_t rows, int32_t groups);

/* The same for one matrix whose rows fall into groups: group e is rows
 * [offsets[e], offsets[e + 1]) (rows at most 2^28 in the calls by groups),
 * offsets being groups + 1 int32 in device memory, rising, within [0, rows]
 * (others are clamped to that, and one below an earlier one counts as that
 * one: no row is of two groups).  Along the rows every group is a matrix of
 * its own: its columns of codes_t start at the sum of the earlier groups'
 * rows, each rounded up to 128, and its blocks at its first row.  A row of
 * codes_t holds ou_mx4_grouped_columns(rows, groups) columns; those behind the
 * last group are not written.  codes/scales (or NULL) get the rows of the
 * groups; rows of no group are not written. */
int ou_mx4_quantize_grouped(int dtype, const void* x, int64_t rows, int64_t cols, int64_t row_stride,
                            const int32_t* offsets, int32_t groups, uint8_t* codes, uint8_t* scales,
                            uint8_t* codes_t, uint8_t* scales_t, void* stream);

/* out (rows x cols of `dtype`, row_stride >= cols) = the values held,
 * rounded to nearest even where the type is coarser. */
int ou_mx4_dequantize(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                      int64_t cols, void* out, int64_t row_stride, void* stream);

/* out[i][j] = sum over k of a[i][k] * b[j][k]: a holds m rows, b n rows, of k
 * columns (k at most 2^25).  Sums in binary32 (where the terms'
 * magnitudes sum to more than it holds, a result may be infinite or NaN),
 * rounded once to out_dtype (nearest even).
 * `workspace` is caller-owned device memory of at least
 * ou_mx4_matmul_workspace_bytes(m, n, k, 0) bytes, 16-byte aligned (NULL if
 * that is 0, as it is where both matrices are held: what a workspace takes is
 * the 4-bit form of a left matrix given as values); calls that may overlap in
 * time need workspaces of their own. */
int64_t ou_mx4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k, int from_values);
int ou_mx4_matmul(int out_dtype, const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                  const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k, void* out,
                  int64_t out_stride, void* workspace, int64_t workspace_bytes, void* stream);

/* The same with the left matrix given as values (m x k of x_dtype, rows
 * x_stride elements apart), quantised along its columns on the way: bitwise
 * the result of ou_mx4_quantize and ou_mx4_matmul.  Workspace:
 * ou_mx4_matmul_workspace_bytes(m, n, k, 1). */
int ou_mx4_matmul_values(int x_dtype, const void* x, int64_t m, int64_t x_stride, int out_dtype,
                         const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                         void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes,
                         void* stream);

/* Rows of a by groups (offsets as in ou_mx4_quantize_grouped): row i of group
 * e meets matrix e of b, out[i][j] = sum_k a[i][k] * b[e][j][k], b holding
 * groups matrices of n rows.  Rows of no group become 0 with zero_rest != 0
 * and are left as they were without.  Workspace:
 * ou_mx4_grouped_workspace_bytes(rows, n, k, groups, 0 or 1). */
int64_t ou_mx4_grouped_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t groups,
                                       int from_values);
int ou_mx4_grouped_matmul(int out_dtype, const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows,
                          const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                          const int32_t* offsets, int32_t groups, void* out, int64_t out_stride,
                          int zero_rest, void* workspace, int64_t workspace_bytes, void* stream);
int ou_mx4_grouped_matmul_values(int x_dtype, const void* x, int64_t rows, int64_t x_stride,
                                 int out_dtype, const uint8_t* b_codes, const uint8_t* b_scales,
                                 int64_t n, int64_t k, const int32_t* offsets, int32_t groups,
                                 void* out, int64_t out_stride, int zero_rest, void* workspace,
                                 int64_t workspace_bytes, void* stream);

/* The contraction by groups: out[e][i][j] = sum over the rows r of group e
 * of a[r][i] * b[r][j], from the transposed forms that
 * ou_mx4_quantize_grouped made with the same rows, offsets and groups: a_t
 * holds m rows, b_t n rows.  out is groups matrices of m x n, one after the
 * other; an empty group's is 0.  At
 * most 2^25 columns are held. */
int ou_mx4_grouped_outer(int out_dtype, const uint8_t* a_codes_t, const uint8_t* a_scales_t, int64_t m,
                         const uint8_t* b_codes_t, const uint8_t* b_scales_t, int64_t n, int64_t rows,
                         const int32_t* offsets, int32_t groups, void* out, void* stream);

/* Thread-local message of the last failure in this library. */
const char* ou_mx4_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* OPTIMIZER_MX4_H */
