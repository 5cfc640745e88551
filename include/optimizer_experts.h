/*
 * optimizer_experts.h -- C ABI of the operators around experts of the MI355X
 * (gfx950) optimizer library: routing (scores, groups, top-k, weights and
 * their gradients), the order of rows by expert, the dispatch of rows to
 * experts and their weighted combination, the balance bias, and products
 * with 4-bit whole-number weights that carry group scales, plain and by
 * expert.
 *
 * It stands next to optimizer_update.h and optimizer_mx4.h (statuses and
 * dtypes are those of the former; the offsets of rows by expert are those of
 * the latter's products by groups) and keeps their manner: plain pointers and
 * sizes, the caller owns every buffer, nothing is allocated, arguments are
 * checked before anything is launched, on an error nothing is launched or
 * written, calls enqueue on `stream` (hipStream_t, NULL = the default stream)
 * and return without synchronising, and all of them may be captured into a
 * graph.  Sizes that pass what one launch can hold are OU_EINVAL.  No result
 * depends on the order in which blocks run.
 * The library is liboptimizer_experts.so.
 */
#ifndef OPTIMIZER_EXPERTS_H
#define OPTIMIZER_EXPERTS_H

#include <stdint.h>

#include "optimizer_update.h"

#ifdef __cplusplus
extern "C" {
#endif

enum ou_route_scores { OU_ROUTE_SOFTMAX = 0, OU_ROUTE_SIGMOID = 1 };
enum ou_route_group_score { OU_ROUTE_BEST = 0, OU_ROUTE_BEST_TWO = 1 };

/* Limits: experts, choices a token, groups of experts, and slots (tokens
 * times choices). */
#define OU_ROUTE_MAX_EXPERTS 1024
#define OU_ROUTE_MAX_CHOICES 64
#define OU_ROUTE_MAX_GROUPS 64
#define OU_ROUTE_MAX_SLOTS (1 << 28)

/* Chooses k experts for each token.  logits: tokens x experts of `dtype`,
 * rows row_stride elements apart.  With x a token's logits,
 *   score   s_e = exp(x_e) / sum_i exp(x_i)   or   1 / (1 + exp(-x_e))
 *   choice  c_e = s_e + bias_e (bias NULL: s_e)
 * An expert whose logit is -inf is absent: it is not chosen and has no score.
 * The experts are `groups` equal parts; a part counts by its largest c, or by
 * the sum of its two largest (one, if it has one; -inf if it has none), and
 * the top_groups parts that count most stay.  ids (tokens x k) gets the k
 * largest c that stay, in falling order, -1 where there are no more.  Equal
 * ones go to the lower index, and a NaN counts as the largest.  c is compared
 * as 64-bit arithmetic has it; without a bias and without sums, where single
 * scores alone are compared, the logits decide.  weights (tokens x k) gets
 * scale * s_e, divided by the sum of the chosen s with renormalize != 0 (which
 * is well-defined where the scores themselves underflow), 0 where ids is -1.
 * With softmax scores, a NaN or +inf among a token's logits makes its weights
 * NaN; its ids are k different experts all the same.
 * mask (NULL, or one byte a token): a token whose byte is 0 chooses nothing
 * (ids -1, weights 0). */
int ou_route_topk(int dtype, const void* logits, int64_t tokens, int32_t experts,
                  int64_t row_stride, int scores, const float* bias, int32_t groups,
                  int32_t top_groups, int group_score, int renormalize, float scale,
                  const uint8_t* mask, int32_t k, float* weights, int32_t* ids, void* stream);

/* The gradient of the logits (tokens x experts of `dtype`, dense rows) from
 * that of the weights (tokens x k, dense): ids are those that ou_route_topk
 * gave for the same logits and arguments, and constants.  With g the
 * weights' gradient, w the weights and r = w / scale:
 *   renormalised     d_j = w_j (g_j - sum_i g_i r_i) for the chosen, times
 *                    (1 - s_j) for sigmoid scores; 0 elsewhere
 *   softmax scores   d_e = scale s_e (g_e [e is chosen] - sum_i g_i s_i)
 *   sigmoid scores   d_j = scale s_j (1 - s_j) g_j for the chosen
 * Rows without a choice get 0. */
int ou_route_topk_backward(int dtype, const void* logits, int64_t tokens, int32_t experts,
                           int64_t row_stride, int scores, int renormalize, float scale,
                           const int32_t* ids, const float* dweights, int32_t k, void* dlogits,
                           void* stream);

/* The order of rows by expert.  Slot i of `slots` has expert ids[i]; an id
 * outside [0, experts) is of none.  Sorted by expert, stable:
 *   offsets (experts + 1): expert e has rows [offsets[e], offsets[e + 1])
 *   slot_of_row (slots): the slot of each row, -1 from offsets[experts] on
 *   row_of_slot (slots): the row of each slot, -1 for those of no expert
 * `workspace`: device memory of ou_route_order_workspace_bytes(slots,
 * experts) bytes, 16-byte aligned (NULL if that is 0); calls that may overlap
 * in time need workspaces of their own. */
int64_t ou_route_order_workspace_bytes(int64_t slots, int32_t experts);
int ou_route_order(const int32_t* ids, int64_t slots, int32_t experts, int32_t* offsets,
                   int32_t* slot_of_row, int32_t* row_of_slot, void* workspace,
                   int64_t workspace_bytes, void* stream);

/* out (tokens * k rows of cols elements): row row_of_slot[t * k + j] becomes
 * row t of x; rows whose slot_of_row is -1 become 0 with zero_rest != 0 and
 * are left as they were without.  Rows are x_stride and out_stride elements
 * apart; the values are copied as they are. */
int ou_route_dispatch(int dtype, const void* x, int64_t tokens, int64_t cols, int64_t x_stride,
                      int32_t k, const int32_t* slot_of_row, const int32_t* row_of_slot, void* out,
                      int64_t out_stride, int zero_rest, void* stream);

/* out[t] = add[t] + sum_j weights[t, j] * y[row_of_slot[t * k + j]], over the
 * slots whose row is not -1, in binary32 and rounded once.  weights NULL: 1
 * (the gradient of ou_route_dispatch); add NULL: 0.  y: tokens * k rows. */
int ou_route_combine(int dtype, const void* y, int64_t tokens, int64_t cols, int64_t y_stride,
                     int32_t k, const float* weights, const int32_t* row_of_slot, const void* add,
                     int64_t add_stride, void* out, int64_t out_stride, void* stream);

/* Its gradients: dy[row of slot] = weights[slot] * dout[t] (0 in the rows of
 * no slot) and dweights[slot] = the sum over the columns of dout[t] times
 * y[row of slot] (0 where the slot has no row).  Either may be NULL (then y,
 * or weights, may be too), not both.  dy: tokens * k dense rows. */
int ou_route_combine_backward(int dtype, const void* dout, int64_t tokens, int64_t cols,
                              int64_t dout_stride, int32_t k, const void* y, int64_t y_stride,
                              const float* weights, const int32_t* slot_of_row,
                              const int32_t* row_of_slot, void* dy, float* dweights, void* stream);

/* out_e = bias_e + rate * sign(mean - rows of e), mean the rows of all
 * experts over their number (compared in whole numbers).  out may be bias. */
int ou_route_balance(const float* bias, const int32_t* offsets, int32_t experts, float rate,
                     float* out, void* stream);

/* 4-bit weights: n rows of k columns, value = (code - zero) * scale.  codes:
 * rows of k / 2 bytes, the even column in the low four bits, 16-byte
 * aligned; scales and zeros: rows of k / group values of scale_dtype, zeros
 * NULL standing for 8.  group is a multiple of 32, k one of group.
 *
 * ou_int4_quantize: x (rows x k of `dtype`) by groups: with zeros, the
 * smallest scale whose 16 steps hold the group's values and 0, and a whole
 * zero; without, the smallest that holds them around code 8; scales are
 * rounded to scale_dtype first, codes to nearest (ties to even) then.  A group
 * of zeros has scale 0.  Non-finite values are not supported: their groups
 * hold unspecified codes. */
int ou_int4_quantize(int dtype, const void* x, int64_t rows, int64_t k, int64_t row_stride,
                     int32_t group, int scale_dtype, uint8_t* codes, void* scales, void* zeros,
                     void* stream);

/* out (n x k of `dtype`, rows out_stride apart) = the values, computed in
 * binary32, rounded once. */
int ou_int4_dequantize(int dtype, const uint8_t* codes, int scale_dtype, const void* scales,
                       const void* zeros, int64_t n, int64_t k, int32_t group, void* out,
                       int64_t out_stride, void* stream);

/* out[i][j] = sum_k x[i][k] * value[j][k]: x m x k of `dtype`, out m x n of
 * out_dtype.  A group's columns are summed in binary32, x (code - c) and x apart,
 * and (zero - c) times the second is subtracted, with c = 7.5 for a binary32 x and
 * 0 for 16 bits.  The products are exact; of a binary32 x what lies below 2^-133
 * is cut off, which shows where all of a row is below 1e-33 or so.  The sums pass
 * through |x| (|code - c| + |zero - c|) |scale|: a result's error goes by that,
 * which its own terms may be smaller than, and it may be infinite or NaN where
 * the sums pass what binary32 holds; rounded once.  A row of x that holds an
 * infinity or a NaN gives NaN or infinities, and no other row does by it.  Made
 * for few rows (tokens in serving): from some hundred on, dequantised weights and
 * a library product are faster. */
int ou_int4_matmul(int dtype, const void* x, int64_t m, int64_t x_stride, int out_dtype,
                   const uint8_t* codes, int scale_dtype, const void* scales, const void* zeros,
                   int64_t n, int64_t k, int32_t group, void* out, int64_t out_stride,
                   void* stream);

/* By groups of rows (experts): rows [offsets[e], offsets[e + 1]) of x meet
 * matrix e, codes, scales and zeros holding `experts` matrices one after the
 * other.  offsets: experts + 1 int32 in device memory, as in
 * ou_mx4_quantize_grouped (m at most 2^28).  Rows of no group become 0 with
 * zero_rest != 0 and are left as they were without. */
int ou_int4_grouped_matmul(int dtype, const void* x, int64_t m, int64_t x_stride, int out_dtype,
                           const uint8_t* codes, int scale_dtype, const void* scales,
                           const void* zeros, int64_t n, int64_t k, int32_t group,
                           const int32_t* offsets, int32_t experts, void* out, int64_t out_stride,
                           int zero_rest, void* stream);

/* Thread-local message of the last failure in this library. */
const char* ou_experts_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* OPTIMIZER_EXPERTS_H */
