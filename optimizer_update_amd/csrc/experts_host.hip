// experts_host.hip -- C ABI of the operators around experts (host side):
// argument checks and launch shapes.  The arithmetic is in route_kernels.hip
// and int4_kernels.hip.
#include <cmath>

#include "../../include/optimizer_experts.h"
#include "call.hpp"
#include "experts.h"
#include "int4_choice.hpp"

using namespace experts;

namespace {

int check_tokens(int64_t tokens, int32_t k)
{
    if (k < 1 || k > OU_ROUTE_MAX_CHOICES) return fail(OU_EINVAL, "k = %d is out of range", k);
    if (tokens < 0 || tokens > OU_ROUTE_MAX_SLOTS / k)
        return fail(OU_EINVAL, "%lld tokens with %d choices: 2^28 slots at most", static_cast<long long>(tokens), k);
    return OU_OK;
}

int check_experts(int32_t experts)
{
    if (experts < 1 || experts > OU_ROUTE_MAX_EXPERTS) return fail(OU_EINVAL, "experts = %d is out of range", experts);
    return OU_OK;
}

int check_stride(int64_t stride, int64_t cols, const char* what)
{
    if (stride < cols || stride > kMaxAxis) return fail(OU_EINVAL, "%s is out of range", what);
    return OU_OK;
}

int check_topk(int dtype, int64_t tokens, int32_t experts, int64_t row_stride, int scores, float scale, int32_t k)
{
    if (!valid_dtype(dtype)) return fail(OU_EINVAL, "unknown dtype %d", dtype);
    if (int st = check_experts(experts)) return st;
    if (int st = check_tokens(tokens, k)) return st;
    if (int st = check_stride(row_stride, experts, "row_stride")) return st;
    if (scores != OU_ROUTE_SOFTMAX && scores != OU_ROUTE_SIGMOID) return fail(OU_EINVAL, "unknown scores %d", scores);
    if (!std::isfinite(scale)) return fail(OU_EINVAL, "scale is not finite");
    if (k > experts) return fail(OU_EINVAL, "%d of %d experts", k, experts);
    return OU_OK;
}

// Where the rows of all slots are more than this, what is written leaves by
// non-temporal stores: it would only push others out of the 256 MiB last cache.
constexpr int64_t kKeptBytes = int64_t(192) << 20;

// Threads of a block that moves rows of `pieces`.
int row_threads(int64_t pieces)
{
    const int64_t t = cut(pieces, kWave) * kWave;
    return static_cast<int>(t < kWave ? kWave : t < kRowThreads ? t : kRowThreads);
}

double dense(int64_t rows, int64_t cols, int bytes) { return extent(rows, cols, cols, bytes); }

// Rows of the three kernels that move them.
struct Rows {
    int dtype;
    int64_t tokens, cols;
    int32_t k;
};

int check_rows(const Rows& r)
{
    if (!valid_dtype(r.dtype)) return fail(OU_EINVAL, "unknown dtype %d", r.dtype);
    if (int st = check_tokens(r.tokens, r.k)) return st;
    return check_axis(r.cols, "cols");
}

// 16-byte pieces of all rows: `p` and strides of up to four operands.
bool wide_cols(const Rows& r, const void* const* p, const int64_t* stride, int n)
{
    const int eb = elem_bytes(r.dtype);
    if (r.cols * eb % 16) return false;
    for (int i = 0; i < n; ++i)
        if (p[i] && !wide_rows(p[i], stride[i], 0, eb, 16)) return false;
    return true;
}

}  // namespace

extern "C" {

#define OU_EXPORT __attribute__((visibility("default")))

OU_EXPORT const char* ou_experts_last_error(void) { return g_error; }

OU_EXPORT int ou_route_topk(int dtype, const void* logits, int64_t tokens, int32_t experts, int64_t row_stride, int scores,
                            const float* bias, int32_t groups, int32_t top_groups, int group_score, int renormalize,
                            float scale, const uint8_t* mask, int32_t k, float* weights, int32_t* ids, void* stream)
{
    if (int st = check_topk(dtype, tokens, experts, row_stride, scores, scale, k)) return st;
    if (groups < 1 || groups > OU_ROUTE_MAX_GROUPS || experts % groups)
        return fail(OU_EINVAL, "%d groups of %d experts", groups, experts);
    if (top_groups < 1 || top_groups > groups) return fail(OU_EINVAL, "top_groups = %d is out of range", top_groups);
    if (group_score != OU_ROUTE_BEST && group_score != OU_ROUTE_BEST_TWO)
        return fail(OU_EINVAL, "unknown group_score %d", group_score);
    if (k > experts / groups * top_groups) return fail(OU_EINVAL, "%d of the %d experts of %d groups", k, experts / groups * top_groups, top_groups);
    if (tokens == 0) return OU_OK;
    const int eb = elem_bytes(dtype);
    const Buffer bufs[] = {{"logits", logits, extent(tokens, experts, row_stride, eb), static_cast<unsigned>(eb), false},
                           {"bias", bias, bias ? 4.0 * experts : 0, 4, false},
                           {"mask", mask, mask ? static_cast<double>(tokens) : 0, 1, false},
                           {"weights", weights, dense(tokens, k, 4), 4, true},
                           {"ids", ids, dense(tokens, k, 4), 4, true}};
    if (int st = check_buffers(bufs, 5)) return st;
    TopkArgs p{logits, bias, mask, weights, ids, tokens, row_stride, experts, k, groups, top_groups, scores,
               group_score == OU_ROUTE_BEST_TWO, renormalize != 0, scale, 0, 0, 0};
    p.wide = experts % 4 == 0 && wide_rows(logits, row_stride, 0, eb, 4 * eb);
    p.bias_wide = experts % 4 == 0 && wide_rows(bias, 0, 0, 4, 16);
    const TopkKernel f = topk_kernel(dtype, experts, k, groups);
    p.exact = f.tokens == 1 && k == kWave;   // no lane for the first one left out
    void* args[] = {&p};
    return launch({f.fn, cut(tokens, kTopkWaves * f.tokens), 1, kTopkWaves * kWave, "k_topk", 0}, args, stream);
}

OU_EXPORT int ou_route_topk_backward(int dtype, const void* logits, int64_t tokens, int32_t experts, int64_t row_stride,
                                     int scores, int renormalize, float scale, const int32_t* ids, const float* dweights,
                                     int32_t k, void* dlogits, void* stream)
{
    if (int st = check_topk(dtype, tokens, experts, row_stride, scores, scale, k)) return st;
    if (tokens == 0) return OU_OK;
    const int eb = elem_bytes(dtype);
    const Buffer bufs[] = {{"logits", logits, extent(tokens, experts, row_stride, eb), static_cast<unsigned>(eb), false},
                           {"ids", ids, dense(tokens, k, 4), 4, false},
                           {"dweights", dweights, dense(tokens, k, 4), 4, false},
                           {"dlogits", dlogits, dense(tokens, experts, eb), static_cast<unsigned>(eb), true}};
    if (int st = check_buffers(bufs, 4)) return st;
    TopkBackwardArgs p{logits, ids, dweights, dlogits, tokens, row_stride, experts, k, scores, renormalize != 0, scale, 0, 0};
    p.wide = experts % 4 == 0 && wide_rows(logits, row_stride, 0, eb, 4 * eb);
    p.dense_wide = experts % 4 == 0 && wide_rows(dlogits, experts, 0, eb, 4 * eb);
    const TopkKernel f = topk_backward_kernel(dtype, experts, k);
    void* args[] = {&p};
    return launch({f.fn, cut(tokens, kTopkWaves * f.tokens), 1, kTopkWaves * kWave, "k_topk_backward", 0}, args, stream);
}

}  // extern "C"

namespace {

// Slots of a block of the order, and blocks.
int64_t order_chunk(int64_t slots)
{
    if (slots <= kOrderAlone) return kOrderAlone;
    const int64_t most = cut(cut(slots, kOrderBlocks), kOrderThreads) * kOrderThreads;
    return most > kOrderChunk ? most : kOrderChunk;
}

int64_t order_blocks(int64_t slots) { return slots ? cut(slots, order_chunk(slots)) : 1; }

int32_t order_bins(int32_t experts) { return (experts + 4) / 4 * 4; }

}  // namespace

extern "C" {

OU_EXPORT int64_t ou_route_order_workspace_bytes(int64_t slots, int32_t experts)
{
    if (slots < 0 || slots > OU_ROUTE_MAX_SLOTS || check_experts(experts)) return -1;
    const int64_t blocks = order_blocks(slots);
    return blocks > 1 ? blocks * order_bins(experts) * 4 : 0;
}

OU_EXPORT int ou_route_order(const int32_t* ids, int64_t slots, int32_t experts, int32_t* offsets, int32_t* slot_of_row,
                             int32_t* row_of_slot, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (int st = check_experts(experts)) return st;
    if (slots < 0 || slots > OU_ROUTE_MAX_SLOTS) return fail(OU_EINVAL, "slots = %lld is out of range", (long long)slots);
    const int64_t need = ou_route_order_workspace_bytes(slots, experts);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(OU_EINVAL, "workspace: %lld bytes are needed", static_cast<long long>(need));
    const double sb = 4.0 * static_cast<double>(slots);
    const Buffer bufs[] = {{"ids", ids, sb, 4, false},
                           {"offsets", offsets, 4.0 * (experts + 1.0), 4, true},
                           {"slot_of_row", slot_of_row, sb, 4, true},
                           {"row_of_slot", row_of_slot, sb, 4, true},
                           {"workspace", workspace, static_cast<double>(need), 16, true}};
    if (int st = check_buffers(bufs, 5)) return st;
    OrderArgs p{ids, offsets, slot_of_row, row_of_slot, static_cast<int32_t*>(workspace), slots, order_chunk(slots), experts,
                static_cast<int32_t>(order_blocks(slots)), order_bins(experts)};
    void* args[] = {&p};
    if (p.blocks > 1)
        if (int st = launch({order_count_kernel(), p.blocks, 1, kOrderThreads, "k_order_count", 0}, args, stream)) return st;
    return launch({order_place_kernel(), p.blocks, 1, kOrderThreads, "k_order_place", 0}, args, stream);
}

OU_EXPORT int ou_route_dispatch(int dtype, const void* x, int64_t tokens, int64_t cols, int64_t x_stride, int32_t k,
                                const int32_t* slot_of_row, const int32_t* row_of_slot, void* out, int64_t out_stride,
                                int zero_rest, void* stream)
{
    const Rows r{dtype, tokens, cols, k};
    if (int st = check_rows(r)) return st;
    if (int st = check_stride(x_stride, cols, "x_stride")) return st;
    if (int st = check_stride(out_stride, cols, "out_stride")) return st;
    if (tokens == 0 || cols == 0) return OU_OK;
    const int eb = elem_bytes(dtype);
    const Buffer bufs[] = {{"x", x, extent(tokens, cols, x_stride, eb), static_cast<unsigned>(eb), false},
                           {"slot_of_row", slot_of_row, dense(tokens, k, 4), 4, false},
                           {"row_of_slot", row_of_slot, dense(tokens, k, 4), 4, false},
                           {"out", out, extent(tokens * k, cols, out_stride, eb), static_cast<unsigned>(eb), true}};
    if (int st = check_buffers(bufs, 4)) return st;
    RowsArgs p{};
    p.x = x;
    p.slot_of_row = slot_of_row;
    p.row_of_slot = row_of_slot;
    p.out = out;
    p.tokens = tokens;
    const void* const ptrs[] = {x, out};
    const int64_t strides[] = {x_stride, out_stride};
    const bool wide = wide_cols(r, ptrs, strides, 2);
    const int per = wide ? 16 / eb : 1;
    p.cols = cols / per;
    p.x_stride = x_stride / per;
    p.out_stride = out_stride / per;
    p.k = k;
    p.past_caches = tokens * k * cols * eb > kKeptBytes;
    p.zero_rest = zero_rest != 0;
    void* args[] = {&p};
    return launch({dispatch_kernel(eb, wide), tokens, 1, row_threads(p.cols), "k_dispatch", 0}, args, stream);
}

OU_EXPORT int ou_route_combine(int dtype, const void* y, int64_t tokens, int64_t cols, int64_t y_stride, int32_t k,
                               const float* weights, const int32_t* row_of_slot, const void* add, int64_t add_stride,
                               void* out, int64_t out_stride, void* stream)
{
    const Rows r{dtype, tokens, cols, k};
    if (int st = check_rows(r)) return st;
    if (int st = check_stride(y_stride, cols, "y_stride")) return st;
    if (int st = check_stride(out_stride, cols, "out_stride")) return st;
    if (add)
        if (int st = check_stride(add_stride, cols, "add_stride")) return st;
    if (tokens == 0 || cols == 0) return OU_OK;
    const int eb = elem_bytes(dtype);
    const unsigned ea = static_cast<unsigned>(eb);
    const Buffer bufs[] = {{"y", y, extent(tokens * k, cols, y_stride, eb), ea, false},
                           {"weights", weights, weights ? dense(tokens, k, 4) : 0, 4, false},
                           {"row_of_slot", row_of_slot, dense(tokens, k, 4), 4, false},
                           {"add", add, add ? extent(tokens, cols, add_stride, eb) : 0, ea, false},
                           {"out", out, extent(tokens, cols, out_stride, eb), ea, true}};
    if (int st = check_buffers(bufs, 5)) return st;
    RowsArgs p{};
    p.x = y;
    p.add = add;
    p.weights = weights;
    p.row_of_slot = row_of_slot;
    p.out = out;
    p.tokens = tokens;
    p.cols = cols;
    p.x_stride = y_stride;
    p.add_stride = add_stride;
    p.out_stride = out_stride;
    p.k = k;
    p.past_caches = tokens * k * cols * eb > kKeptBytes;
    const void* const ptrs[] = {y, add, out};
    const int64_t strides[] = {y_stride, add_stride, out_stride};
    void* args[] = {&p};
    const bool wide = wide_cols(r, ptrs, strides, 3);
    return launch({combine_kernel(dtype, wide), tokens, 1, row_threads(wide ? cols * eb / 16 : cols), "k_combine", 0}, args,
                  stream);
}

OU_EXPORT int ou_route_combine_backward(int dtype, const void* dout, int64_t tokens, int64_t cols, int64_t dout_stride,
                                        int32_t k, const void* y, int64_t y_stride, const float* weights,
                                        const int32_t* slot_of_row, const int32_t* row_of_slot, void* dy, float* dweights,
                                        void* stream)
{
    const Rows r{dtype, tokens, cols, k};
    if (int st = check_rows(r)) return st;
    if (int st = check_stride(dout_stride, cols, "dout_stride")) return st;
    if (!dy && !dweights) return fail(OU_EINVAL, "dy and dweights are null");
    if (dweights)
        if (int st = check_stride(y_stride, cols, "y_stride")) return st;
    if (tokens == 0 || (cols == 0 && !dweights)) return OU_OK;   // without columns the weights' gradient is 0
    const int eb = elem_bytes(dtype);
    const unsigned ea = static_cast<unsigned>(eb);
    const Buffer bufs[] = {{"dout", dout, extent(tokens, cols, dout_stride, eb), ea, false},
                           {"y", y, dweights ? extent(tokens * k, cols, y_stride, eb) : 0, ea, false},
                           {"weights", weights, dy ? dense(tokens, k, 4) : 0, 4, false},
                           {"slot_of_row", slot_of_row, dense(tokens, k, 4), 4, false},
                           {"row_of_slot", row_of_slot, dense(tokens, k, 4), 4, false},
                           {"dy", dy, dy ? dense(tokens * k, cols, eb) : 0, ea, true},
                           {"dweights", dweights, dweights ? dense(tokens, k, 4) : 0, 4, true}};
    if (int st = check_buffers(bufs, 7)) return st;
    RowsArgs p{};
    p.x = dout;
    p.y = y;
    p.weights = weights;
    p.slot_of_row = slot_of_row;
    p.row_of_slot = row_of_slot;
    p.out = dy;
    p.dweights = dweights;
    p.tokens = tokens;
    p.cols = cols;
    p.x_stride = dout_stride;
    p.y_stride = y_stride;
    p.out_stride = cols;
    p.k = k;
    p.past_caches = tokens * k * cols * eb > kKeptBytes;
    const void* const ptrs[] = {dout, dweights ? y : nullptr, dy};
    const int64_t strides[] = {dout_stride, y_stride, cols};
    void* args[] = {&p};
    const bool wide = wide_cols(r, ptrs, strides, 3);
    return launch({combine_backward_kernel(dtype, wide), tokens, 1, row_threads(wide ? cols * eb / 16 : cols),
                   "k_combine_backward", 0}, args, stream);
}

OU_EXPORT int ou_route_balance(const float* bias, const int32_t* offsets, int32_t experts, float rate, float* out,
                               void* stream)
{
    if (int st = check_experts(experts)) return st;
    if (!std::isfinite(rate)) return fail(OU_EINVAL, "rate is not finite");
    const Buffer bufs[] = {{"bias", bias, bias == out ? 0 : 4.0 * experts, 4, false},
                           {"offsets", offsets, 4.0 * (experts + 1.0), 4, false},
                           {"out", out, 4.0 * experts, 4, true}};
    if (int st = check_buffers(bufs, 3)) return st;
    void* args[] = {&bias, &offsets, &experts, &rate, &out};
    return launch({balance_kernel(), 1, 1, 256, "k_balance", 0}, args, stream);
}

}  // extern "C"

namespace {

constexpr int64_t kMaxDepth = int64_t(1) << 25;

// What the calls with 4-bit weights share: n rows (of each matrix), k columns.
int check_weights(int64_t n, int64_t k, int32_t group, int scale_dtype)
{
    if (!valid_dtype(scale_dtype)) return fail(OU_EINVAL, "unknown dtype %d of scales", scale_dtype);
    if (int st = check_axis(n, "n")) return st;
    if (k < 0 || k > kMaxDepth) return fail(OU_EINVAL, "k = %lld is out of range", static_cast<long long>(k));
    if (group < 32 || group % 32 || k % group)
        return fail(OU_EINVAL, "group = %d: a multiple of 32 that divides k", group);
    return OU_OK;
}

double code_bytes(double n, int64_t k) { return n * static_cast<double>(k) / 2; }
double scale_bytes(double n, int64_t k, int32_t group, int bytes) { return n * static_cast<double>(k / group) * bytes; }

// Where x is held: in about so many blocks, up to 16 tiles of 16 rows of weights a
// block.  2001 tiles, k = 1024: 10.5 us by runs of 4, 11.9 by 6, 16.6 by 2; 512
// rows, 64 experts, k = 2048: 80 by 8 or 16, 88 by 4.
constexpr int64_t kInt4Blocks = 640;

int int4_product(int dtype, Int4Args& p, void* stream)
{
    const bool grouped = p.offsets || p.experts;
    if (!valid_dtype(dtype) || !valid_dtype(p.out_dtype)) return fail(OU_EINVAL, "unknown dtype");
    if (int st = check_weights(p.n, p.k, p.group, p.scale_dtype)) return st;
    if (int st = check_axis(p.m, "m")) return st;
    if (int st = check_stride(p.x_stride, p.k, "x_stride")) return st;
    if (int st = check_stride(p.out_stride, p.n, "out_stride")) return st;
    if (p.m == 0 || p.n == 0) return OU_OK;
    const int ex = elem_bytes(dtype), eo = elem_bytes(p.out_dtype), es = elem_bytes(p.scale_dtype);
    const double all = static_cast<double>(p.n) * (grouped ? p.experts : 1);
    const Buffer bufs[] = {{"x", p.x, extent(p.m, p.k, p.x_stride, ex), static_cast<unsigned>(ex), false},
                           {"codes", p.codes, code_bytes(all, p.k), 16, false},
                           {"scales", p.scales, scale_bytes(all, p.k, p.group, es), static_cast<unsigned>(es), false},
                           {"zeros", p.zeros, p.zeros ? scale_bytes(all, p.k, p.group, es) : 0, static_cast<unsigned>(es), false},
                           {"offsets", p.offsets, grouped ? 4.0 * (p.experts + 1.0) : 0, 4, false},
                           {"out", p.out, extent(p.m, p.n, p.out_stride, eo), static_cast<unsigned>(eo), true}};
    if (int st = check_buffers(bufs, 6)) return st;
    const int64_t tiles = int4_tiles(p.m, p.n, grouped, p.experts);
    const Int4Kernel f = int4_matmul_kernel(dtype, int4_scales(p.group), grouped, cut(p.k, 128), tiles, es == 2);
    // by groups: two more, the rows in front of the first and behind the last
    const int64_t units = grouped ? cut(p.m + 15 * static_cast<int64_t>(p.experts + 2), 16) : cut(p.m, 16);
    const int64_t run = cut(tiles, kInt4Blocks);
    p.tiles = static_cast<int32_t>(f.held ? cut(run > 16 ? 16 : run, f.width) : 1);
    void* args[] = {&p};
    return launch({f.fn, units * cut(cut(p.n, 16 * f.width), p.tiles), 1, kWave * f.waves, "k_int4_matmul", 0}, args, stream);
}

}  // namespace

extern "C" {

OU_EXPORT int ou_int4_quantize(int dtype, const void* x, int64_t rows, int64_t k, int64_t row_stride, int32_t group,
                               int scale_dtype, uint8_t* codes, void* scales, void* zeros, void* stream)
{
    if (!valid_dtype(dtype)) return fail(OU_EINVAL, "unknown dtype %d", dtype);
    if (int st = check_weights(rows, k, group, scale_dtype)) return st;
    if (int st = check_stride(row_stride, k, "row_stride")) return st;
    if (rows == 0 || k == 0) return OU_OK;
    const int eb = elem_bytes(dtype), es = elem_bytes(scale_dtype);
    const double n = static_cast<double>(rows);
    const Buffer bufs[] = {{"x", x, extent(rows, k, row_stride, eb), static_cast<unsigned>(eb), false},
                           {"codes", codes, code_bytes(n, k), 16, true},
                           {"scales", scales, scale_bytes(n, k, group, es), static_cast<unsigned>(es), true},
                           {"zeros", zeros, zeros ? scale_bytes(n, k, group, es) : 0, static_cast<unsigned>(es), true}};
    if (int st = check_buffers(bufs, 4)) return st;
    Int4QuantArgs q{x, codes, scales, zeros, rows, k, row_stride, group, scale_dtype, 0, 0};
    q.wide = wide_rows(x, row_stride, 0, eb, 16);
    q.lanes_log2 = group / 8 % 16 == 0 ? 4 : group / 8 % 8 == 0 ? 3 : 2;
    void* args[] = {&q};
    return launch({int4_quantize_kernel(dtype), cut(rows * (k / group), kInt4Threads >> q.lanes_log2), 1, kInt4Threads,
                   "k_int4_quantize", 0}, args, stream);
}

OU_EXPORT int ou_int4_dequantize(int dtype, const uint8_t* codes, int scale_dtype, const void* scales, const void* zeros,
                                 int64_t n, int64_t k, int32_t group, void* out, int64_t out_stride, void* stream)
{
    if (!valid_dtype(dtype)) return fail(OU_EINVAL, "unknown dtype %d", dtype);
    if (int st = check_weights(n, k, group, scale_dtype)) return st;
    if (int st = check_stride(out_stride, k, "out_stride")) return st;
    if (n == 0 || k == 0) return OU_OK;
    const int eb = elem_bytes(dtype), es = elem_bytes(scale_dtype);
    const double rows = static_cast<double>(n);
    const Buffer bufs[] = {{"codes", codes, code_bytes(rows, k), 16, false},
                           {"scales", scales, scale_bytes(rows, k, group, es), static_cast<unsigned>(es), false},
                           {"zeros", zeros, zeros ? scale_bytes(rows, k, group, es) : 0, static_cast<unsigned>(es), false},
                           {"out", out, extent(n, k, out_stride, eb), static_cast<unsigned>(eb), true}};
    if (int st = check_buffers(bufs, 4)) return st;
    Int4Args p{};
    p.codes = codes;
    p.scales = scales;
    p.zeros = zeros;
    p.out = out;
    p.n = n;
    p.k = k;
    p.out_stride = out_stride;
    p.group = group;
    p.scale_dtype = scale_dtype;
    p.out_wide = wide_rows(out, out_stride, 0, eb, 16);
    void* args[] = {&p};
    return launch({int4_dequantize_kernel(dtype), cut(n * (k / 8), kInt4Threads), 1, kInt4Threads, "k_int4_dequantize", 0}, args,
                  stream);
}

OU_EXPORT int ou_int4_matmul(int dtype, const void* x, int64_t m, int64_t x_stride, int out_dtype, const uint8_t* codes,
                             int scale_dtype, const void* scales, const void* zeros, int64_t n, int64_t k, int32_t group,
                             void* out, int64_t out_stride, void* stream)
{
    Int4Args p{x, codes, scales, zeros, out, nullptr, m, n, k, x_stride, out_stride, group, 0, 0, out_dtype, scale_dtype, 0, 1};
    return int4_product(dtype, p, stream);
}

OU_EXPORT int ou_int4_grouped_matmul(int dtype, const void* x, int64_t m, int64_t x_stride, int out_dtype,
                                     const uint8_t* codes, int scale_dtype, const void* scales, const void* zeros, int64_t n,
                                     int64_t k, int32_t group, const int32_t* offsets, int32_t experts, void* out,
                                     int64_t out_stride, int zero_rest, void* stream)
{
    if (int st = check_groups(offsets, experts, m)) return st;
    Int4Args p{x, codes, scales, zeros, out, offsets, m, n, k, x_stride, out_stride, group, experts, zero_rest != 0, out_dtype,
               scale_dtype, 0, 1};
    return int4_product(dtype, p, stream);
}

}  // extern "C"
