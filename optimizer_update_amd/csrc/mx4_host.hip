// mx4_host.hip -- C ABI of the microscaled 4-bit operators (host side):
// argument checks, launch shapes and workspaces.  The arithmetic is in
// mx4_kernels.hip.
#include "../../include/optimizer_mx4.h"
#include "call.hpp"
#include "mx4.h"

using namespace mx4;

namespace {

constexpr int64_t kMaxDepth = int64_t(1) << 25;   // contracted columns of a product

int64_t pad(int64_t k) { return (k + kPad - 1) / kPad * kPad; }

double held_codes(int64_t rows, int64_t pcols) { return static_cast<double>(rows) * static_cast<double>(pcols) / 2; }
double held_scales(int64_t rows, int64_t pcols) { return static_cast<double>(rows) * static_cast<double>(pcols) / kBlock; }

int64_t grouped_units(int64_t rows, int32_t groups, int64_t unit)
{
    return (rows + (unit - 1) * static_cast<int64_t>(groups)) / unit;
}

int launch_quantize(int dtype, QuantArgs& q, int64_t batch, int64_t units, void* stream)
{
    q.wide = wide_rows(q.x, q.row_stride, batch > 1 ? q.batch_stride : 0, elem_bytes(dtype), 16);
    if (!q.codes_t) {
        if (q.rows * (q.pcols / kPad) > UINT32_MAX / 2) return fail(OU_EINVAL, "x is too large");
        uint32_t n = static_cast<uint32_t>(q.rows * (q.pcols / kPad));
        void* args[] = {&q, &n};
        return launch({quant_rows_kernel(dtype), cut(n, (kQuantThreads / 16) * kQuantUnits), batch, kQuantThreads,
                       "k_quant_rows", 0}, args, stream);
    }
    void* args[] = {&q};
    return launch({quant_tile_kernel(dtype), units * (q.pcols / kQuantTile), batch, kQuantThreads, "k_quant_tile", 0},
                  args, stream);
}

// Which kernel makes a product: a tile of k_matmul_tile, or 0 and the columns of
// a block of k_matmul_few.
struct Choice {
    int tile, cols;
    bool values;   // the left matrix may come as values
    bool shared;   // the 64-tile's k-steps
};

// The rows in LDS (k_matmul_few) are quantised by every block again: that pays
// while they are few and short.  Rows times k-steps, measured with n = 4096,
// k = 4096 against a kernel of its own: 4 rows 6.9 us against 9.3, 8 rows 8.8
// against 9.4, 16 rows 12.3 against 10.1 (22 KiB hold them).
constexpr int64_t kValuesSteps = 320;

// rows: those of the left matrix, by groups their mean; room: the rows of a
// block, at most (by groups not known here: 16).
Choice choose(int64_t rows, int64_t n, int64_t steps, int64_t batch, int64_t room)
{
    if (rows <= 16) return {0, cut(n, 16) * batch <= 1024 ? 16 : 64, room * steps <= kValuesSteps, false};
    // a tile addresses its rows of a and b by 31 bits (kMaxDepth: 64 of them)
    if (steps >= (int64_t(1) << 17)) return {64, 0, false, true};
    const int64_t t64 = cut(rows, 64) * cut(n, 64) * batch;
    const int64_t t128 = cut(rows, 128) * cut(n, 128) * batch, t256 = cut(rows, 256) * cut(n, 256) * batch;
    // While they are at most two a CU, 64-tiles: 512 x 4096 x 1024 6.3 us, by
    // 128-tiles 6.7; 1024 x 2048 x 4096 13.7 against 15.0; but 1500 x 1500 x
    // 1500 (576 tiles) 10.9 against 10.3.  Two groups of waves share a long
    // chain of k-steps: k = 4096 10.1 us against 11.3 with one tile a CU and
    // 13.7 against 14.1 with two, k = 1024 5.3 against 5.1 and 7.4 against 6.3
    // (four groups: 10.4 and 18.3 us with k = 4096).  Rows of results that
    // are not 16-byte aligned and an odd number of k-steps cost every tile
    // about as much: 777 x 2063 x 4104 17.6 us, by 128-tiles 17.2; x 2064 x
    // 4096 13.0 against 14.1.
    if (t64 <= 512) return {64, 0, false, steps >= (t64 <= 256 ? 16 : 32)};
    // Rounds of the device, in tenths of a microsecond per pair of k-steps as
    // measured with 4096 columns: 256-tiles one a CU, 12 + 7 by how full the
    // round is (3000 x 3000 29.7 us, 4096 x 4096 37.3); 128-tiles two a CU,
    // 11.5, or 7.3 while they are one (35.0 and 44.1 us; 2048 x 4096 24.4 us,
    // by 256-tiles 29.9).
    const int64_t r256 = t256 % 256, r128 = t128 % 512;
    const int64_t by256 = t256 / 256 * 190 + (r256 ? 120 + 70 * r256 / 256 : 0);
    const int64_t by128 = t128 / 512 * 115 + (r128 > 256 ? 115 : r128 ? 73 : 0);
    if (by256 <= by128) return {256, 0, false, false};
    return {128, 0, false, false};
}

// By groups: the mean of the groups' rows decides, as the rows themselves are
// known on the device only.
Choice choose_grouped(int64_t rows, int64_t n, int64_t steps, int32_t groups)
{
    const int64_t g = groups > 0 ? groups : 1;
    return choose(cut(rows, g), n, steps, g < rows ? g : (rows > 0 ? rows : 1), rows < 16 ? rows : 16);
}

// Results beyond this leave by non-temporal stores: they would only push
// others out of the 256 MiB last cache.  256 MiB of them (16 x 4096 x 2048,
// 512 rows each) 112 us against 125, and the product behind it 67 against 81;
// 128 MiB (8192 x 8192, k = 4096) 148 against 135 us, where the next reader
// finds them in the cache otherwise.
constexpr int64_t kKeptBytes = int64_t(192) << 20;

// The launch of a product, and what goes by it in p.
Launch matmul_launch(int out_dtype, int grouping, const Choice& c, MatmulArgs& p, int64_t batch)
{
    const TileKernel t = c.tile ? matmul_tile_kernel(out_dtype, grouping, c.tile, c.shared) : TileKernel{};
    const FewKernel f = c.tile ? FewKernel{} : matmul_few_kernel(p.x ? p.x_dtype : kHeld, grouping, c.cols);
    const int rows = c.tile ? t.tile : 16, cols = c.tile ? t.tile : f.cols;
    // by rows: two groups more, the rows in front of the first and behind the last
    p.units = grouping == kByRows ? grouped_units(p.m, p.groups + 2, rows) : cut(p.m, rows);
    p.n_tiles = cut(p.n, cols);
    p.out_dtype = out_dtype;
    p.wide = wide_rows(p.out, p.out_stride, grouping == kByContraction ? p.m * p.out_stride : 0, elem_bytes(out_dtype),
                       c.tile ? 16 : 4 * elem_bytes(out_dtype));
    p.past_caches = p.m * (grouping == kByContraction ? p.groups : 1) * p.n * elem_bytes(out_dtype) > kKeptBytes;
    return {c.tile ? t.fn : f.fn, p.units * p.n_tiles, batch, c.tile ? t.threads : kWave * f.waves,
            "the product's kernel", c.tile ? 0 : few_lds(p.few_rows, p.steps, cols, f.waves)};
}

// x's 4-bit form at the start of a workspace.
int64_t values_bytes(int64_t m, int64_t k) { return m * (pad(k) / 2) + (m * (pad(k) / kBlock) + 15) / 16 * 16; }

}  // namespace

extern "C" {

#define OU_EXPORT __attribute__((visibility("default")))

OU_EXPORT const char* ou_mx4_last_error(void) { return g_error; }

OU_EXPORT int64_t ou_mx4_columns(int64_t k) { return k < 0 || k > kMaxAxis ? -1 : pad(k); }

OU_EXPORT int64_t ou_mx4_grouped_columns(int64_t rows, int32_t groups)
{
    return rows < 0 || rows > kMaxAxis || groups < 0 ? -1 : grouped_units(rows, groups, kPad) * kPad;
}

OU_EXPORT int ou_mx4_quantize(int dtype, const void* x, int64_t batch, int64_t rows, int64_t cols, int64_t row_stride,
                              int64_t batch_stride, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                              uint8_t* scales_t, void* stream)
{
    if (!valid_dtype(dtype)) return fail(OU_EINVAL, "unknown dtype %d", dtype);
    if (int st = check_axis(rows, "rows")) return st;
    if (int st = check_axis(cols, "cols")) return st;
    if (batch < 0 || batch > kMaxBatch) return fail(OU_EINVAL, "batch = %lld is out of range", (long long)batch);
    if (row_stride < cols || row_stride > kMaxAxis) return fail(OU_EINVAL, "row_stride is out of range");
    if (batch_stride < 0 || (batch > 1 && rows > 0 && batch_stride < cols)) return fail(OU_EINVAL, "batch_stride is out of range");
    if (batch == 0 || rows == 0 || cols == 0) return OU_OK;
    if (!codes != !scales || !codes_t != !scales_t || (!codes && !codes_t))
        return fail(OU_EINVAL, "codes and scales come in pairs, one pair at least");
    const int eb = elem_bytes(dtype);
    const double xb = extent(rows, cols, row_stride, eb) + static_cast<double>(batch - 1) * batch_stride * eb;
    const Buffer bufs[] = {{"x", x, xb, static_cast<unsigned>(eb), false},
                           {"codes", codes, codes ? held_codes(batch * rows, pad(cols)) : 0, 16, true},
                           {"scales", scales, scales ? held_scales(batch * rows, pad(cols)) : 0, 4, true},
                           {"codes_t", codes_t, codes_t ? held_codes(batch * cols, pad(rows)) : 0, 16, true},
                           {"scales_t", scales_t, scales_t ? held_scales(batch * cols, pad(rows)) : 0, 4, true}};
    if (int st = check_buffers(bufs, 5)) return st;
    QuantArgs q{x, codes, scales, codes_t, scales_t, rows, cols, row_stride, batch_stride, pad(cols), pad(rows), nullptr,
                0, 0};
    return launch_quantize(dtype, q, batch, pad(rows) / kQuantTile, stream);
}

OU_EXPORT int ou_mx4_quantize_grouped(int dtype, const void* x, int64_t rows, int64_t cols, int64_t row_stride,
                                      const int32_t* offsets, int32_t groups, uint8_t* codes, uint8_t* scales,
                                      uint8_t* codes_t, uint8_t* scales_t, void* stream)
{
    if (!valid_dtype(dtype)) return fail(OU_EINVAL, "unknown dtype %d", dtype);
    if (int st = check_axis(rows, "rows")) return st;
    if (int st = check_axis(cols, "cols")) return st;
    if (row_stride < cols || row_stride > kMaxAxis) return fail(OU_EINVAL, "row_stride is out of range");
    if (int st = check_groups(offsets, groups, rows)) return st;
    if (rows == 0 || cols == 0 || groups == 0) return OU_OK;
    if (!codes != !scales) return fail(OU_EINVAL, "codes and scales come in pairs");
    if (!codes_t || !scales_t) return fail(OU_EINVAL, "codes_t or scales_t is null");
    const int eb = elem_bytes(dtype);
    const int64_t pr = ou_mx4_grouped_columns(rows, groups);
    const Buffer bufs[] = {{"x", x, extent(rows, cols, row_stride, eb), static_cast<unsigned>(eb), false},
                           {"offsets", offsets, 4.0 * (groups + 1.0), 4, false},
                           {"codes", codes, codes ? held_codes(rows, pad(cols)) : 0, 16, true},
                           {"scales", scales, scales ? held_scales(rows, pad(cols)) : 0, 4, true},
                           {"codes_t", codes_t, held_codes(cols, pr), 16, true},
                           {"scales_t", scales_t, held_scales(cols, pr), 4, true}};
    if (int st = check_buffers(bufs, 6)) return st;
    QuantArgs q{x, codes, scales, codes_t, scales_t, rows, cols, row_stride, 0, pad(cols), pr, offsets, groups, 0};
    return launch_quantize(dtype, q, 1, pr / kQuantTile, stream);
}

OU_EXPORT int ou_mx4_dequantize(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                void* out, int64_t row_stride, void* stream)
{
    if (!valid_dtype(dtype)) return fail(OU_EINVAL, "unknown dtype %d", dtype);
    if (rows < 0 || rows > (int64_t(1) << 40)) return fail(OU_EINVAL, "rows is out of range");
    if (int st = check_axis(cols, "cols")) return st;
    if (row_stride < cols || row_stride > kMaxAxis) return fail(OU_EINVAL, "row_stride is out of range");
    if (rows == 0 || cols == 0) return OU_OK;
    const int eb = elem_bytes(dtype);
    const Buffer bufs[] = {{"codes", codes, held_codes(rows, pad(cols)), 16, false},
                           {"scales", scales, held_scales(rows, pad(cols)), 4, false},
                           {"out", out, extent(rows, cols, row_stride, eb), static_cast<unsigned>(eb), true}};
    if (int st = check_buffers(bufs, 3)) return st;
    DequantArgs d{codes, scales, out, rows, cols, pad(cols), row_stride, wide_rows(out, row_stride, 0, eb, 16)};
    if (rows * (pad(cols) / kPad) > UINT32_MAX / 2) return fail(OU_EINVAL, "the matrix is too large");
    uint32_t units = static_cast<uint32_t>(rows * (pad(cols) / kPad));
    void* args[] = {&d, &units};
    return launch({dequant_kernel(dtype), cut(units, (kQuantThreads / 16) * kQuantUnits), 1, kQuantThreads, "k_dequant",
                   0}, args, stream);
}

OU_EXPORT int64_t ou_mx4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k, int from_values)
{
    if (check_axis(m, "m") || check_axis(n, "n") || check_axis(k, "k")) return -1;
    return from_values && !choose(m, n, pad(k) / kPad, 1, m).values ? values_bytes(m, k) : 0;
}

OU_EXPORT int64_t ou_mx4_grouped_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t groups, int from_values)
{
    if (groups < 0 || groups > kMaxBatch) return -1;
    if (check_axis(rows, "rows") || check_axis(n, "n") || check_axis(k, "k")) return -1;
    return from_values && !choose_grouped(rows, n, pad(k) / kPad, groups).values ? values_bytes(rows, k) : 0;
}

}  // extern "C"

namespace {

// What the four products share.  x (or a): the left matrix as values (or held).
struct Product {
    int x_dtype;
    const void* x;
    int64_t x_stride;
    const uint8_t *a, *as;
    int64_t m;
    int out_dtype;
    const uint8_t *b, *bs;
    int64_t n, k;
    const int32_t* offsets;   // nullptr: not grouped
    int32_t groups;
    void* out;
    int64_t out_stride;
    int zero_rest;
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
};

int product(Product& q, bool values, bool grouped)
{
    if (!valid_dtype(q.out_dtype) || (values && !valid_dtype(q.x_dtype))) return fail(OU_EINVAL, "unknown dtype");
    if (int st = check_axis(q.m, "m")) return st;
    if (int st = check_axis(q.n, "n")) return st;
    if (int st = check_axis(q.k, "k")) return st;
    if (q.k > kMaxDepth) return fail(OU_EINVAL, "k = %lld: 2^25 at most", static_cast<long long>(q.k));
    if (values && (q.x_stride < q.k || q.x_stride > kMaxAxis)) return fail(OU_EINVAL, "x_stride is out of range");
    if (q.out_stride < q.n || q.out_stride > kMaxAxis) return fail(OU_EINVAL, "out_stride is out of range");
    if (grouped)
        if (int st = check_groups(q.offsets, q.groups, q.m)) return st;
    if (q.m == 0 || q.n == 0) return OU_OK;
    const int64_t need = grouped ? ou_mx4_grouped_workspace_bytes(q.m, q.n, q.k, q.groups, values)
                                 : ou_mx4_matmul_workspace_bytes(q.m, q.n, q.k, values);
    if (need > 0 && (!q.workspace || q.workspace_bytes < need))
        return fail(OU_EINVAL, "workspace: %lld bytes are needed", static_cast<long long>(need));
    const int64_t pk = pad(q.k);
    const int eo = elem_bytes(q.out_dtype), ex = values ? elem_bytes(q.x_dtype) : 1;
    const double bm = grouped ? q.groups : 1;
    const Buffer bufs[] = {{"x", q.x, values ? extent(q.m, q.k, q.x_stride, ex) : 0, static_cast<unsigned>(ex), false},
                           {"a_codes", q.a, values ? 0 : held_codes(q.m, pk), 16, false},
                           {"a_scales", q.as, values ? 0 : held_scales(q.m, pk), 4, false},
                           {"b_codes", q.b, bm * held_codes(q.n, pk), 16, false},
                           {"b_scales", q.bs, bm * held_scales(q.n, pk), 4, false},
                           {"offsets", q.offsets, grouped ? 4.0 * (q.groups + 1.0) : 0, 4, false},
                           {"workspace", q.workspace, static_cast<double>(need), 16, true},
                           {"out", q.out, extent(q.m, q.n, q.out_stride, eo), static_cast<unsigned>(eo), true}};
    if (int st = check_buffers(bufs, 8)) return st;
    const Choice c = grouped ? choose_grouped(q.m, q.n, pk / kPad, q.groups) : choose(q.m, q.n, pk / kPad, 1, q.m);
    MatmulArgs p{};
    if (values && c.values) {   // quantised where it is multiplied
        p.x = q.x;
        p.x_dtype = q.x_dtype;
        p.x_stride = q.x_stride;
        p.k = q.k;
        p.few_rows = static_cast<int32_t>(q.m < 16 ? q.m : 16);
        p.x_wide = wide_rows(q.x, q.x_stride, 0, ex, 16);
    }
    uint8_t* const wc = static_cast<uint8_t*>(q.workspace);
    const bool first = values && !c.values && pk > 0;   // quantised by a kernel of its own
    p.a = first ? wc : q.a;
    p.as = first ? wc + q.m * (pk / 2) : q.as;
    p.b = q.b;
    p.bs = q.bs;
    p.out = q.out;
    p.m = q.m;
    p.n = q.n;
    p.out_stride = q.out_stride;
    p.steps = pk / kPad;
    p.offsets = q.offsets;
    p.rows = q.m;
    p.groups = q.groups;
    p.zero_rest = q.zero_rest != 0;
    const Launch l = matmul_launch(q.out_dtype, grouped ? kByRows : kPlain, c, p, 1);
    if (int st = check_grid(l)) return st;
    if (first) {
        QuantArgs qa{q.x, wc, wc + q.m * (pk / 2), nullptr, nullptr, q.m, q.k, q.x_stride, 0, pk, 0, nullptr, 0, 0};
        if (int st = launch_quantize(q.x_dtype, qa, 1, 0, q.stream)) return st;
    }
    void* args[] = {&p};
    return launch(l, args, q.stream);
}

}  // namespace

extern "C" {

OU_EXPORT int ou_mx4_matmul(int out_dtype, const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                            const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k, void* out,
                            int64_t out_stride, void* workspace, int64_t workspace_bytes, void* stream)
{
    Product q{0,         nullptr, 0, a_codes, a_scales, m,          out_dtype, b_codes,   b_scales,        n, k,
              nullptr,   0,       out, out_stride, 0,   workspace,  workspace_bytes, stream};
    return product(q, false, false);
}

OU_EXPORT int ou_mx4_matmul_values(int x_dtype, const void* x, int64_t m, int64_t x_stride, int out_dtype,
                                   const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k, void* out,
                                   int64_t out_stride, void* workspace, int64_t workspace_bytes, void* stream)
{
    Product q{x_dtype, x, x_stride, nullptr, nullptr, m, out_dtype, b_codes, b_scales, n, k,
              nullptr, 0, out, out_stride, 0, workspace, workspace_bytes, stream};
    return product(q, true, false);
}

OU_EXPORT int ou_mx4_grouped_matmul(int out_dtype, const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows,
                                    const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                                    const int32_t* offsets, int32_t groups, void* out, int64_t out_stride,
                                    int zero_rest, void* workspace, int64_t workspace_bytes, void* stream)
{
    Product q{0, nullptr, 0, a_codes, a_scales, rows, out_dtype, b_codes, b_scales, n, k,
              offsets, groups, out, out_stride, zero_rest, workspace, workspace_bytes, stream};
    return product(q, false, true);
}

OU_EXPORT int ou_mx4_grouped_matmul_values(int x_dtype, const void* x, int64_t rows, int64_t x_stride, int out_dtype,
                                           const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                                           const int32_t* offsets, int32_t groups, void* out, int64_t out_stride,
                                           int zero_rest, void* workspace, int64_t workspace_bytes, void* stream)
{
    Product q{x_dtype, x, x_stride, nullptr, nullptr, rows, out_dtype, b_codes, b_scales, n, k,
              offsets, groups, out, out_stride, zero_rest, workspace, workspace_bytes, stream};
    return product(q, true, true);
}

OU_EXPORT int ou_mx4_grouped_outer(int out_dtype, const uint8_t* a_codes_t, const uint8_t* a_scales_t, int64_t m,
                                   const uint8_t* b_codes_t, const uint8_t* b_scales_t, int64_t n, int64_t rows,
                                   const int32_t* offsets, int32_t groups, void* out, void* stream)
{
    if (!valid_dtype(out_dtype)) return fail(OU_EINVAL, "unknown dtype %d", out_dtype);
    if (int st = check_axis(m, "m")) return st;
    if (int st = check_axis(n, "n")) return st;
    if (int st = check_axis(rows, "rows")) return st;
    if (int st = check_groups(offsets, groups, rows)) return st;
    if (m == 0 || n == 0 || groups == 0) return OU_OK;
    const int64_t pr = ou_mx4_grouped_columns(rows, groups);
    if (pr > kMaxDepth) return fail(OU_EINVAL, "%lld columns are held: 2^25 at most", static_cast<long long>(pr));
    const int eo = elem_bytes(out_dtype);
    const Buffer bufs[] = {{"a_codes_t", a_codes_t, held_codes(m, pr), 16, false},
                           {"a_scales_t", a_scales_t, held_scales(m, pr), 4, false},
                           {"b_codes_t", b_codes_t, held_codes(n, pr), 16, false},
                           {"b_scales_t", b_scales_t, held_scales(n, pr), 4, false},
                           {"offsets", offsets, 4.0 * (groups + 1.0), 4, false},
                           {"out", out, static_cast<double>(groups) * m * n * eo, static_cast<unsigned>(eo), true}};
    if (int st = check_buffers(bufs, 6)) return st;
    MatmulArgs p{};
    p.a = a_codes_t;
    p.as = a_scales_t;
    p.b = b_codes_t;
    p.bs = b_scales_t;
    p.out = out;
    p.m = m;
    p.n = n;
    p.out_stride = n;
    p.steps = pr / kPad;
    p.offsets = offsets;
    p.rows = rows;
    p.groups = groups;
    // Few rows have no kernel of their own here.  The steps are those of all
    // groups: how they are dealt is known on the device only.
    const Choice c = choose(m > 16 ? m : 17, n, p.steps, groups, 16);
    void* args[] = {&p};
    return launch(matmul_launch(out_dtype, kByContraction, c, p, groups), args, stream);
}

}  // extern "C"
