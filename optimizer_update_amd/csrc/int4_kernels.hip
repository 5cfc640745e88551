// int4_kernels.hip -- 4-bit whole-number weights with group scales (device):
// quantisation, dequantisation and products, plain and by expert.
//
// codes [n][k / 2], the even column in the low four bits; value = (code -
// zero) * scale, scales and zeros [n][k / group].
#include "groups.hpp"
#include "values.hpp"

#pragma clang fp contract(off)

namespace experts {
namespace {

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
    return x;
}

// `x` as the type holds it, at most its largest finite number.
__device__ __forceinline__ float rounded(float x, int dtype)
{
    if (dtype == kF32) return x;
    if (dtype == kF16) return fminf(Value<kF16>::to_float(Value<kF16>::from_float(x)), 65504.0f);
    const float r = Value<kBF16>::to_float(Value<kBF16>::from_float(x));
    return r > 3.3895313892515355e38f ? 3.3895313892515355e38f : r;
}

// 16 lanes a group of columns: its extremes, then its codes, two a byte.
template <int DT>
__global__ __launch_bounds__(kInt4Threads) void k_int4_quantize(Int4QuantArgs q)
{
    const int64_t groups = q.k / q.group, unit = static_cast<int64_t>(blockIdx.x) * (kInt4Threads / 16) + (threadIdx.x >> 4);
    const bool in = unit < q.rows * groups;
    const int lane = static_cast<int>(threadIdx.x) & 15;
    const int64_t row = in ? unit / groups : 0, g = in ? unit - row * groups : 0;
    const typename Value<DT>::Elem* x = static_cast<const typename Value<DT>::Elem*>(q.x) + row * q.row_stride + g * q.group;
    float lo = 0.0f, hi = 0.0f;
    if (in) {
        for (int i = lane; i < q.group; i += 16) {
            const float v = Value<DT>::load(x, i);
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
    }
#pragma unroll
    for (int s = 8; s; s >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, s));
        hi = fmaxf(hi, __shfl_xor(hi, s));
    }
    if (!in) return;
    // the quotients first, so that nothing passes the largest number
    const float scale = rounded(q.zeros ? hi / 15.0f - lo / 15.0f : fmaxf(hi / 7.0f, lo / -8.0f), q.scale_dtype);
    const float zero = !q.zeros ? 8.0f : scale > 0.0f ? fminf(fmaxf(rintf(-lo / scale), 0.0f), 15.0f) : 0.0f;
    if (lane == 0) {
        store_value(q.scales, unit, scale, q.scale_dtype);
        if (q.zeros) store_value(q.zeros, unit, zero, q.scale_dtype);
    }
    uint8_t* codes = q.codes + row * (q.k / 2) + g * (q.group / 2);
    for (int i = lane; i < q.group / 2; i += 16) {
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float v = scale > 0.0f ? rintf(Value<DT>::load(x, 2 * i + h) / scale) + zero : zero;
            c[h] = static_cast<uint32_t>(fminf(fmaxf(v, 0.0f), 15.0f));
        }
        codes[i] = static_cast<uint8_t>(c[0] | c[1] << 4);
    }
}

// Eight columns a thread.
template <int DT>
__global__ __launch_bounds__(kInt4Threads) void k_int4_dequantize(Int4Args p)
{
    const int64_t octets = p.k / 8, u = static_cast<int64_t>(blockIdx.x) * kInt4Threads + threadIdx.x;
    if (u >= p.n * octets) return;
    const int64_t row = u / octets, o = u - row * octets;
    const int64_t g = row * (p.k / p.group) + o * 8 / p.group;
    const uint32_t c = reinterpret_cast<const uint32_t*>(p.codes)[u];
    const float scale = load_value(p.scales, g, p.scale_dtype);
    const float zero = p.zeros ? load_value(p.zeros, g, p.scale_dtype) : 8.0f;
    typename Value<DT>::Elem* out = static_cast<typename Value<DT>::Elem*>(p.out) + row * p.out_stride + o * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        Value<DT>::store(out, i, (static_cast<float>(c >> (4 * i) & 15u) - zero) * scale);
}

// A wave per row of weights and 16 rows of x.
template <bool GROUPED>
__global__ __launch_bounds__(kInt4Threads) void k_int4_matmul(Int4Args p)
{
    constexpr int kRows = 16, W = kInt4Threads / 64;
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const uint32_t n_tiles = static_cast<uint32_t>((p.n + W - 1) / W);
    const uint32_t unit = blockIdx.x / n_tiles;
    const int64_t n = static_cast<int64_t>(blockIdx.x - unit * n_tiles) * W + wave;
    int64_t row0 = static_cast<int64_t>(unit) * kRows, rows = p.m - row0, matrix = 0;
    if constexpr (GROUPED) {
        const groups::Place at = groups::Groups(p.offsets, p.experts, p.m, kRows).locate(unit);
        row0 = at.row;
        rows = at.rows;
        matrix = at.group;
        if (rows <= 0) return;
    }
    if (n >= p.n) return;
    if (rows > kRows) rows = kRows;
    if (GROUPED && matrix < 0) {
        if (p.zero_rest && lane < rows) store_value(p.out, (row0 + lane) * p.out_stride + n, 0.0f, p.out_dtype);
        return;
    }
    const int64_t row = matrix * p.n + n, groups = p.k / p.group;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(p.codes) + row * (p.k / 8);
    float acc[kRows] = {};
    for (int64_t o = lane; o < p.k / 8; o += 64) {
        const uint32_t c = codes[o];
        const int64_t g = row * groups + o * 8 / p.group;
        const float scale = load_value(p.scales, g, p.scale_dtype);
        const float zero = p.zeros ? load_value(p.zeros, g, p.scale_dtype) : 8.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= rows) break;
            float part = 0.0f;
            for (int i = 0; i < 8; ++i) {
                const float v = load_value(p.x, (row0 + r) * p.x_stride + o * 8 + i, p.x_dtype);
                part = __builtin_fmaf(v, static_cast<float>(c >> (4 * i) & 15u) - zero, part);
            }
            acc[r] = __builtin_fmaf(part, scale, acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float sum = wave_sum(acc[r]);
        if (lane == 0 && r < rows) store_value(p.out, (row0 + r) * p.out_stride + n, sum, p.out_dtype);
    }
}

}  // namespace

const void* int4_quantize_kernel(int dtype)
{
    return dtype == kF32   ? reinterpret_cast<const void*>(k_int4_quantize<kF32>)
           : dtype == kF16 ? reinterpret_cast<const void*>(k_int4_quantize<kF16>)
                           : reinterpret_cast<const void*>(k_int4_quantize<kBF16>);
}
const void* int4_dequantize_kernel(int dtype)
{
    return dtype == kF32   ? reinterpret_cast<const void*>(k_int4_dequantize<kF32>)
           : dtype == kF16 ? reinterpret_cast<const void*>(k_int4_dequantize<kF16>)
                           : reinterpret_cast<const void*>(k_int4_dequantize<kBF16>);
}
const void* int4_matmul_kernel(bool grouped)
{
    return grouped ? reinterpret_cast<const void*>(k_int4_matmul<true>) : reinterpret_cast<const void*>(k_int4_matmul<false>);
}

}  // namespace experts
