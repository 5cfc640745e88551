// int4_kernels.hip -- 4-bit whole-number weights with group scales (device):
// quantisation, dequantisation and products, plain and by expert.
//
// codes [n][k / 2], the even column in the low four bits; value = (code -
// zero) * scale, scales and zeros [n][k / group].
#include <type_traits>

#include "groups.hpp"
#include "int4_choice.hpp"
#include "values.hpp"

#pragma clang fp contract(off)

namespace experts {
namespace {

// `x` as the type holds it, at most its largest finite number.
__device__ __forceinline__ float rounded(float x, int dtype)
{
    if (dtype == kF32) return x;
    if (dtype == kF16) return fminf(Value<kF16>::to_float(Value<kF16>::from_float(x)), 65504.0f);
    const float r = Value<kBF16>::to_float(Value<kBF16>::from_float(x));
    return r > 3.3895313892515355e38f ? 3.3895313892515355e38f : r;
}

// Quotient and rest; 64-bit division only where it is needed.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t* rest)
{
    if (a >> 32 || b >> 32) {
        *rest = a % b;
        return a / b;
    }
    const uint32_t q = static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    *rest = static_cast<uint32_t>(a) - q * static_cast<uint32_t>(b);
    return q;
}

// 4, 8 or 16 lanes a group of columns, eight columns a lane and turn: its
// extremes, then its codes.  32768 x 8192 bf16: 289 us, bound by eight correctly
// rounded quotients a lane and turn; weights are laid out once.
template <int DT>
__global__ __launch_bounds__(kInt4Threads) void k_int4_quantize(Int4QuantArgs q)
{
    using P = Piece<DT, true>;
    using Elem = typename Value<DT>::Elem;
    const int lanes = 1 << q.lanes_log2, octets = q.group / 8;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kInt4Threads >> q.lanes_log2) + (threadIdx.x >> q.lanes_log2);
    const bool in = unit < q.rows * (q.k / q.group);
    const int lane = static_cast<int>(threadIdx.x) & (lanes - 1);
    int64_t g;
    const int64_t row = divide(in ? unit : 0, q.k / q.group, &g);
    const Elem* const x = static_cast<const Elem*>(q.x) + row * q.row_stride + g * q.group;
    float v[8];
    auto load = [&](int o) {
        if (q.wide) {
#pragma unroll
            for (int i = 0; i < 8; i += P::kValues) P::unpack(P::fetch(x, o * 8 + i), v + i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = Value<DT>::load(x, o * 8 + i);
        }
    };
    float lo = 0.0f, hi = 0.0f;
    for (int o = lane; o < octets; o += lanes) {
        load(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
        }
    }
    for (int s = lanes / 2; s; s >>= 1) {
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
    uint32_t* const codes = reinterpret_cast<uint32_t*>(q.codes) + (row * q.k + g * q.group) / 8;
    for (int o = lane; o < octets; o += lanes) {
        if (octets > lanes) load(o);   // else still there
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = scale > 0.0f ? rintf(v[i] / scale) + zero : zero;
            c |= static_cast<uint32_t>(fminf(fmaxf(u, 0.0f), 15.0f)) << (4 * i);
        }
        codes[o] = c;
    }
}

// Eight columns a thread, written as one or two pieces where rows allow it.
// 32768 x 8192 to bf16: 680 MB in 183 us, 3.7 TB/s.
template <int DT>
__global__ __launch_bounds__(kInt4Threads) void k_int4_dequantize(Int4Args p)
{
    using P = Piece<DT, true>;
    const int64_t octets = p.k / 8, u = static_cast<int64_t>(blockIdx.x) * kInt4Threads + threadIdx.x;
    if (u >= p.n * octets) return;
    int64_t o;
    const int64_t row = divide(u, octets, &o);
    const int64_t g = row * (p.k / p.group) + static_cast<uint32_t>(o * 8) / static_cast<uint32_t>(p.group);
    const uint32_t c = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p.codes) + u);
    const float scale = load_value(p.scales, g, p.scale_dtype);
    const float zero = p.zeros ? load_value(p.zeros, g, p.scale_dtype) : 8.0f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (static_cast<float>(c >> (4 * i) & 15u) - zero) * scale;
    const int64_t at = row * p.out_stride + o * 8;
    if (p.out_wide) {
#pragma unroll
        for (int i = 0; i < 8; i += P::kValues) P::store(p.out, at + i, v + i, true);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) Value<DT>::store(static_cast<typename Value<DT>::Elem*>(p.out), at + i, v[i]);
    }
}

// ---- products --------------------------------------------------------------------
//
// out[i][j] = sum over the groups g of scale[j][g] * (sum_k x[i][k] (code[j][k]
// - c) - (zero[j][g] - c) * sum_k x[i][k]), both inner sums over the group's
// columns by the 16x16x32 matrix instruction: code - c is a whole or half number
// of four bits and a sign, which bfloat16 and binary16 hold exactly, and x goes
// in as it is (binary32 in three bfloat16 parts that add up to it, down to
// 2^-133), so that every product is exact.  The sum of x is a product with ones.
// Weights are the instruction's second operand: lane l holds columns of row l
// mod 16, and its four results are of that row, so that a lane needs one scale a
// group.
//
// c is 7.5 for binary32 x and 0 for 16 bits.  With 0 the inner sums pass through
// twice the magnitude that (code - zero) has.  For binary32 x their error is then
// 1.4 to 1.6 times that of binary32 weights and a library product at 256 and 512
// columns (less from 1024 on); with 7.5 it is half of that, below the library's
// from 512 columns on and 1.05 times it at 256 (1.4e-7 to 0.9e-7 of the result).
// It costs 1 to 15 %: 16 x 1024 x 4096, 16 experts, 14.2 to 15.8 us, 16 rows x
// 14336 x 4096 20.2 to 22.4.  16-bit x, whose products are shorter, is at 0.2 to
// 0.7 times the library's error with 0 (binary32 results; others are rounded far
// above that) and would pay 5 to 17 %.

using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using f32x4 = float __attribute__((ext_vector_type(4)));

constexpr int kChunk = 128;   // columns of a step: 16 bytes of codes a lane

template <int DT>
constexpr float kCentre = DT == kF32 ? 7.5f : 0.0f;

// Eight codes less kCentre as values of the matrix instruction's type, in the
// order 0, 2, 4, 6, 1, 3, 5, 7.  A byte of 0 .. 15 is an 8-bit float (e4m3) of so
// many times 2^-9, subnormal numbers and the first binade being in line, and the
// converter multiplies by 2^9: seven instructions, fifteen by way of binary32.
// Less 7.5: twice the value is an odd number up to 15, its sign the code's top
// bit, the rest the three bits below, inverted where it is negative.

template <int DT>
__device__ __forceinline__ u32x4 code_values(uint32_t c)
{
    constexpr float kUnit = kCentre<DT> != 0.0f ? 256.0f : 512.0f;
    int lo, hi;
    if constexpr (kCentre<DT> != 0.0f) {
        const uint32_t above = c & 0x88888888u, n = ~(c ^ (above - (above >> 3)));
        lo = static_cast<int>((n << 1 & 0x0e0e0e0eu) | (n << 4 & 0x80808080u) | 0x01010101u);
        hi = static_cast<int>((n >> 3 & 0x0e0e0e0eu) | (n & 0x80808080u) | 0x01010101u);
    } else {
        lo = static_cast<int>(c & 0x0f0f0f0fu);
        hi = static_cast<int>(c >> 4 & 0x0f0f0f0fu);
    }
    if constexpr (DT == kF16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, kUnit, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, kUnit, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, kUnit, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, kUnit, true))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, kUnit, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, kUnit, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, kUnit, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, kUnit, true))};
}

// x's eight neighbouring values as operands: one, or three parts of binary32.
template <int DT>
struct Rows8 {
    static constexpr int kParts = DT == kF32 ? 3 : 1;
    static constexpr int kWords = DT == kF32 ? 8 : 4;
    u32x4 w[kWords / 4];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) w[i] = u32x4{0, 0, 0, 0};
    }
    // of any alignment that the elements have: the device's loads need no more
    __device__ __forceinline__ void load(const typename Value<DT>::Elem* p)
    {
        struct __attribute__((packed, aligned(sizeof(*p)))) Any {
            u32x4 w[kWords / 4];
        };
        const Any v = *reinterpret_cast<const Any*>(p);
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) w[i] = v.w[i];
    }
    // in the order of code_values()
    static __device__ __forceinline__ u32x4 ordered(u32x4 w)
    {
        constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
        return u32x4{__builtin_amdgcn_perm(w[1], w[0], kLow), __builtin_amdgcn_perm(w[3], w[2], kLow),
                     __builtin_amdgcn_perm(w[1], w[0], kHigh), __builtin_amdgcn_perm(w[3], w[2], kHigh)};
    }
    __device__ __forceinline__ void operands(u32x4* out) const
    {
        if constexpr (DT != kF32) {
            out[0] = ordered(w[0]);
        } else {
            // eight bits of the fraction each, cut off: the rests are exact
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = w[i / 2][2 * i % 4], b0 = w[i / 2][2 * i % 4 + 1];
                const float a1 = __builtin_bit_cast(float, a0) - __builtin_bit_cast(float, a0 & 0xffff0000u);
                const float b1 = __builtin_bit_cast(float, b0) - __builtin_bit_cast(float, b0 & 0xffff0000u);
                const uint32_t am = __builtin_bit_cast(uint32_t, a1), bm = __builtin_bit_cast(uint32_t, b1);
                const float a2 = a1 - __builtin_bit_cast(float, am & 0xffff0000u);
                const float b2 = b1 - __builtin_bit_cast(float, bm & 0xffff0000u);
                out[0][i] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
                out[1][i] = __builtin_amdgcn_perm(bm, am, 0x07060302u);
                out[2][i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b2), __builtin_bit_cast(uint32_t, a2), 0x07060302u);
            }
#pragma unroll
            for (int h = 0; h < 3; ++h) out[h] = ordered(out[h]);
        }
    }
};

template <int DT>
__device__ __forceinline__ f32x4 multiply(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT == kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The block's barrier for LDS alone: loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// 16 NT rows of weights and 16 rows of x a block, the steps of 128 columns dealt
// to its W waves in runs; U steps of a wave are in flight.  Lane group g (of 16
// lanes) loads columns 32 g .. of a step, one request of 64 bytes a row; the
// groups then exchange registers so that register i of group g holds columns
// 32 i + 8 g .., for two reasons: an instruction's 32 columns are of one group of
// columns, and x is asked for by 64 bytes a row (by 16 where the codes were
// loaded).  S groups of columns are in a step: a lane group loads the scale of
// one of four in a row, and a lane gets its row's from there.  HALF: scales have
// 16 bits.  No load of the steady loop stands behind a condition: the compiler
// could not tell how many are younger than the one that it waits for, and would
// wait for all; what is not there is loaded from elsewhere and does not count.
// One token, 4096 x 4096 bf16: 5.6 us, 9 MB at 1.6 TB/s, bound by the latency of
// launch and first loads; 32000 x 4096 21 us, 70 MB at 3.3 TB/s, 16 rows 25.8 us,
// 64 rows x 14336 x 4096 44 us, where codes become operands for every 16 rows.
// 32 or 64 rows a block instead were slower up to 64 rows (32 rows x 14336 x 4096:
// 42 and 52 us by one tile of weights, 27 and 31 by two, 24 as it is).
template <int DT, int S, int W, int U, int NT, bool HALF, bool GROUPED>
__global__ __launch_bounds__(kWave * W) void k_int4_matmul(Int4Args p)
{
    constexpr int P = Rows8<DT>::kParts, T = U > 4 / S ? U : 4 / S;   // T: steps of a turn of the loop
    using Elem = typename Value<DT>::Elem;
    using Bits = std::conditional_t<HALF, uint16_t, uint32_t>;
    __shared__ f32x4 sums[W][NT][kWave];
    const int t = static_cast<int>(threadIdx.x), lane = t & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t n_tiles = static_cast<uint32_t>((p.n + 16 * NT - 1) / (16 * NT));
    const uint32_t unit = blockIdx.x / n_tiles, ntile = blockIdx.x - unit * n_tiles;
    int64_t row0 = static_cast<int64_t>(unit) * 16, mrows = p.m - row0, matrix = 0;
    if constexpr (GROUPED) {
        const groups::Place at = groups::Groups(p.offsets, p.experts, p.m, 16).locate(unit);
        row0 = at.row;
        mrows = at.rows;
        matrix = at.group;
        if (mrows <= 0) return;
        if (matrix < 0 && !p.zero_rest) return;
    }
    const int rows = mrows < 16 ? static_cast<int>(mrows) : 16;
    const int64_t n0 = static_cast<int64_t>(ntile) * (16 * NT);
    const uint32_t columns = static_cast<uint32_t>(p.k / p.group), k = static_cast<uint32_t>(p.k);
    const int chunks = GROUPED && matrix < 0 ? 0 : static_cast<int>((k + kChunk - 1) / kChunk);
    const int run = (chunks + W - 1) / W, first = wave * run, last = first + run < chunks ? first + run : chunks;
    // rows behind the edge read the last one (of weights) or the first (of x), columns the last 32
    const uint8_t* codes[NT];
    const Bits *scales[NT], *zeros[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = (n0 + 16 * j + r < p.n ? n0 + 16 * j + r : p.n - 1) + (GROUPED && matrix > 0 ? matrix * p.n : 0);
        codes[j] = p.codes + n * (p.k / 2);
        scales[j] = static_cast<const Bits*>(p.scales) + n * columns;
        zeros[j] = p.zeros ? static_cast<const Bits*>(p.zeros) + n * columns : scales[j];
    }
    const Elem* const x = static_cast<const Elem*>(p.x) + (row0 + (r < rows ? r : 0)) * p.x_stride + g * 8;
    struct Step {
        u32x4 c[NT];
        Rows8<DT> x[4];
    } step[U];
    auto load = [&](Step& s, int at) {
        const uint32_t k0 = static_cast<uint32_t>(at) * kChunk, mine = k0 + static_cast<uint32_t>(g) * 32;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            s.c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes[j] + (mine < k ? mine : k - 32) / 2));
#pragma unroll
        for (int q = 0; q < 4; ++q) s.x[q].load(x + (k0 + q * 32 < k ? k0 + q * 32 : k - 32));
    };
    // scale and zero (less kCentre) of the group of columns `4 at + g` of the wave's run
    float scale[NT], zero[NT];
    Bits next_scale[NT], next_zero[NT];
    auto load_scales = [&](int at) {
        const uint32_t from = static_cast<uint32_t>(first) * kChunk + static_cast<uint32_t>(4 * at + g) * (kChunk / S);
        const uint32_t of = from / static_cast<uint32_t>(p.group), column = of < columns ? of : columns - 1;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            next_scale[j] = scales[j][column];
            next_zero[j] = zeros[j][column];
        }
    };
    f32x4 y[NT] = {};
    constexpr uint32_t kOne = DT == kF16 ? 0x3c003c00u : 0x3f803f80u;
    const u32x4 ones{kOne, kOne, kOne, kOne};
    auto compute = [&](const Step& s, int at) {
        const int of = (at - first) * S;   // the step's first group of columns in the run
        f32x4 sum[NT][S] = {}, plain[S] = {};
        uint32_t word[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint32_t c0 = s.c[j][0], c1 = s.c[j][1], c2 = s.c[j][2], c3 = s.c[j][3];
            swap32(c0, c2);
            swap32(c1, c3);
            swap16(c0, c1);
            swap16(c2, c3);
            word[j][0] = c0;
            word[j][1] = c1;
            word[j][2] = c2;
            word[j][3] = c3;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            constexpr int kPer = 4 / S;
            u32x4 b[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) b[j] = code_values<DT>(word[j][q]);
            u32x4 a[P];
            s.x[q].operands(a);
#pragma unroll
            for (int h = 0; h < P; ++h) {
                plain[q / kPer] = multiply<DT>(a[h], ones, plain[q / kPer]);
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[j][q / kPer] = multiply<DT>(a[h], b[j], sum[j][q / kPer]);
            }
        }
#pragma unroll
        for (int q = 0; q < S; ++q) {
            if (S > 1 && static_cast<uint32_t>(at) * kChunk + q * (kChunk / S) >= k) continue;   // k is a whole number of them
            const int from = ((of + q) & 3) * 64 + r * 4;   // the lane that has them
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float sc = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(from, __builtin_bit_cast(int, scale[j])));
                const float ze = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(from, __builtin_bit_cast(int, zero[j])));
#pragma unroll
                for (int e = 0; e < 4; ++e) y[j][e] = __builtin_fmaf(sc, __builtin_fmaf(-ze, plain[q][e], sum[j][q][e]), y[j][e]);
            }
        }
    };
    int at = first;
    auto turn = [&](auto steady) {
#pragma unroll
        for (int u = 0; u < T; ++u) {
            if (!steady.value && at + u >= last) break;
            if (u * S % 4 == 0) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    scale[j] = bits_value(next_scale[j], p.scale_dtype);
                    zero[j] = (p.zeros ? bits_value(next_zero[j], p.scale_dtype) : 8.0f) - kCentre<DT>;
                }
                if (steady.value || at + u + 4 / S < last) load_scales((at + u - first) * S / 4 + 1);
            }
            compute(step[u % U], at + u);
            if (steady.value || at + u + U < last) load(step[u % U], at + u + U);
        }
        at += T;
    };
    if (first + U + T <= last) {
        load_scales(0);
#pragma unroll
        for (int u = 0; u < U; ++u) load(step[u], first + u);
        do turn(std::true_type{});
        while (at + U + T <= last);
    } else if (first < last) {
        load_scales(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (first + u < last) load(step[u], first + u);
    }
    while (at < last) turn(std::false_type{});
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[wave][j][lane] = y[j];
    __syncthreads();
    static_assert(NT <= W, "a wave adds up 16 by 16 results");
    const int64_t column = n0 + 16 * wave + r;
    if (wave >= NT || column >= p.n) return;
    f32x4 out = sums[0][wave][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) out += sums[w][wave][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = g * 4 + e;
        if (row < rows) store_value(p.out, (row0 + row) * p.out_stride + column, out[e], p.out_dtype);
    }
}

// The same with x held: a block takes 16 rows of x and `p.tiles` tiles of 16 NT
// rows of weights one after the other, its W waves RC steps each of the
// columns, whose x they keep in registers; codes of the next two tiles are on
// their way.  The waves' sums meet in LDS, and the waves take turns at adding
// them up.  Here too no load of the steady loop stands behind a condition (the
// type of the scales has 16 bits).  The waves load the scales of 16 NT / W rows
// each, whole rows of them, and share them through LDS: when each loaded what it
// multiplies, they were 16 requests like the codes' own (21 us of 75 without any
// arithmetic); they are asked for a tile ahead of the codes.
// 512 rows over 64 experts, k = 2048, n = 4096 bf16: 80 us, 302 MB of codes and
// scales (experts of more than 16 rows read twice), 3.8 TB/s.  Loads alone take 58
// us with the 64 registers of x free for more waves: bound by how much three
// waves a SIMD keep on its way.
template <int DT, int S, int NT, int W, int RC, bool GROUPED>
__global__ __launch_bounds__(kWave * W) void k_int4_tiles(Int4Args p)
{
    constexpr int P = Rows8<DT>::kParts, D = 2, kUnits = W * RC * S;   // kUnits: groups of columns, at most
    constexpr int kRows = 16 * NT, kPart = kUnits * kRows / W, Q = kPart > kWave ? kPart / kWave : 1;   // loads of scales a lane and tile
    using Elem = typename Value<DT>::Elem;
    __shared__ f32x4 sums[2][W][NT][kWave];
    __shared__ f32x4 plain[W][RC * S][4];   // x's sums over a group of columns, four rows
    __shared__ float2 scaling[2][kRows][kUnits + 1];   // scale and zero less kCentre
    const int t = static_cast<int>(threadIdx.x), lane = t & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t all_tiles = static_cast<uint32_t>((p.n + kRows - 1) / kRows);
    const uint32_t parts = (all_tiles + p.tiles - 1) / p.tiles, unit = blockIdx.x / parts, part = blockIdx.x - unit * parts;
    int64_t row0 = static_cast<int64_t>(unit) * 16, mrows = p.m - row0, matrix = 0;
    if constexpr (GROUPED) {
        const groups::Place at = groups::Groups(p.offsets, p.experts, p.m, 16).locate(unit);
        row0 = at.row;
        mrows = at.rows;
        matrix = at.group;
        if (mrows <= 0) return;
        if (matrix < 0 && !p.zero_rest) return;
    }
    const int rows = mrows < 16 ? static_cast<int>(mrows) : 16;
    const int tile0 = static_cast<int>(part * p.tiles), left = static_cast<int>(all_tiles) - tile0;
    const int tiles = left < p.tiles ? left : p.tiles;
    const uint32_t columns = static_cast<uint32_t>(p.k / p.group);
    const int chunks = GROUPED && matrix < 0 ? 0 : static_cast<int>((p.k + kChunk - 1) / kChunk);
    const int run = (chunks + W - 1) / W, first = wave * run, count = first + run < chunks ? run : chunks - first;   // may be below 0
    const uint8_t* const codes = p.codes + (GROUPED && matrix > 0 ? matrix : 0) * p.n * (p.k / 2);
    const uint16_t *const scales = static_cast<const uint16_t*>(p.scales), *const zeros = static_cast<const uint16_t*>(p.zeros ? p.zeros : p.scales);
    const int64_t scale0 = (GROUPED && matrix > 0 ? matrix : 0) * p.n * columns;
    // the scales that the lane loads: rows wave * 16 / W .., all groups of columns
    uint32_t scale_at[Q], scale_row[Q], scale_unit[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const uint32_t f = (i * kWave + lane) % kPart;
        scale_row[i] = wave * (kRows / W) + f / kUnits;
        scale_unit[i] = f % kUnits;
        const uint32_t of = scale_unit[i] * (kChunk / S) / static_cast<uint32_t>(p.group);
        scale_at[i] = of < columns ? of : columns - 1;
    }
    // where the lane's codes of a step are; the row's first where there are none (x is 0 there)
    uint32_t place[RC];
#pragma unroll
    for (int c = 0; c < RC; ++c) {
        const bool inside = c < count && static_cast<int64_t>(first + c) * kChunk + g * 32 < p.k;
        place[c] = inside ? (static_cast<uint32_t>(first + c) * kChunk + g * 32) / 2 : 0;
    }

    struct Codes {
        u32x4 c[NT][RC];
    } tile[D];
    struct Scales {
        uint32_t scale[Q], zero[Q];   // their bits
    } scaled[D];
    const uint32_t row_bytes = static_cast<uint32_t>(p.k / 2);
    // rows behind the edge read the last one; the lanes' offsets from a tile fit 32 bits
    auto behind = [&](int at) { return p.n - 1 - static_cast<int64_t>(tile0 + at) * kRows; };
    auto load = [&](Codes& s, int at) {
        const int64_t last = behind(at);
        const uint8_t* const from = codes + static_cast<int64_t>(tile0 + at) * kRows * row_bytes;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t row = 16 * j + r < last ? 16 * j + r : static_cast<uint32_t>(last);
#pragma unroll
            for (int c = 0; c < RC; ++c)
                s.c[j][c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + (row * row_bytes + place[c])));
        }
    };
    auto load_scales = [&](Scales& s, int at) {
        const int64_t last = behind(at), base = scale0 + static_cast<int64_t>(tile0 + at) * kRows * columns;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const uint32_t of = (scale_row[i] < last ? scale_row[i] : static_cast<uint32_t>(last)) * columns + scale_at[i];
            s.scale[i] = scales[base + of];
            s.zero[i] = zeros[base + of];
        }
    };
    // a tile's scales to LDS, ahead of a barrier
    auto share = [&](const Scales& s, int at) {
#pragma unroll
        for (int i = 0; i < Q; ++i)
            scaling[at & 1][scale_row[i]][scale_unit[i]] =
                float2{bits_value(s.scale[i], p.scale_dtype), (p.zeros ? bits_value(s.zero[i], p.scale_dtype) : 8.0f) - kCentre<DT>};
    };
    const bool some = chunks > 0;
    const int most = tiles - 1;
    if (some) {   // those behind the last tile are that one's again
        load_scales(scaled[0], 0);
#pragma unroll
        for (int u = 0; u < D; ++u) load(tile[u], u < most ? u : most);
    }

    u32x4 a[RC][4][P];
    constexpr uint32_t kOne = DT == kF16 ? 0x3c003c00u : 0x3f803f80u;
    const u32x4 ones{kOne, kOne, kOne, kOne};
    const Elem* const x = static_cast<const Elem*>(p.x) + (row0 + (r < rows ? r : 0)) * p.x_stride + static_cast<int64_t>(first) * kChunk + g * 8;
#pragma unroll
    for (int c = 0; c < RC; ++c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            Rows8<DT> v;
            v.zero();
            if (r < rows && c < count && static_cast<int64_t>(first + c) * kChunk + q * 32 < p.k) v.load(x + c * kChunk + q * 32);
            v.operands(a[c][q]);
        }
    }
#pragma unroll
    for (int c = 0; c < RC; ++c) {
        f32x4 sum[S] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int h = 0; h < P; ++h) sum[q * S / 4] = multiply<DT>(a[c][q][h], ones, sum[q * S / 4]);
        if (r == 0) {
#pragma unroll
            for (int q = 0; q < S; ++q) plain[wave][c * S + q][g] = sum[q];
        }
    }
    if (some) {
        share(scaled[0], 0);
        load_scales(scaled[1], 1 < most ? 1 : most);
        load_scales(scaled[0], 2 < most ? 2 : most);
    }
    lds_barrier();

    auto store = [&](int at, int j, f32x4 v) {
        const int64_t n = static_cast<int64_t>(tile0 + at) * kRows + 16 * j + r;
        if (n >= p.n) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = g * 4 + e;
            if (row < rows) store_value(p.out, (row0 + row) * p.out_stride + n, v[e], p.out_dtype);
        }
    };
    auto compute = [&](const Codes& s, const Scales& then, int at) {
        // the steps' chains of instructions beside one another
        uint32_t word[NT][RC][4];
        f32x4 sum[NT][RC][S] = {}, y[NT] = {};
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < RC; ++c) {   // x and its sums are 0 in the steps that are not there
                uint32_t c0 = s.c[j][c][0], c1 = s.c[j][c][1], c2 = s.c[j][c][2], c3 = s.c[j][c][3];
                swap32(c0, c2);
                swap32(c1, c3);
                swap16(c0, c1);
                swap16(c2, c3);
                word[j][c][0] = c0;
                word[j][c][1] = c1;
                word[j][c][2] = c2;
                word[j][c][3] = c3;
            }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int c = 0; c < RC; ++c)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const u32x4 b = code_values<DT>(word[j][c][q]);
#pragma unroll
                    for (int h = 0; h < P; ++h) sum[j][c][q * S / 4] = multiply<DT>(a[c][q][h], b, sum[j][c][q * S / 4]);
                }
#pragma unroll
        for (int i = 0; i < RC * S; ++i) {
            const f32x4 xs = plain[wave][i][g];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float2 w = scaling[at & 1][16 * j + r][first * S + i];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[j][e] = __builtin_fmaf(w.x, __builtin_fmaf(-w.y, xs[e], sum[j][i / S][i % S][e]), y[j][e]);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[at & 1][wave][j][lane] = y[j];
        share(then, at + 1);
        lds_barrier();   // the tile before the last one was added up before its wave came here
        const int j = wave - at * NT % W;
        if (j < 0 || j >= NT) return;
        f32x4 v = sums[at & 1][0][j][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += sums[at & 1][w][j][lane];
        store(at, j, v);
    };
    if (!some) {   // rows of no group, or no columns
        for (int at = wave; at < tiles * NT; at += W) store(at / NT, at % NT, f32x4{0, 0, 0, 0});
        return;
    }
    static_assert(D == 2, "a tile's scales stand in the place of the one after the next");
    int at = 0;
    for (; at + D + 1 < tiles; at += D) {   // three tiles behind this one are there
#pragma unroll
        for (int u = 0; u < D; ++u) {
            compute(tile[u], scaled[1 - u], at + u);
            load_scales(scaled[1 - u], at + u + 3 < most ? at + u + 3 : most);
            load(tile[u], at + u + 2);
        }
    }
    for (; at < tiles; at += D) {   // three at most
#pragma unroll
        for (int u = 0; u < D; ++u) {
            if (at + u >= tiles) break;
            compute(tile[u], scaled[1 - u], at + u);
            if (at + u + 2 < tiles) load(tile[u], at + u + 2);
        }
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

namespace {

template <int DT, int S, bool HALF, bool GROUPED>
const void* streamed(const Int4Choice& c)
{
    if constexpr (DT != kF32 || S == 1)
        if (c.tiles == 4) return reinterpret_cast<const void*>(k_int4_matmul<DT, S, 4, 2, 4, HALF, GROUPED>);
    if (c.tiles == 2) return reinterpret_cast<const void*>(k_int4_matmul<DT, S, S == 1 ? 8 : 4, 2, 2, HALF, GROUPED>);
    return reinterpret_cast<const void*>(k_int4_matmul<DT, S, 8, 2, 1, HALF, GROUPED>);
}

template <int DT, int S, bool GROUPED>
const void* held(const Int4Choice& c)
{
    if (c.steps == 1) return reinterpret_cast<const void*>(k_int4_tiles<DT, S, 2, 8, 1, GROUPED>);
    if constexpr (DT != kF32)
        return reinterpret_cast<const void*>(k_int4_tiles<DT, S, 1, 4, 4, GROUPED>);
    else if constexpr (S > 1)
        return reinterpret_cast<const void*>(k_int4_tiles<DT, S, 1, 8, 2, GROUPED>);
    return nullptr;   // not reached: int4_holds() leaves binary32 with one group a step at 8 steps
}

template <int DT, int S, bool GROUPED>
Int4Kernel choose(int64_t steps, int64_t tiles, bool half)
{
    const Int4Choice c = int4_choice(DT == kF32, S, half, steps, tiles);
    const void* const fn = c.held ? held<DT, S, GROUPED>(c) : half ? streamed<DT, S, true, GROUPED>(c) : streamed<DT, S, false, GROUPED>(c);
    return {fn, c.waves, c.tiles, c.held};
}
template <int DT>
Int4Kernel choose(int scales, bool grouped, int64_t steps, int64_t tiles, bool half)
{
    if (grouped)
        return scales == 1   ? choose<DT, 1, true>(steps, tiles, half)
               : scales == 2 ? choose<DT, 2, true>(steps, tiles, half)
                             : choose<DT, 4, true>(steps, tiles, half);
    return scales == 1   ? choose<DT, 1, false>(steps, tiles, half)
           : scales == 2 ? choose<DT, 2, false>(steps, tiles, half)
                         : choose<DT, 4, false>(steps, tiles, half);
}

}  // namespace

Int4Kernel int4_matmul_kernel(int dtype, int scales, bool grouped, int64_t steps, int64_t tiles, bool half)
{
    return dtype == kF32   ? choose<kF32>(scales, grouped, steps, tiles, half)
           : dtype == kF16 ? choose<kF16>(scales, grouped, steps, tiles, half)
                           : choose<kBF16>(scales, grouped, steps, tiles, half);
}

}  // namespace experts
