// mx4_kernels.hip -- microscaled 4-bit floats (device): quantisation,
// dequantisation and products.
//
// Format.  A block of 32 neighbouring values along the contracted axis holds
// one scale code s (the power of two 2^(s - 127); 255: the block has a NaN
// or an infinity and stands for NaN) and 32 codes of 4 bits: sign, two bits
// of exponent, one of mantissa, magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
// s = max(0, e - 2) with e the biased binary32 exponent of the block's
// largest magnitude, so the largest value lands in [4, 8) and what exceeds 6
// gives 6; all others round to nearest, ties to the even code.
//
// Held matrices: codes [rows][P / 2], the even column in the low four bits,
// and scales [rows][P / 32], P the columns padded to 128 with zeros.  A row
// is a whole number of 64-byte pieces, one k-step of the 16x16x128 matrix
// instruction.
#include <type_traits>

#include "mx4.h"

#pragma clang fp contract(off)

namespace mx4 {
namespace {

using i32x4 = int __attribute__((ext_vector_type(4)));
using i32x8 = int __attribute__((ext_vector_type(8)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));   // scales: 4-byte aligned
using f32x4 = float __attribute__((ext_vector_type(4)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));

// ---- storage types ------------------------------------------------------
// pack(): two neighbouring values as the converter takes them; the block's
// largest magnitude is found on the bit patterns without their signs, whose
// order as integers is that of the magnitudes with infinities and NaNs above.

template <int DT>
struct Type;

template <>
struct Type<kF32> {
    using Elem = float;
    static constexpr int kBytes = 4;
};
template <>
struct Type<kF16> {
    using Elem = uint16_t;
    static constexpr int kBytes = 2;
};
template <>
struct Type<kBF16> {
    using Elem = uint16_t;
    static constexpr int kBytes = 2;
};

// Biased binary32 exponent of a magnitude given by its storage bits.
template <int DT>
__device__ __forceinline__ uint32_t exponent_of(uint32_t mag)
{
    if constexpr (DT == kF32) return mag >> 23;
    if constexpr (DT == kBF16) return mag >> 7;
    const float f = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(mag)));
    return __builtin_bit_cast(uint32_t, f) >> 23;
}

__device__ __forceinline__ uint32_t scale_code(uint32_t e)
{
    return e == 255u ? 255u : (e < 2u ? 0u : e - 2u);
}

// The converter's scale operand: a binary32 whose exponent field is the scale
// code.
__device__ __forceinline__ float scale_operand(uint32_t s) { return __builtin_bit_cast(float, s << 23); }

// Packed maximum of the magnitudes of two 16-bit values.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    using u16x2 = uint16_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// Byte SEL of `old` becomes the codes of the pair (lo first).
template <int SEL>
__device__ __forceinline__ uint32_t convert_f32(uint32_t old, uint32_t lo, uint32_t hi, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __builtin_bit_cast(float, lo),
                                                    __builtin_bit_cast(float, hi), scale, SEL);
}
template <int DT, int SEL>
__device__ __forceinline__ uint32_t convert_16(uint32_t old, uint32_t pair, float scale)
{
    if constexpr (DT == kBF16)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), scale, SEL);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, pair), scale, SEL);
}

// Eight neighbouring values: storage bits, four dwords (16-bit types) or
// eight (binary32).
template <int DT>
struct Octet {
    static constexpr int kWords = Type<DT>::kBytes * 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }

    // n of the eight values starting at p (0 <= n <= 8), the rest 0.
    __device__ __forceinline__ void load(const typename Type<DT>::Elem* p, int n, bool wide)
    {
        if (n >= 8 && wide) {
            const u32x4* q = reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const u32x4 v = __builtin_nontemporal_load(q + i);
                w[4 * i] = v[0];
                w[4 * i + 1] = v[1];
                w[4 * i + 2] = v[2];
                w[4 * i + 3] = v[3];
            }
            return;
        }
        zero();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= n) continue;
            if constexpr (DT == kF32)
                w[i] = __builtin_bit_cast(uint32_t, p[i]);
            else
                w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        }
    }

    // Bits of the largest magnitude.
    __device__ __forceinline__ uint32_t top() const
    {
        if constexpr (DT == kF32) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
            uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
            for (int i = 1; i < 4; ++i) m = max_u16x2(m, w[i] & 0x7fff7fffu);
            return max(m & 0xffffu, m >> 16);
        }
    }

    __device__ __forceinline__ uint32_t codes(float scale) const
    {
        uint32_t r = 0;
        if constexpr (DT == kF32) {
            r = convert_f32<0>(r, w[0], w[1], scale);
            r = convert_f32<1>(r, w[2], w[3], scale);
            r = convert_f32<2>(r, w[4], w[5], scale);
            r = convert_f32<3>(r, w[6], w[7], scale);
        } else {
            r = convert_16<DT, 0>(r, w[0], scale);
            r = convert_16<DT, 1>(r, w[1], scale);
            r = convert_16<DT, 2>(r, w[2], scale);
            r = convert_16<DT, 3>(r, w[3], scale);
        }
        return r;
    }
};

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xf, 0xf, false)));
    return x;
}

// ---- groups ---------------------------------------------------------------

struct Place {
    int32_t group;    // -1: of no group (rows = 0: behind everything)
    int32_t row;      // first row of the unit
    int32_t rows;     // rows of the unit inside its group
};

// Sum over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x)
{
    // within rows of 16 lanes, then the rows' ends to the lanes behind them
    x += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x111, 0xf, 0xf, false));
    x += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x112, 0xf, 0xf, false));
    x += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x114, 0xf, 0xf, false));
    x += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x118, 0xf, 0xf, false));
    x += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x142, 0xa, 0xf, false));
    x += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x143, 0xc, 0xf, false));
    return x;
}

// Largest value over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x111, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x112, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x114, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x118, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x142, 0xa, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x143, 0xc, 0xf, false)));
    return x;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane)
{
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}

// The groups of a call, cut into units of `unit` rows each.  Offsets may be
// anything: they are clamped to [0, rows], and one below an earlier one counts
// as that one.  So every row is of one group at most, in front of the first or
// behind the last, and the units are no more than a grid that is sized for any
// rising offsets.  All lanes of a wave take part and get the same answers;
// lane l looks at group base + l.  The chunks of 64 groups are taken in order.
struct Groups {
    const int32_t* offsets;
    int32_t groups, rows, unit;
    // the chunk of 64 groups at hand
    int32_t base = -1;
    uint32_t lo, n, scan;

    __device__ __forceinline__ Groups(const int32_t* o, int32_t g, int64_t r, int u)
        : offsets(o), groups(g), rows(static_cast<int32_t>(r)), unit(u)
    {
    }
    __device__ __forceinline__ uint32_t offset(int32_t i) const
    {
        const int32_t o = offsets[i < groups ? i : groups];
        return static_cast<uint32_t>(o < 0 ? 0 : (o > rows ? rows : o));
    }
    __device__ __forceinline__ uint32_t units(uint32_t count) const { return (count + unit - 1) / unit; }
    __device__ __forceinline__ void chunk(int32_t at)
    {
        if (base == at) return;
        const uint32_t reached = at ? lane_value(lo + n, kWave - 1) : 0;   // by the chunk before
        base = at;
        const int32_t e = at + (static_cast<int>(threadIdx.x) & (kWave - 1));
        lo = offset(e);
        uint32_t hi = offset(e + 1);
        if (__ballot(hi < lo || lo < reached)) {
            lo = max(wave_max(lo), reached);
            hi = max(lo, hi);
        }
        n = hi - lo;
        scan = wave_scan(units(n));
    }
    // units of all groups
    __device__ __forceinline__ uint32_t total()
    {
        uint32_t before = 0;
        for (int32_t at = 0; at < groups; at += kWave) {
            chunk(at);
            before += lane_value(scan, kWave - 1);
        }
        return before;
    }
    // end of the rows in front of the first group; start of those behind the
    // last one, whose chunk is at hand; units of both
    __device__ __forceinline__ uint32_t front() const { return groups ? offset(0) : 0; }
    __device__ __forceinline__ uint32_t back() const { return groups ? lane_value(lo + n, kWave - 1) : 0; }
    __device__ __forceinline__ uint32_t rest() const { return units(front()) + units(rows - back()); }
    // unit `index` of all, those of no group last
    __device__ __forceinline__ Place locate(uint32_t index)
    {
        uint32_t before = 0;
        for (int32_t at = 0; at < groups; at += kWave) {
            chunk(at);
            const uint64_t past = __ballot(before + scan > index);
            if (past) {
                const int hit = __builtin_ctzll(past);
                const uint32_t count = lane_value(n, hit);
                const uint32_t first = before + lane_value(scan, hit) - units(count);
                const uint32_t from = (index - first) * unit;
                return Place{at + hit, static_cast<int32_t>(lane_value(lo, hit) + from),
                             static_cast<int32_t>(count - from < static_cast<uint32_t>(unit) ? count - from : unit)};
            }
            before += lane_value(scan, kWave - 1);
        }
        const uint32_t f = front(), b = back(), nf = units(f), j = index - before;
        if (j >= nf + units(rows - b)) return Place{-1, 0, 0};
        const uint32_t row = j < nf ? j * unit : b + (j - nf) * unit, end = j < nf ? f : rows;
        return Place{-1, static_cast<int32_t>(row),
                     static_cast<int32_t>(end - row < static_cast<uint32_t>(unit) ? end - row : unit)};
    }
    // units of the groups before `group`, and its own
    __device__ __forceinline__ void span(int32_t group, uint32_t* first, uint32_t* count)
    {
        uint32_t before = 0;
        for (int32_t at = 0;; at += kWave) {
            chunk(at);
            if (group < at + kWave) break;
            before += lane_value(scan, kWave - 1);
        }
        const uint32_t own = units(lane_value(n, group - base));
        *first = before + lane_value(scan, group - base) - own;
        *count = own;
    }
};

// The tile of a block: XCDs (blocks b mod 8) take contiguous runs of the tile
// order, which walks bands of 8 units down, then along n, so that the blocks
// that run together on one XCD share rows of a and of b in its L2.
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t units, uint32_t n_tiles, uint32_t* unit, uint32_t* ntile)
{
    const uint32_t total = units * n_tiles, x = b & 7, per = total >> 3, extra = total & 7;
    const uint32_t t = x * per + (x < extra ? x : extra) + (b >> 3);
    constexpr uint32_t kBand = 8;
    const uint32_t band = t / (kBand * n_tiles), in = t - band * kBand * n_tiles;
    const uint32_t left = units - band * kBand, h = left < kBand ? left : kBand;
    *ntile = in / h;
    *unit = band * kBand + (in - *ntile * h);
}

// ---- quantisation along the columns --------------------------------------

// 16 lanes hold one unit of 128 columns of a row, eight values a lane, so a
// block is a quad and its largest magnitude two lane exchanges away.  Bound by
// memory: lanes keep kQuantUnits units in flight (2 and 8 of them measured
// within 3%).  32000 x 1024 bf16 16.4 us, 5.1 TB/s; 8192 x 8192 31 us, 5.5.
template <int DT>
__global__ __launch_bounds__(kQuantThreads) void k_quant_rows(QuantArgs q, uint32_t units)
{
    using Elem = typename Type<DT>::Elem;
    const uint32_t per_row = static_cast<uint32_t>(q.pcols / kPad);
    const int sub = static_cast<int>(threadIdx.x) & 15;
    const uint32_t first = blockIdx.x * (kQuantThreads / 16 * kQuantUnits) + (threadIdx.x >> 4);
    const int64_t batch = blockIdx.y;
    const Elem* x = static_cast<const Elem*>(q.x) + batch * q.batch_stride;
    uint8_t* codes = q.codes + batch * q.rows * (q.pcols / 2);
    uint8_t* scales = q.scales + batch * q.rows * (q.pcols / kBlock);
    Octet<DT> v[kQuantUnits];
#pragma unroll
    for (int i = 0; i < kQuantUnits; ++i) {
        const uint32_t u = first + i * (kQuantThreads / 16);
        if (u >= units) {
            v[i].zero();
            continue;
        }
        const uint32_t row = u / per_row;
        const int64_t col = static_cast<int64_t>(u - row * per_row) * kPad + sub * 8, left = q.cols - col;
        v[i].load(x + row * q.row_stride + col, left < 0 ? 0 : (left > 8 ? 8 : static_cast<int>(left)), q.wide);
    }
#pragma unroll
    for (int i = 0; i < kQuantUnits; ++i) {
        const uint32_t u = first + i * (kQuantThreads / 16);
        const uint32_t s = scale_code(exponent_of<DT>(quad_max(v[i].top())));
        const uint32_t c = s == kScaleNaN ? 0u : v[i].codes(scale_operand(s));
        if (u >= units) continue;
        reinterpret_cast<uint32_t*>(codes)[static_cast<int64_t>(u) * 16 + sub] = c;
        if ((sub & 3) == 0) scales[static_cast<int64_t>(u) * (kPad / kBlock) + (sub >> 2)] = static_cast<uint8_t>(s);
    }
}

// ---- quantisation along the rows, or along both axes ---------------------

// One tile of 128 x 128 values, bound by memory (16384 x 8192 bf16 along both
// axes: 411 MB in 86 us, the rate of a copy).  It is read along the columns (eight values
// a lane), quantised that way from registers if wanted, and left in LDS;
// then each lane takes two neighbouring columns and a block of 32 rows.
// The lanes of a wave read neighbouring dwords of one row of LDS, so they meet
// on no bank; the row pitch of four dwords more than a row keeps the writes,
// four rows a wave, apart.
template <int DT>
__global__ __launch_bounds__(kQuantThreads) void k_quant_tile(QuantArgs q)
{
    using Elem = typename Type<DT>::Elem;
    constexpr int T = kQuantTile;
    constexpr int kRowWords = T * Type<DT>::kBytes / 4 + 4;
    __shared__ __attribute__((aligned(16))) uint32_t tile[T * kRowWords];
    const int t = static_cast<int>(threadIdx.x);
    const int64_t batch = blockIdx.y;
    const uint32_t col_tiles = static_cast<uint32_t>(q.pcols / T);
    uint32_t unit, col_tile;                            // block of 128 padded rows, of columns
    tile_of(blockIdx.x, gridDim.x / col_tiles, col_tiles, &unit, &col_tile);
    int64_t row0 = static_cast<int64_t>(unit) * T, nrows = q.rows - row0;
    if (q.offsets) {
        const Place p = Groups(q.offsets, q.groups, q.rows, T).locate(unit);
        if (p.group < 0) return;
        row0 = p.row;
        nrows = p.rows;
    }
    if (nrows > T) nrows = T;
    const int64_t col0 = static_cast<int64_t>(col_tile) * T;
    const Elem* x = static_cast<const Elem*>(q.x) + batch * q.batch_stride;
    const int sub = t & 15;
    const int64_t col = col0 + sub * 8, left = q.cols - col;
    const int n = left < 0 ? 0 : (left > 8 ? 8 : static_cast<int>(left));
    Octet<DT> v[T / 16];
#pragma unroll
    for (int i = 0; i < T / 16; ++i) {
        const int r = i * 16 + (t >> 4);
        v[i].load(x + (row0 + r) * q.row_stride + col, r < nrows ? n : 0, q.wide);
    }
#pragma unroll
    for (int i = 0; i < T / 16; ++i) {
        const int r = i * 16 + (t >> 4);
#pragma unroll
        for (int j = 0; j < Octet<DT>::kWords / 4; ++j)
            *reinterpret_cast<u32x4*>(&tile[r * kRowWords + sub * Octet<DT>::kWords + 4 * j]) =
                u32x4{v[i].w[4 * j], v[i].w[4 * j + 1], v[i].w[4 * j + 2], v[i].w[4 * j + 3]};
        if (!q.codes) continue;
        const uint32_t s = scale_code(exponent_of<DT>(quad_max(v[i].top())));
        const uint32_t c = s == kScaleNaN ? 0u : v[i].codes(scale_operand(s));
        if (r >= nrows || col >= q.pcols) continue;
        const int64_t at = (batch * q.rows + row0 + r) * (q.pcols / kBlock) + (col0 >> 5);
        *reinterpret_cast<uint32_t*>(q.codes + at * (kBlock / 2) + sub * 4) = c;
        if ((sub & 3) == 0) q.scales[at + (sub >> 2)] = static_cast<uint8_t>(s);
    }
    __syncthreads();
    const int pair = t & 63, rb = t >> 6;               // columns 2 pair, 2 pair + 1; rows 32 rb ..
    uint32_t top[2] = {0, 0};
    u32x4 out[2] = {};
    float sc[2];
    uint32_t s[2];
    if constexpr (DT == kF32) {
        u32x2 d[kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            d[i] = *reinterpret_cast<const u32x2*>(&tile[(rb * kBlock + i) * kRowWords + 2 * pair]);
            top[0] = max(top[0], d[i][0] & 0x7fffffffu);
            top[1] = max(top[1], d[i][1] & 0x7fffffffu);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            s[c] = scale_code(exponent_of<DT>(top[c]));
            sc[c] = scale_operand(s[c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t r = 0;
                r = convert_f32<0>(r, d[8 * i][c], d[8 * i + 1][c], sc[c]);
                r = convert_f32<1>(r, d[8 * i + 2][c], d[8 * i + 3][c], sc[c]);
                r = convert_f32<2>(r, d[8 * i + 4][c], d[8 * i + 5][c], sc[c]);
                r = convert_f32<3>(r, d[8 * i + 6][c], d[8 * i + 7][c], sc[c]);
                out[c][i] = r;
            }
        }
    } else {
        uint32_t d[kBlock], m = 0;
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            d[i] = tile[(rb * kBlock + i) * kRowWords + pair];
            m = max_u16x2(m, d[i] & 0x7fff7fffu);
        }
        top[0] = m & 0xffffu;
        top[1] = m >> 16;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            s[c] = scale_code(exponent_of<DT>(top[c]));
            sc[c] = scale_operand(s[c]);
            // the same column of two neighbouring rows as one pair
            constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
            const uint32_t sel = c ? kHigh : kLow;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t r = 0;
                r = convert_16<DT, 0>(r, __builtin_amdgcn_perm(d[8 * i + 1], d[8 * i], sel), sc[c]);
                r = convert_16<DT, 1>(r, __builtin_amdgcn_perm(d[8 * i + 3], d[8 * i + 2], sel), sc[c]);
                r = convert_16<DT, 2>(r, __builtin_amdgcn_perm(d[8 * i + 5], d[8 * i + 4], sel), sc[c]);
                r = convert_16<DT, 3>(r, __builtin_amdgcn_perm(d[8 * i + 7], d[8 * i + 6], sel), sc[c]);
                out[c][i] = r;
            }
        }
    }
    // Through LDS, so that a column's 64 bytes of codes and 4 of scales go out
    // as one piece each (80 bytes a column: no bank is met twice by a quad).
    __syncthreads();
    constexpr int kOut = 20;   // words a column
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (s[c] == kScaleNaN) out[c] = u32x4{0, 0, 0, 0};
        uint32_t* to = &tile[(2 * pair + c) * kOut];
        *reinterpret_cast<u32x4*>(to + 4 * rb) = out[c];
        reinterpret_cast<uint8_t*>(to + 16)[rb] = static_cast<uint8_t>(s[c]);
    }
    __syncthreads();
    const int64_t cols = q.cols - col0 < T ? q.cols - col0 : T;
    const int64_t at = (batch * q.cols + col0) * (q.prows / kBlock) + static_cast<int64_t>(unit) * (T / kBlock);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 64 + (t >> 2);
        if (c >= cols) continue;
        *reinterpret_cast<u32x4*>(q.codes_t + (at + c * (q.prows / kBlock)) * (kBlock / 2) + (t & 3) * 16) =
            *reinterpret_cast<const u32x4*>(&tile[c * kOut + 4 * (t & 3)]);
    }
    if (t < cols)
        *reinterpret_cast<uint32_t*>(q.scales_t + at + t * (q.prows / kBlock)) = tile[t * kOut + 16];
}

// ---- results in the storage types -----------------------------------------

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}

// Stores n (1..4) of four neighbouring results, rounded once to nearest even.
template <int DT>
__device__ __forceinline__ void store4(void* out, int64_t at, f32x4 v, int n, bool wide)
{
    if constexpr (DT == kF32) {
        float* p = static_cast<float*>(out) + at;
        if (n >= 4 && wide) {
            *reinterpret_cast<f32x4*>(p) = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = v[i];
    } else {
        const u32x2 w = DT == kBF16 ? u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}
                                    : u32x2{f16_pair(v[0], v[1]), f16_pair(v[2], v[3])};
        uint16_t* p = static_cast<uint16_t*>(out) + at;
        if (n >= 4 && wide) {
            *reinterpret_cast<u32x2*>(p) = w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

// ---- dequantisation ---------------------------------------------------------

// Two neighbouring codes (byte SEL of c) as values of the type, for scale
// codes whose values are all normal numbers of it (the converter flushes
// subnormal results): from 2^-126 and 2^-14 = 0.5 * 2^(s - 127) on, up to
// 6 * 2^(s - 127) within the type.
template <int DT>
struct Normal {
    static constexpr uint32_t kFirst = DT == kF16 ? 114 : 2, kLast = DT == kF16 ? 140 : 252;
};
template <int DT, int SEL>
__device__ __forceinline__ void values_of(uint32_t c, float scale, uint32_t* out)
{
    if constexpr (DT == kF32) {
        // by way of bfloat16, which holds these values exactly
        const uint32_t v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, SEL));
        out[0] = v << 16;
        out[1] = v & 0xffff0000u;
    } else if constexpr (DT == kBF16) {
        out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, SEL));
    } else {
        out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, SEL));
    }
}

// The value of one code under any scale code, in binary32.
__device__ __forceinline__ float value_of(uint32_t code, uint32_t s)
{
    const uint32_t e = (code >> 1) & 3u, m = code & 1u;
    const float scale = s == kScaleNaN ? __builtin_nanf("") : __builtin_bit_cast(float, s ? s << 23 : 1u << 22);
    const float mag = e ? __builtin_bit_cast(float, ((e + 126u) << 23) | (m << 22)) : 0.5f * static_cast<float>(m);
    return (code & 8u ? -mag : mag) * scale;
}

// As k_quant_rows: 16 lanes a unit of 128 columns, eight values a lane,
// kQuantUnits units of a lane in flight.  Bound by the values' way out:
// 16384 x 8192 to bf16 339 MB in 49 us by non-temporal stores, 60 to 77 by
// others.
template <int DT>
__global__ __launch_bounds__(kQuantThreads) void k_dequant(DequantArgs d, uint32_t units)
{
    using Elem = typename Type<DT>::Elem;
    constexpr int kWords = Type<DT>::kBytes * 2;
    const uint32_t per_row = static_cast<uint32_t>(d.pcols / kPad);
    const int sub = static_cast<int>(threadIdx.x) & 15;
    const uint32_t first = blockIdx.x * (kQuantThreads / 16 * kQuantUnits) + (threadIdx.x >> 4);
    uint32_t c[kQuantUnits], s[kQuantUnits];
#pragma unroll
    for (int i = 0; i < kQuantUnits; ++i) {
        const uint32_t u = first + i * (kQuantThreads / 16), v = u < units ? u : units - 1;
        c[i] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(d.codes) + static_cast<int64_t>(v) * 16 + sub);
        s[i] = d.scales[static_cast<int64_t>(v) * (kPad / kBlock) + (sub >> 2)];
    }
#pragma unroll
    for (int i = 0; i < kQuantUnits; ++i) {
        const uint32_t u = first + i * (kQuantThreads / 16);
        if (u >= units) continue;
        const uint32_t row = u / per_row;
        const int64_t col = static_cast<int64_t>(u - row * per_row) * kPad + sub * 8, left = d.cols - col;
        if (left <= 0) continue;
        uint32_t w[kWords];
        if (s[i] >= Normal<DT>::kFirst && s[i] <= Normal<DT>::kLast) {
            const float scale = scale_operand(s[i]);
            values_of<DT, 0>(c[i], scale, w);
            values_of<DT, 1>(c[i], scale, w + kWords / 4);
            values_of<DT, 2>(c[i], scale, w + kWords / 2);
            values_of<DT, 3>(c[i], scale, w + 3 * kWords / 4);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = value_of((c[i] >> (8 * j)) & 15u, s[i]), b = value_of((c[i] >> (8 * j + 4)) & 15u, s[i]);
                if constexpr (DT == kF32) {
                    w[2 * j] = __builtin_bit_cast(uint32_t, a);
                    w[2 * j + 1] = __builtin_bit_cast(uint32_t, b);
                } else {
                    w[j] = DT == kBF16 ? bf16_pair(a, b) : f16_pair(a, b);
                }
            }
        }
        Elem* out = static_cast<Elem*>(d.out) + row * d.row_stride + col;
        if (left >= 8 && d.wide) {
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j)
                __builtin_nontemporal_store(u32x4{w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]},
                                            reinterpret_cast<u32x4*>(reinterpret_cast<uint32_t*>(out) + 4 * j));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= left) continue;
                if constexpr (DT == kF32)
                    out[j] = __builtin_bit_cast(float, w[j]);
                else
                    out[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
            }
        }
    }
}

// ---- products -----------------------------------------------------------------

// A wave's fragment of a matrix for the 16x16x128 instruction: lane l holds
// the 32 columns 32 (l / 16) .. of row l mod 16, and the scale of that block.
__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// The block's barrier alone; no LDS access moves across it.
__device__ __forceinline__ void block_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Up to 16 rows (of a group): 16 x 16 NT results a block, the k-steps dealt to
// its W waves in contiguous runs of pairs, b's fragments loaded straight to
// registers.  Such a product waits for b from memory: its first U pairs are
// under way before anything else.  Which block of 32 columns a lane holds is
// free as long as a and b agree: here lane group g holds blocks 2 g (for the
// first product of a pair) and 2 g + 1 (for the second) of the pair's eight,
// so that the four lanes of a row ask for 128 bytes together.  With XT the
// left matrix is given as values of that type: the block meanwhile quantises
// its rows into LDS.  The fragment of b is the instruction's first operand, so
// that a lane's four results are neighbours in a row of out.
// 16 x 4096 x 4096, held: 10.0 us; 17.0 where a row's lanes ask for 64 bytes
// and each step for its scales by itself.
template <int XT, int G, int NT, int W, int U>
__global__ __launch_bounds__(kWave * W) void k_matmul_few(MatmulArgs p)
{
    constexpr bool kValues = XT != kHeld;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = static_cast<int>(threadIdx.x), lane = t & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t unit = blockIdx.x / static_cast<uint32_t>(p.n_tiles);
    const uint32_t ntile = blockIdx.x - unit * static_cast<uint32_t>(p.n_tiles);
    int64_t row0 = static_cast<int64_t>(unit) * 16, mrows = p.m - row0;
    const int row_steps = static_cast<int>(p.steps);   // at most 2^18
    int steps = row_steps;
    const uint8_t *b = p.b, *bs = p.bs;
    if constexpr (G == kByRows) {
        const Place at = Groups(p.offsets, p.groups, p.rows, 16).locate(unit);
        row0 = at.row;
        mrows = at.rows;
        if (mrows <= 0) return;
        if (at.group < 0) {
            if (!p.zero_rest) return;
            steps = 0;   // rows of no group: the sum over nothing
        } else {
            b += at.group * p.n * p.steps * (kPad / 2);
            bs += at.group * p.n * p.steps * (kPad / kBlock);
        }
    }
    const int rows = mrows < 16 ? static_cast<int>(mrows) : 16;
    const int64_t n0 = static_cast<int64_t>(ntile) * (16 * NT);
    const uint8_t *bp[NT], *bsp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        int64_t n = n0 + 16 * j + r;
        n = n < p.n ? n : p.n - 1;           // rows behind the edge read the last one
        bp[j] = b + n * p.steps * (kPad / 2) + g * 32;
        bsp[j] = bs + n * p.steps * (kPad / kBlock);
    }
    const int pairs = (steps + 1) / 2, run = (pairs + W - 1) / W, first = wave * run;
    const int last = first + run < pairs ? first + run : pairs;
    i32x4 bv[U][NT][2];
    uint32_t bsc[U][NT];   // the lane's two scale codes, in the low bytes
    // An odd last step is half a pair: lanes of groups 2 and 3 hold nothing of it.
    auto whole = [&](int q) { return 2 * q + 1 < steps; };
    auto load_b = [&](int q0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (U == 2 && q0 + 1 < last && whole(q0 + 1)) {   // four steps' scales of a row by one request
                const u32x4_any w = *reinterpret_cast<const u32x4_any*>(bsp[j] + q0 * 8);
#pragma unroll
                for (int u = 0; u < U; ++u) bsc[u][j] = (g & 2 ? w[2 * u + 1] : w[2 * u]) >> (16 * (g & 1));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u < last ? q0 + u : last - 1;
                const i32x4* c = reinterpret_cast<const i32x4*>(bp[j] + static_cast<int64_t>(q) * 128);
                const uint16_t* w = reinterpret_cast<const uint16_t*>(bsp[j] + q * 8 + 2 * g);
                const bool scales = !(U == 2 && q0 + 1 < last && whole(q0 + 1));
                if (whole(q)) {
                    bv[u][j][0] = c[0];
                    bv[u][j][1] = c[1];
                    if (scales) bsc[u][j] = *w;
                } else {
                    bv[u][j][0] = g < 2 ? c[0] : i32x4{0, 0, 0, 0};
                    bv[u][j][1] = g < 2 ? c[1] : i32x4{0, 0, 0, 0};
                    bsc[u][j] = g < 2 ? *w : 0;
                }
            }
        }
    };
    if (first < last) load_b(first);
    // the left fragments' source: row, or the last one
    const int ar = r < rows ? r : rows - 1;
    const uint8_t *ap, *asp;
    uint8_t* tail = lds;
    if constexpr (kValues) {
        // codes of the rows, 16 bytes more apart than they are long, then scales
        const int pitch = row_steps * (kPad / 2) + 16, spitch = row_steps * 4 + 4;
        using Elem = typename Type<XT>::Elem;
        const Elem* x = static_cast<const Elem*>(p.x) + row0 * p.x_stride;
        const int units = steps ? rows * row_steps : 0, sub = t & 15;
        uint8_t* const sc = lds + p.few_rows * pitch;
        constexpr int kAhead = 4;
        for (int u0 = t >> 4; u0 < units; u0 += 4 * W * kAhead) {
            Octet<XT> v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int u = u0 + i * 4 * W;
                v[i].zero();
                if (u >= units) continue;
                const int row = u / row_steps, step = u - row * row_steps;
                const int64_t col = static_cast<int64_t>(step) * kPad + sub * 8, left = p.k - col;
                v[i].load(x + row * p.x_stride + col, left < 0 ? 0 : (left > 8 ? 8 : static_cast<int>(left)), p.x_wide);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int u = u0 + i * 4 * W;
                const uint32_t s = scale_code(exponent_of<XT>(quad_max(v[i].top())));
                if (u >= units) continue;
                const int row = u / row_steps, step = u - row * row_steps;
                *reinterpret_cast<uint32_t*>(lds + row * pitch + step * (kPad / 2) + sub * 4) =
                    s == kScaleNaN ? 0u : v[i].codes(scale_operand(s));
                if ((sub & 3) == 0) sc[row * spitch + step * 4 + (sub >> 2)] = static_cast<uint8_t>(s);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        block_barrier();
        ap = lds + ar * pitch + g * 32;
        asp = sc + ar * spitch + 2 * g;
        tail = sc + (p.few_rows * spitch + 15) / 16 * 16;
    } else {
        ap = p.a + (row0 + ar) * p.steps * (kPad / 2) + g * 32;
        asp = p.as + (row0 + ar) * p.steps * (kPad / kBlock) + 2 * g;
    }
    f32x4 acc[NT] = {};
    for (int q0 = first; q0 < last; q0 += U) {
        if (q0 > first) load_b(q0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = q0 + u;
            if (q >= last) break;
            i32x4 av[2] = {};
            uint32_t as = 0;
            if (whole(q) || g < 2) {
                av[0] = *reinterpret_cast<const i32x4*>(ap + static_cast<int64_t>(q) * 128);
                av[1] = *reinterpret_cast<const i32x4*>(ap + static_cast<int64_t>(q) * 128 + 16);
                as = *reinterpret_cast<const uint16_t*>(asp + q * 8);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    widen(bv[u][j][0]), widen(av[0]), acc[j], 4, 4, 0, static_cast<int>(bsc[u][j]), 0, static_cast<int>(as));
                acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    widen(bv[u][j][1]), widen(av[1]), acc[j], 4, 4, 1, static_cast<int>(bsc[u][j]), 1, static_cast<int>(as));
            }
        }
    }
    // the waves' sums, joined in LDS in the order of the waves, rounded once
    f32x4 (*part)[NT][kWave] = reinterpret_cast<f32x4(*)[NT][kWave]>(tail);
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < NT; j += W) {
        f32x4 sum = part[0][j][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += part[w][j][lane];
        const int64_t n = n0 + 16 * j + 4 * g, left = p.n - n;
        if (r >= rows || left <= 0) continue;
        const int64_t at = (row0 + r) * p.out_stride + n;
        const int have = left > 4 ? 4 : static_cast<int>(left);
        if (p.out_dtype == kF32)
            store4<kF32>(p.out, at, sum, have, p.wide);
        else if (p.out_dtype == kF16)
            store4<kF16>(p.out, at, sum, have, p.wide);
        else
            store4<kBF16>(p.out, at, sum, have, p.wide);
    }
}

// ---- products, tiled through LDS ------------------------------------------

// 16 bytes a lane from `rsrc` + voff to LDS at lds + lane * 16; what lies
// behind the resource's end arrives as 0.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, 0);
}

// All but the newest LEFT transfers of the wave have arrived.
template <int LEFT>
__device__ __forceinline__ void wait_transfers()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
}

// acc += the product of two fragments, in place.  Written as assembly because
// the builtin's result may be another register than its addend, and with the
// whole accumulator file in use the compiler then moves and spills
// accumulators.  settle_products() stands before the first other use of acc:
// the compiler does not know that this is a matrix instruction.
__device__ __forceinline__ void multiply_add(f32x4& acc, i32x4 b, i32x4 a, int sb, int sa)
{
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(acc)
                 : "v"(b), "v"(a), "v"(sb), "v"(sa));
}
__device__ __forceinline__ void settle_products() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(uint64_t address, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(address), 0, static_cast<int>(bytes), 0x00020000);
}

// f(0), f(1), .. f(N - 1), each with its index as a constant.
template <int N, int X = 0, class F>
__device__ __forceinline__ void each(F&& f)
{
    if constexpr (X < N) {
        f(std::integral_constant<int, X>{});
        each<N, X + 1>(f);
    }
}

// Bound by the matrix units, as far as power lets them: 8192^3 in 233 to 241 us,
// 4.6 to 4.7 PFLOP/s, where the instruction alone reaches 7.3 on random codes
// and is busy 57% of the cycles here.  256 x 256 results a block read the least
// from L2; its registers leave one wave a SIMD, so everything else must fit
// between the matrix instructions.
//
// Four waves in a square, 16 WM x 16 WN results each.  A pair is two k-steps,
// 256 columns: 128 bytes of codes of every row, moved to LDS in two
// alternating buffers (pieces of 128 bytes: the memory pipeline takes about
// 0.42 requests a cycle and CU whether they are of 64 or of 128 bytes); the
// scales of four pairs (32 bytes a row) move together, a quarter with each
// pair.  A wave multiplies the fragments of one k-step from registers while
// it reads those of the next from LDS; transfers start as soon as a buffer is
// free and are laid between the matrix instructions.  In LDS the eight
// 16-byte pieces of a row are exchanged by (row / 2) mod 8: a read of one
// piece of 16 rows by 64 lanes then meets no bank twice (lanes 0-3, 12-15,
// 20-27 of it go together, and so on).
// With few tiles KG such groups of waves share a block, each with its part of
// LDS and a contiguous part of the pairs; their sums are added in order.
template <int DT, int G, int WM, int WN, int KG>
__global__ __launch_bounds__(256 * KG, 1) void k_matmul_tile(MatmulArgs p)
{
    constexpr int BM = 32 * WM, BN = 32 * WN;
    constexpr int kCodes = (BM + BN) * 128, kScales = (BM + BN) * 32, kGroup = 2 * kCodes + 2 * kScales;
    __shared__ __attribute__((aligned(16))) uint8_t all_lds[KG * kGroup];
    const int lane = static_cast<int>(threadIdx.x) & 63, r = lane & 15, g = lane >> 4;
    const int block_wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int wave = block_wave & 3, kg = block_wave >> 2;   // of the group; the group
    uint8_t* const lds = all_lds + kg * kGroup;
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

    uint32_t unit, ntile;   // a grid holds fewer than 2^31 tiles
    int64_t row0, mrows, step0 = 0, steps = p.steps, out0 = 0;
    const uint8_t *b = p.b, *bs = p.bs;
    if constexpr (G == kByRows) {
        Groups groups(p.offsets, p.groups, p.rows, BM);
        uint32_t units = groups.total();
        if (p.zero_rest) units += groups.rest();
        if (static_cast<int64_t>(blockIdx.x) >= static_cast<int64_t>(units) * p.n_tiles) return;
        tile_of(blockIdx.x, units, static_cast<uint32_t>(p.n_tiles), &unit, &ntile);
        const Place at = groups.locate(unit);
        row0 = at.row;
        mrows = at.rows;
        if (mrows <= 0) return;
        if (at.group < 0) {
            steps = 0;   // rows of no group: the sum over nothing
        } else {
            b += static_cast<int64_t>(at.group) * p.n * p.steps * (kPad / 2);
            bs += static_cast<int64_t>(at.group) * p.n * p.steps * (kPad / kBlock);
        }
    } else {
        tile_of(blockIdx.x, static_cast<uint32_t>(p.units), static_cast<uint32_t>(p.n_tiles), &unit, &ntile);
        row0 = static_cast<int64_t>(unit) * BM;
        mrows = p.m - row0;
        if constexpr (G == kByContraction) {
            uint32_t before, own;
            Groups(p.offsets, p.groups, p.rows, kPad).span(static_cast<int32_t>(blockIdx.y), &before, &own);
            step0 = before;
            steps = own;
            out0 = static_cast<int64_t>(blockIdx.y) * p.m * p.out_stride;
        }
    }
    if (mrows > BM) mrows = BM;
    // the group's pairs; all groups turn as often, over nothing at the end
    const uint32_t turns = static_cast<uint32_t>(((steps + 1) / 2 + KG - 1) / KG);
    if constexpr (KG > 1) {
        const int64_t skip = 2 * static_cast<int64_t>(turns) * kg;
        step0 += skip < steps ? skip : steps;
        steps = skip < steps ? (steps - skip < 2 * turns ? steps - skip : 2 * turns) : 0;
    }
    const int64_t n0 = static_cast<int64_t>(ntile) * BN;
    const int64_t ncols = p.n - n0 < BN ? p.n - n0 : BN;

    // sources: the tile's rows from the first step on, up to the last row's end
    const uint32_t crow = static_cast<uint32_t>(p.steps) * (kPad / 2), srow = static_cast<uint32_t>(p.steps) * 4;
    const uint32_t c0 = static_cast<uint32_t>(step0) * (kPad / 2), s0 = static_cast<uint32_t>(step0) * 4;
    const uint8_t* ac = p.a + row0 * crow + c0;
    const uint8_t* asc = p.as + row0 * srow + s0;
    const uint8_t* bc = b + n0 * crow + c0;
    const uint8_t* bsc = bs + n0 * srow + s0;
    const uint32_t ace = static_cast<uint32_t>(mrows) * crow - c0, ase = static_cast<uint32_t>(mrows) * srow - s0;
    const uint32_t bce = static_cast<uint32_t>(ncols) * crow - c0, bse = static_cast<uint32_t>(ncols) * srow - s0;

    // a transfer covers 8 rows of codes, or 32 rows of scales
    constexpr int kMoves = (BM + BN) / 32 + 1;   // transfers of a wave for a pair
    const uint32_t cvoff = static_cast<uint32_t>(wave * 8 + (lane >> 3)) * crow +
                           static_cast<uint32_t>(((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) * 16);
    const uint32_t svoff = static_cast<uint32_t>(lane >> 1) * srow +
                           static_cast<uint32_t>(((lane & 1) ^ ((lane >> 4) & 1)) * 16);
    const uint32_t pairs = static_cast<uint32_t>((steps + 1) >> 1);
    // an odd last step has a pair of its own, whose second half is nobody's:
    // its lanes read behind the resource's end (a tile's rows end below 2^31)
    // and bring zeros
    const uint32_t odd = steps & 1 ? pairs - 1 : ~0u;
    const uint32_t cvoff_odd = cvoff | (((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) & 4 ? 0x80000000u : 0);
    // The transfers of the pair whose turn it is: where from (a resource each,
    // of no bytes behind the last pair), and where to.  The quarter of the
    // scales that is due comes with them (those of pairs 4 u .. with the pairs
    // 4 u - 3 .. 4 u).
    uint64_t pa = reinterpret_cast<uint64_t>(ac), pb = reinterpret_cast<uint64_t>(bc), ps;
    uint32_t ea = pairs > 0 ? ace : 0, eb = pairs > 0 ? bce : 0, es;
    uint32_t from = odd == 0 ? cvoff_odd : cvoff, to = lds0 + wave * 1024, sfrom, sto;
    // scale transfers of four pairs: BM / 32 of a's, then as many of b's
    static_assert(BM == BN, "a's and b's scales are told apart by a bit");
    const uint64_t asc0 = reinterpret_cast<uint64_t>(asc), bsc0 = reinterpret_cast<uint64_t>(bsc);
    auto scale_index = [&](uint32_t part) { return (part * 4 + wave) & ((BM + BN) / 32 - 1); };
    auto of_b = [&](uint32_t i) { return (i / (BM / 32)) & 1; };   // 0 or 1
    auto aim_scales = [&](uint32_t quad, uint32_t part, int step) {
        const uint32_t i = scale_index(part);
        if (step == 0) {
            sfrom = svoff + (i & (BM / 32 - 1)) * 32 * srow;
            asm volatile("" : "+v"(sfrom));
        } else if (step == 1) {
            sto = lds0 + 2 * kCodes + (quad & 1) * kScales + i * 1024;
            asm volatile("" : "+s"(sto));
        } else if (step == 2) {
            ps = (asc0 ^ ((asc0 ^ bsc0) & (uint64_t(0) - of_b(i)))) + quad * 32;
            asm volatile("" : "+s"(ps));
        } else {
            const uint32_t on = 0u - static_cast<uint32_t>(quad * 4 < pairs);
            es = ((ase ^ ((ase ^ bse) & (0u - of_b(i)))) - quad * 32) & on;
            asm volatile("" : "+s"(es));
        }
    };
    auto move_scales = [&]() { to_lds(resource(ps, es), sfrom, sto); };
    auto move = [&](int i) {
        if (i == kMoves - 1)
            move_scales();
        else if (i < BM / 32)
            to_lds(resource(pa, ea), from + i * 32 * crow, to + i * 4096);
        else
            to_lds(resource(pb, eb), from + (i - BM / 32) * 32 * crow, to + i * 4096);
    };
    // Turns to pair q in kAims steps of a few scalar instructions, which are
    // laid apart: a wave is alone on its SIMD, and more of them between two
    // matrix instructions than their 16 cycles hold would stop those.
    constexpr int kAims = 7;
    auto aim = [&](uint32_t q, int step) {
        asm volatile("" : "+s"(q));   // not to be computed earlier
        if (step == 0) {
            pa += 128;
            pb += 128;
            asm volatile("" : "+s"(pa));
            asm volatile("" : "+s"(pb));
        } else if (step == 1) {
            ea = q < pairs ? ea - 128 : 0;
            eb = q < pairs ? eb - 128 : 0;
            asm volatile("" : "+s"(ea));
            asm volatile("" : "+s"(eb));
        } else if (step == 2) {
            from = q == odd ? cvoff_odd : cvoff;
            asm volatile("" : "+v"(from));
            to = lds0 + (q & 1) * kCodes + wave * 1024;
            asm volatile("" : "+s"(to));
        } else {
            aim_scales((q + 3) >> 2, (q + 3) & 3, step - 3);
        }
    };

    // a lane's place in LDS: row r of a 16-row fragment, piece 4 (k-step) + g
    const int wm = wave >> 1, wn = wave & 1, shift = 8 * g;
    const uint32_t place[2] = {static_cast<uint32_t>(r * 128 + ((g ^ (r >> 1)) * 16)),
                               static_cast<uint32_t>(r * 128 + (((4 + g) ^ (r >> 1)) * 16))};
    uint32_t codes_at[2] = {place[0], place[1]};   // of the pair to be read
    uint32_t scales_at = 0;
    auto find_codes = [&](uint32_t q, int k) {
        codes_at[k] = place[k] + (q & 1) * kCodes;
        asm volatile("" : "+v"(codes_at[k]));
    };
    auto find_scales = [&](uint32_t q) {
        asm volatile("" : "+s"(q));
        scales_at = 2 * kCodes + ((q >> 2) & 1) * kScales + (q & 1) * 8 + r * 32 + ((((q >> 1) & 1) ^ ((r >> 3) & 1)) * 16);
        asm volatile("" : "+v"(scales_at));
    };
    f32x4 acc[WM][WN];
    i32x4 fa[2][WM], fb[2][WN];   // fragments by k-step of the pair
    u32x2 qa[WM], qb[WN];         // scale codes of a pair, four blocks a word
    int sa[2][WM], sb[2][WN];     // scale codes by k-step, the lane's own
    constexpr int kReads = WM + WN;
    // fragment x of k-step k of the pair that codes_at and scales_at name (a's
    // and b's in turn), and with the first k-step its scales
    auto read = [&](int k, int x) {
        const uint8_t *c = lds + codes_at[k], *w = lds + scales_at;
        const int i = x >> 1;
        if (x & 1) {
            fb[k][i] = *reinterpret_cast<const i32x4*>(c + BM * 128 + (wn * WN + i) * 2048);
            if (k == 0) qb[i] = *reinterpret_cast<const u32x2*>(w + BM * 32 + (wn * WN + i) * 512);
        } else {
            fa[k][i] = *reinterpret_cast<const i32x4*>(c + (wm * WM + i) * 2048);
            if (k == 0) qa[i] = *reinterpret_cast<const u32x2*>(w + (wm * WM + i) * 512);
        }
    };
    // The lane's scale code x (a's, then b's) of k-step k; width: 8, or 0 for
    // the step behind the last one (scales 2^-127, codes zero).
    auto take_scale = [&](int k, int x, uint32_t width) {
        if (x < WM)
            sa[k][x] = static_cast<int>(__builtin_amdgcn_ubfe(qa[x][k], shift, width));
        else
            sb[k][x - WM] = static_cast<int>(__builtin_amdgcn_ubfe(qb[x - WM][k], shift, width));
    };
    auto take_first = [&](uint32_t q, int x) { take_scale(0, x, KG == 1 || q < pairs ? 8 : 0); };
    // The products of k-step K; between them what next(x) starts.  The scale
    // codes are taken in the k-step before: a matrix instruction may not follow
    // within two of the one that makes its operand, and the compiler does not
    // see to that where the instruction is written as assembly.
    auto multiply = [&](auto kstep, auto next) {
        constexpr int K = decltype(kstep)::value;
        asm volatile("s_nop 1" ::: "memory");
        each<WM * WN>([&](auto index) {
            constexpr int x = decltype(index)::value, i = x / WN, j = x % WN;
            multiply_add(acc[i][j], fb[K][j], fa[K][i], sb[K][j], sa[K][i]);
            next(index);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 1>;
    constexpr int kProducts = WM * WN;
    static_assert(WM == WN, "reads take a's and b's fragments in turn");
    constexpr int kReadEvery = kProducts / kReads / 2 ? kProducts / kReads / 2 : 1;
    // transfers start within the first four fifths of a k-step (16384^3: 4.94
    // PFLOP/s, spread over three quarters of a pair 4.76)
    constexpr int kMoveEvery = 4 * kProducts / 5 / kMoves ? 4 * kProducts / 5 / kMoves : 1;
    constexpr int kEarly = kProducts / kMoveEvery < kMoves ? kProducts / kMoveEvery : kMoves;   // with the second k-step
    // behind the last transfer of the pair before (move kMoves - 1)
    constexpr int kFirstAim = kMoves * kMoveEvery - kProducts > 0 ? kMoves * kMoveEvery - kProducts : 0;
    constexpr int kAimEvery = (kProducts - kFirstAim) / (kAims + 2);   // 0: all behind the last product
    constexpr int kFindScales = kAimEvery ? kFirstAim + kAims * kAimEvery : kProducts - 1;
    constexpr int kFindCodes = kAimEvery ? kFindScales + kAimEvery : kProducts - 1;
    static_assert(kReadEvery * kReads <= kProducts && kMoveEvery >= 1, "spacing");

    auto zero = [&]() {
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) {
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                asm volatile("" : "+a"(acc[i][j]));
            }
    };
    if (turns == 0) zero();
    if (turns > 0) {
#pragma unroll
        for (int part = 0; part < 4; ++part) {
#pragma unroll
            for (int step = 0; step < 4; ++step) aim_scales(0, part, step);
            if (part < 3) move_scales();
        }
#pragma unroll
        for (int i = 0; i < kMoves; ++i) move(i);
#pragma unroll
        for (int i = 0; i < kAims; ++i) aim(1, i);
#pragma unroll
        for (int i = 0; i < kEarly; ++i) move(i);
        find_scales(0);
        zero();   // while they are on their way
        wait_transfers<kEarly>();
        block_barrier();
#pragma unroll
        for (int x = 0; x < kReads; ++x) read(0, x);
#pragma unroll
        for (int x = 0; x < kReads; ++x) take_first(0, x);
        settle_products();   // and behind acc's first values
        for (uint32_t q = 0; q < turns; ++q) {
            // The first k-step of pair q.  The last transfers of pair q + 1
            // start; then the aim turns to pair q + 2.
            multiply(First{}, [&](auto index) {
                constexpr int x = decltype(index)::value, y = kProducts + x, z = x - kFirstAim;
                if constexpr (x % kReadEvery == 0 && x / kReadEvery < kReads) read(1, x / kReadEvery);
                // the second k-step's scales, before the next pair's replace them
                if constexpr (x >= kProducts - kReads)
                    take_scale(1, x - (kProducts - kReads), q == odd || (KG > 1 && q >= pairs) ? 0 : 8);
                if constexpr (y % kMoveEvery == kMoveEvery - 1 && y / kMoveEvery < kMoves) move(y / kMoveEvery);
                if constexpr (kAimEvery > 0) {
                    if constexpr (z >= 0 && z % kAimEvery == 0 && z / kAimEvery < kAims) aim(q + 2, z / kAimEvery);
                } else if constexpr (x == kProducts - 1) {
                    each<kAims>([&](auto step) { aim(q + 2, decltype(step)::value); });
                }
                // and the reads to pair q + 1
                if constexpr (x == kFindCodes) find_codes(q + 1, 0);
                if constexpr (x == kFindScales) find_scales(q + 1);
            });
            // all waves hold the second k-step in registers, pair q + 1 is here
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            wait_transfers<0>();
            block_barrier();
            __builtin_amdgcn_sched_barrier(0);
            multiply(Second{}, [&](auto index) {
                constexpr int x = decltype(index)::value;
                if constexpr (x % kReadEvery == 0 && x / kReadEvery < kReads) read(0, x / kReadEvery);
                if constexpr (x % kMoveEvery == kMoveEvery - 1 && x / kMoveEvery < kMoves) move(x / kMoveEvery);
                // the next pair's first scales, read in this k-step
                if constexpr (kProducts >= 2 * kReads) {
                    if constexpr (x >= kProducts - kReads) take_first(q + 1, x - (kProducts - kReads));
                } else if constexpr (x == kProducts - 1) {
                    each<kReads>([&](auto y) { take_first(q + 1, decltype(y)::value); });
                }
                if constexpr (x == kProducts - 1) find_codes(q + 1, 1);
            });
        }
        wait_transfers<0>();   // none may arrive in what LDS holds next
        settle_products();
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) asm volatile("" : "+a"(acc[i][j]));   // read behind that
    }

    block_barrier();
    if constexpr (KG > 1) {
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j)
                    reinterpret_cast<f32x4*>(lds)[((wave * WM + i) * WN + j) * kWave + lane] = acc[i][j];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        block_barrier();
        if (kg > 0) return;
#pragma unroll
        for (int k = 1; k < KG; ++k)
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j)
                    acc[i][j] += reinterpret_cast<const f32x4*>(lds + k * kGroup)[((wave * WM + i) * WN + j) * kWave + lane];
    }
    // Result (i, j, e) of a lane is row 16 i + r, column 16 j + 4 g + e.  They
    // pass through the wave's part of LDS (the codes are done with), so that
    // whole pieces of rows go out together.
    constexpr int kSize = DT == kF32 ? 4 : 2, kRow = 16 * WN * kSize, kPitch = kRow + 16, kPieces = kRow / 16;
    constexpr int kPart = kGroup / 4;
    constexpr int kFrags = kPart / (16 * kPitch) < WM ? (kPart / (16 * kPitch) < WM / 2 ? WM / 4 : WM / 2) : WM;
    static_assert(kFrags * 16 * kPitch <= kPart && WM % kFrags == 0, "room in LDS");
    uint8_t* const mine = lds + wave * kPart;
    const int64_t left = ncols - wn * (16 * WN);
    constexpr int kTurn = kWave / kPieces;   // rows that a wave stores at once
    const int row = lane / kPieces, n = (lane % kPieces) * (16 / kSize);
#pragma unroll
    for (int f = 0; f < WM; f += kFrags) {
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) {
                const f32x4 v = acc[f + i][j];
                uint8_t* to = mine + (16 * i + r) * kPitch + (16 * j + 4 * g) * kSize;
                if constexpr (DT == kF32)
                    *reinterpret_cast<f32x4*>(to) = v;
                else
                    *reinterpret_cast<u32x2*>(to) = DT == kBF16
                                                        ? u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}
                                                        : u32x2{f16_pair(v[0], v[1]), f16_pair(v[2], v[3])};
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const int m0 = (wm * WM + f) * 16;
        const int have = mrows - m0 < 16 * kFrags ? static_cast<int>(mrows - m0) : 16 * kFrags;
        const uint8_t* from = mine + row * kPitch + n * kSize;
        uint8_t* out = static_cast<uint8_t*>(p.out) +
                       (out0 + (row0 + m0 + row) * p.out_stride + n0 + wn * (16 * WN) + n) * kSize;
        const int64_t step = kTurn * p.out_stride * kSize;
        if (p.wide && n + 16 / kSize <= left) {
            if (p.past_caches) {
#pragma unroll 8
                for (int y = row; y < have; y += kTurn, from += kTurn * kPitch, out += step)
                    __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(from), reinterpret_cast<u32x4*>(out));
            } else {
#pragma unroll 8
                for (int y = row; y < have; y += kTurn, from += kTurn * kPitch, out += step)
                    *reinterpret_cast<u32x4*>(out) = *reinterpret_cast<const u32x4*>(from);
            }
        } else if (n < left) {
            const int some = left - n < 16 / kSize ? static_cast<int>(left - n) : 16 / kSize;
#pragma unroll 1
            for (int y = row; y < have; y += kTurn, from += kTurn * kPitch, out += step)
#pragma unroll 1
                for (int e = 0; e < some; ++e) {
                    if constexpr (DT == kF32)
                        reinterpret_cast<uint32_t*>(out)[e] = reinterpret_cast<const uint32_t*>(from)[e];
                    else
                        reinterpret_cast<uint16_t*>(out)[e] = reinterpret_cast<const uint16_t*>(from)[e];
                }
        }
        if (f + kFrags < WM) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

}  // namespace

const void* quant_rows_kernel(int dtype)
{
    const void* fns[3] = {reinterpret_cast<const void*>(&k_quant_rows<kF32>),
                          reinterpret_cast<const void*>(&k_quant_rows<kF16>),
                          reinterpret_cast<const void*>(&k_quant_rows<kBF16>)};
    return fns[dtype];
}

const void* quant_tile_kernel(int dtype)
{
    const void* fns[3] = {reinterpret_cast<const void*>(&k_quant_tile<kF32>),
                          reinterpret_cast<const void*>(&k_quant_tile<kF16>),
                          reinterpret_cast<const void*>(&k_quant_tile<kBF16>)};
    return fns[dtype];
}

const void* dequant_kernel(int dtype)
{
    const void* fns[3] = {reinterpret_cast<const void*>(&k_dequant<kF32>),
                          reinterpret_cast<const void*>(&k_dequant<kF16>),
                          reinterpret_cast<const void*>(&k_dequant<kBF16>)};
    return fns[dtype];
}

template <int G, int W, int KG>
TileKernel tile_of_type(int dtype)
{
    const void* fns[3] = {reinterpret_cast<const void*>(&k_matmul_tile<kF32, G, W, W, KG>),
                          reinterpret_cast<const void*>(&k_matmul_tile<kF16, G, W, W, KG>),
                          reinterpret_cast<const void*>(&k_matmul_tile<kBF16, G, W, W, KG>)};
    return {fns[dtype], 32 * W, 256 * KG};
}

template <int G>
TileKernel tile_of_shape(int dtype, int tile, bool shared)
{
    return tile == 256   ? tile_of_type<G, 8, 1>(dtype)
           : tile == 128 ? tile_of_type<G, 4, 1>(dtype)
           : shared      ? tile_of_type<G, 2, 2>(dtype)
                         : tile_of_type<G, 2, 1>(dtype);
}

TileKernel matmul_tile_kernel(int out_dtype, int grouping, int tile, bool shared)
{
    return grouping == kPlain    ? tile_of_shape<kPlain>(out_dtype, tile, shared)
           : grouping == kByRows ? tile_of_shape<kByRows>(out_dtype, tile, shared)
                                 : tile_of_shape<kByContraction>(out_dtype, tile, shared);
}

template <int XT, int G>
FewKernel few_of(int cols)
{
    if (cols == 16) return {reinterpret_cast<const void*>(&k_matmul_few<XT, G, 1, 8, 2>), 16, 8};
    return {reinterpret_cast<const void*>(&k_matmul_few<XT, G, 4, 4, 1>), 64, 4};
}

template <int G>
FewKernel few_of_type(int x_dtype, int cols)
{
    return x_dtype == kF32    ? few_of<kF32, G>(cols)
           : x_dtype == kF16  ? few_of<kF16, G>(cols)
           : x_dtype == kBF16 ? few_of<kBF16, G>(cols)
                              : few_of<kHeld, G>(cols);
}

FewKernel matmul_few_kernel(int x_dtype, int grouping, int cols)
{
    return grouping == kPlain ? few_of_type<kPlain>(x_dtype, cols) : few_of_type<kByRows>(x_dtype, cols);
}

}  // namespace mx4
