// mx4.h -- declarations shared by the kernels and the host code of the
// microscaled 4-bit operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx4 {

constexpr int kWave = 64;
constexpr int kBlock = 32;   // values that share one scale
constexpr int kPad = 128;    // columns of a held matrix are padded to this
constexpr int kScaleNaN = 255;

enum Dtype { kF32 = 0, kF16 = 1, kBF16 = 2, kHeld = 3 };   // kHeld: 4-bit codes and scales

// Quantisation of x [batch][rows][cols] (element strides given) along its
// columns (codes/scales, nullptr: not wanted) and along its rows
// (codes_t/scales_t, nullptr: not wanted).  pcols, prows: cols and rows
// padded to kPad.  With offsets the row axis is cut into groups
// [offsets[e], offsets[e+1]), each padded to kPad by itself, and prows is
// the capacity of the padded axis.
struct QuantArgs {
    const void* x;
    uint8_t* codes;
    uint8_t* scales;
    uint8_t* codes_t;
    uint8_t* scales_t;
    int64_t rows, cols, row_stride, batch_stride;
    int64_t pcols, prows;
    const int32_t* offsets;
    int32_t groups;
    int32_t wide;   // 16-byte loads of whole octets of x are allowed
};

// out [rows][cols] = the values of codes [rows][pcols / 2].
struct DequantArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    void* out;
    int64_t rows, cols, pcols, row_stride;
    int32_t wide;   // 16-byte stores of whole octets are allowed
};

// out[m][n] = sum_k a[m][k] b[n][k].  Plain: a has m rows, b n rows, steps
// k-steps of 128.  Grouped by rows: rows [offsets[e], offsets[e+1]) of a
// meet b's matrix e (n rows each).  Grouped by the contraction: out [e][m][n]
// contracts the padded columns of group e (QuantArgs) of both.
struct MatmulArgs {
    const uint8_t* a;
    const uint8_t* as;
    const uint8_t* b;
    const uint8_t* bs;
    void* out;
    int64_t m, n, out_stride;
    int64_t units, n_tiles;   // tiles along m (plain, by contraction) and n
    int64_t steps;            // k-steps of a row of a and b as stored
    const int32_t* offsets;
    int64_t rows;             // grouped: rows that offsets may point to
    int32_t groups;
    int32_t zero_rest;        // grouped by rows: rows of no group become 0
    int32_t wide;             // stores of 4 neighbouring results (tiles: of 16 bytes) are aligned
    int32_t past_caches;      // tiles: out is too large to stay in the last cache
    int32_t out_dtype;        // k_matmul_few
    // the left matrix as values (k_matmul_few)
    const void* x;
    int64_t x_stride, k;
    int32_t x_dtype;
    int32_t few_rows;         // rows that k_matmul_few has room for
    int32_t x_wide;           // 16-byte loads of whole octets of x are allowed
};

enum Grouping { kPlain = 0, kByRows = 1, kByContraction = 2 };

const void* quant_rows_kernel(int dtype);
const void* quant_tile_kernel(int dtype);
const void* dequant_kernel(int dtype);
// tile: rows and columns of a block's tile, 256, 128 or 64; shared: the k-steps
// of a 64-tile by two groups of waves.
struct TileKernel {
    const void* fn;
    int tile, threads;
};
TileKernel matmul_tile_kernel(int out_dtype, int grouping, int tile, bool shared);

// Products of up to 16 rows (by groups: in units of 16): 16 or 64 columns a
// block of `waves` waves, with few_lds() bytes of dynamic LDS.
struct FewKernel {
    const void* fn;
    int cols, waves;
};
inline int64_t few_lds(int64_t rows, int64_t steps, int cols, int waves)   // rows: 0 for a held left matrix
{
    return rows * (steps * 64 + 16) + (rows * (steps * 4 + 4) + 15) / 16 * 16 + static_cast<int64_t>(waves) * cols * 64;
}
FewKernel matmul_few_kernel(int x_dtype, int grouping, int cols);

constexpr int kQuantThreads = 256;
constexpr int kQuantUnits = 4;      // units of 128 columns per 16 lanes of k_quant_rows
constexpr int kQuantTile = 128;     // rows and columns of a tile of k_quant_tile

}  // namespace mx4
