// experts.h -- declarations shared by the kernels and the host code of the
// operators around experts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace experts {

constexpr int kWave = 64;

enum Dtype { kF32 = 0, kF16 = 1, kBF16 = 2 };
enum Scores { kSoftmax = 0, kSigmoid = 1 };

struct TopkArgs {
    const void* logits;
    const float* bias;      // nullptr: none
    const uint8_t* mask;    // nullptr: every token chooses
    float* weights;
    int32_t* ids;
    int64_t tokens, row_stride;
    int32_t experts, k, groups, top_groups;
    int32_t scores, best_two, renormalize;
    float scale;
    int32_t wide, bias_wide;   // loads of four neighbours are aligned
    int32_t exact;             // every token's choice in 64 bits
};

struct TopkBackwardArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    void* dlogits;
    int64_t tokens, row_stride;
    int32_t experts, k, scores, renormalize;
    float scale;
    int32_t wide, dense_wide;   // four neighbours of a row of logits, of dlogits are aligned
};

struct OrderArgs {
    const int32_t* ids;
    int32_t* offsets;
    int32_t* slot_of_row;
    int32_t* row_of_slot;
    int32_t* counts;        // [blocks][bins]
    int64_t slots, chunk;   // slots of a block
    int32_t experts, blocks;
    int32_t bins;           // experts and those of none, rounded up to 4
};

// Rows of x or y.  `cols` and the strides count elements; for the dispatch, which
// copies, 16-byte pieces where rows allow them.
struct RowsArgs {
    const void* x;          // dispatch: x; combine: y; its gradient: dout
    const void* y;          // gradient: y
    const void* add;
    const float* weights;
    const int32_t* slot_of_row;
    const int32_t* row_of_slot;
    void* out;              // gradient: dy
    float* dweights;
    int64_t tokens, cols, x_stride, y_stride, add_stride, out_stride;
    int32_t k, zero_rest;
    int32_t past_caches;    // the rows are too many to stay in the last cache
};

// 4-bit weights; experts 0: one matrix, no groups of rows.
struct Int4Args {
    const void* x;
    const uint8_t* codes;
    const void* scales;
    const void* zeros;      // nullptr: 8
    void* out;
    const int32_t* offsets;
    int64_t m, n, k, x_stride, out_stride;
    int32_t group, experts, zero_rest, out_dtype, scale_dtype;
    int32_t out_wide;       // dequantisation: 16-byte stores are allowed
    int32_t tiles;          // of rows of weights a block, where x is held
};

struct Int4QuantArgs {
    const void* x;
    uint8_t* codes;
    void* scales;
    void* zeros;
    int64_t rows, k, row_stride;
    int32_t group, scale_dtype;
    int32_t wide;           // 16-byte loads of x are allowed
    int32_t lanes_log2;     // of a group
};

// `tokens` a wave
struct TopkKernel {
    const void* fn;
    int tokens;
};
TopkKernel topk_kernel(int dtype, int32_t experts, int32_t k, int32_t groups);
TopkKernel topk_backward_kernel(int dtype, int32_t experts, int32_t k);
const void* order_count_kernel();
const void* order_place_kernel();
const void* dispatch_kernel(int bytes, bool wide);
const void* combine_kernel(int dtype, bool wide);
const void* combine_backward_kernel(int dtype, bool wide);
const void* balance_kernel();
const void* int4_quantize_kernel(int dtype);
const void* int4_dequantize_kernel(int dtype);

// scales: groups of columns in 128 (1, 2 or 4); steps: of 128 columns in k; tiles:
// of 16 rows of weights and 16 of x, about; half: scales have 16 bits.  A block
// takes 16 `width` columns of results, `tiles` times with x held.
struct Int4Kernel {
    const void* fn;
    int waves;
    int width;
    bool held;
};
Int4Kernel int4_matmul_kernel(int dtype, int scales, bool grouped, int64_t steps, int64_t tiles, bool half);

constexpr int kTopkWaves = 4;          // of a block
constexpr int kOrderThreads = 512;
constexpr int kOrderAlone = 4096;      // slots that one block takes by itself
constexpr int kOrderChunk = 2048;      // slots of a block, at least
constexpr int kOrderBlocks = 256;      // at most
constexpr int kRowThreads = 512;       // at most: a row's pieces, in whole waves
constexpr int kInt4Threads = 256;

}  // namespace experts
