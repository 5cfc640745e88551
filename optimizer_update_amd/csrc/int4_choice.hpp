// int4_choice.hpp -- which kernel takes a product with 4-bit group-scaled weights,
// by sizes and types alone (host code, no device needed).
#pragma once

#include <stdint.h>

namespace experts {

// held: k_int4_tiles, x in registers over a run of tiles; else k_int4_matmul.
// tiles: of 16 rows of weights a block (held: and turn); waves: of a block;
// steps: of 128 columns a wave holds.
struct Int4Choice {
    bool held;
    int tiles, waves, steps;
};

// Tiles of 16 rows of weights by 16 of x, about: experts that have rows are no
// more than there are rows.
constexpr int64_t int4_tiles(int64_t m, int64_t n, bool grouped, int64_t experts)
{
    return (n + 15) / 16 * (grouped ? (m < experts ? m : experts) : (m + 15) / 16);
}

// Groups of columns in a step of 128.
constexpr int int4_scales(int32_t group) { return group % 128 == 0 ? 1 : group % 64 == 0 ? 2 : 4; }

// x is held where tiles are many and the waves' registers of it are filled (and
// scales have 16 bits).  8 steps: 2001 tiles 11.8 us, streamed 13.6, but 1024 tiles
// 8.2 and 6.2, and 6 steps, 6144 tiles 25.9 and 23.9.  16 steps: 16384 tiles 77 and
// 88, 8000 tiles 45 and 50, 4096 tiles 20.2 and 19.1, 2000 tiles 16.5 and 15.6, 12
// steps 78 and 73.  Streamed binary32 is taken apart for every tile, which small
// groups of columns leave no time for: 16 steps, 16384 tiles, groups of 64, 125 and
// 183 us, of 128 149 and 126 (codes as they are; less 7.5, 129 held for groups of
// 64 and 125 streamed for 128).
constexpr bool int4_holds(bool f32, int scales, int64_t steps, int64_t tiles)
{
    if (f32 && scales > 1) return steps <= 16 && tiles >= 1536;
    return steps > 6 && steps <= 8 ? tiles >= 1536 : !f32 && steps > 12 && steps <= 16 && tiles >= 6144;
}

// scales: int4_scales(); half: scales have 16 bits; steps: of 128 columns in k.
constexpr Int4Choice int4_choice(bool f32, int scales, bool half, int64_t steps, int64_t tiles)
{
    if (half && int4_holds(f32, scales, steps, tiles)) {
        // 2001 tiles of 8 steps: eight waves of one 10.5 us by pairs of tiles, 11.2 by
        // single ones, four waves of two 11.6 and 12.8.  16 steps, 64 experts: four
        // waves of four 80 us, by pairs 95, eight of two 96, by pairs 82.
        if (steps <= 8) return {true, 2, 8, 1};
        return f32 ? Int4Choice{true, 1, 8, 2} : Int4Choice{true, 1, 4, 4};
    }
    // x streams past 4 tiles of rows of weights from 896 tiles on, past 2 from 512.  One
    // row, k = 4096, groups of 128: 256 tiles 5.6 us by one, 7.3 by two; 896 tiles 13.8,
    // 11.5, 11.7 by four; 16 rows 23.0, 16.7, 13.8; 512 tiles, k = 8192, 23.1, 17.2,
    // 23.5; 2000 tiles 43, 30, 25.8.  Groups of 32, 2000 tiles of 16 rows: 43.7 by two,
    // 40.1 by four, one row 34.1 and 37.8.  Four waves do by four what eight take 10 %
    // longer for, and by two where smaller groups take the registers for a second block
    // of eight: 768 tiles, k = 2560, groups of 64, 10.3 and 12.5.  Binary32 with small
    // groups by two at most: the sums of four leave one wave a SIMD.
    if ((!f32 || scales == 1) && tiles >= 896) return {false, 4, 4, 0};
    if (tiles >= 512) return {false, 2, scales == 1 ? 8 : 4, 0};
    return {false, 1, 8, 0};
}

}  // namespace experts
