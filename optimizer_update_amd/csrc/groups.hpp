// groups.hpp -- ragged groups of rows (device): which group a unit of rows is
// of, from offsets in device memory.  Shared by the products by expert.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace groups {
namespace {

constexpr int kWave = 64;

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

}  // namespace
}  // namespace groups
