// call.hpp -- what the C entry points of the operators' libraries share (host
// side): the message of the last failure, argument checks and launches.  Each
// library has a copy of its own.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/optimizer_update.h"

namespace {

thread_local char g_error[512] = "";

[[maybe_unused]] __attribute__((format(printf, 2, 3))) int fail(int status, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return status;
}

[[maybe_unused]] int hip_fail(hipError_t e, const char* what) { return fail(OU_EHIP, "%s: %s", what, hipGetErrorString(e)); }

constexpr int kMaxDevices = 64;
std::atomic<int> g_arch[kMaxDevices];   // 0 unknown, 1 gfx950, 2 another

// OU_OK if the current device is a gfx950 (looked up once per device).
[[maybe_unused]] int check_device()
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(OU_EUNSUPPORTED, "no HIP device: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(OU_EUNSUPPORTED, "device %d", dev);
    int a = g_arch[dev].load(std::memory_order_relaxed);
    if (!a) {
        hipDeviceProp_t p;
        e = hipGetDeviceProperties(&p, dev);
        if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
        a = std::strncmp(p.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_arch[dev].store(a, std::memory_order_relaxed);
    }
    return a == 1 ? OU_OK : fail(OU_EUNSUPPORTED, "device %d is not a gfx950", dev);
}

// Largest extent of any axis, and of any product of axes in bytes: every
// address and count below stays far inside 64 bits.
constexpr int64_t kMaxAxis = int64_t(1) << 31;
constexpr int64_t kMaxBytes = int64_t(1) << 46;
constexpr int32_t kMaxBatch = 65535;      // second axis of a grid

[[maybe_unused]] int elem_bytes(int dtype) { return dtype == OU_F32 ? 4 : 2; }
[[maybe_unused]] bool valid_dtype(int dtype) { return dtype == OU_F32 || dtype == OU_F16 || dtype == OU_BF16; }
[[maybe_unused]] int64_t cut(int64_t n, int64_t d) { return (n + d - 1) / d; }

[[maybe_unused]] int check_axis(int64_t n, const char* what)
{
    if (n < 0 || n > kMaxAxis) return fail(OU_EINVAL, "%s = %lld is out of range", what, static_cast<long long>(n));
    return OU_OK;
}

// A buffer of a call; check() tests all of them.
struct Buffer {
    const char* name;
    const void* p;
    double bytes;      // extent, as a double so that no product wraps
    unsigned align;
    bool written;
};

[[maybe_unused]] int check_buffers(const Buffer* b, int n)
{
    for (int i = 0; i < n; ++i) {
        if (b[i].bytes <= 0) continue;
        if (!b[i].p) return fail(OU_EINVAL, "%s is null", b[i].name);
        if (b[i].bytes > static_cast<double>(kMaxBytes)) return fail(OU_EINVAL, "%s is too large", b[i].name);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(b[i].p);
        if (lo % b[i].align) return fail(OU_EALIGN, "%s is not %u-byte aligned", b[i].name, b[i].align);
        if (lo + static_cast<uintptr_t>(b[i].bytes) < lo) return fail(OU_EINVAL, "%s wraps", b[i].name);
    }
    for (int i = 0; i < n; ++i) {
        if (!b[i].written || b[i].bytes <= 0) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(b[i].p), hi = lo + static_cast<uintptr_t>(b[i].bytes);
        for (int j = 0; j < n; ++j) {
            if (j == i || b[j].bytes <= 0) continue;
            const uintptr_t lj = reinterpret_cast<uintptr_t>(b[j].p), hj = lj + static_cast<uintptr_t>(b[j].bytes);
            if (lo < hj && lj < hi) return fail(OU_EOVERLAP, "%s overlaps %s", b[i].name, b[j].name);
        }
    }
    return OU_OK;
}

// Bytes of `rows` rows of `cols` elements, `stride` elements apart.
[[maybe_unused]] double extent(int64_t rows, int64_t cols, int64_t stride, int bytes)
{
    if (rows == 0 || cols == 0) return 0;
    return (static_cast<double>(rows - 1) * static_cast<double>(stride) + static_cast<double>(cols)) * bytes;
}

struct Launch {
    const void* fn;
    int64_t gx, gy;
    int threads;
    const char* what;
    int64_t lds;
};

// A grid's threads along an axis are counted in 32 bits.
[[maybe_unused]] int check_grid(const Launch& l)
{
    if (l.gx > INT32_MAX || l.gx * l.threads > UINT32_MAX || l.gy > kMaxBatch)
        return fail(OU_EINVAL, "%s: too many tiles", l.what);
    return OU_OK;
}

[[maybe_unused]] int launch(const Launch& l, void** args, void* stream)
{
    if (int st = check_grid(l)) return st;
    if (int st = check_device()) return st;
    const hipError_t e = hipLaunchKernel(l.fn, dim3(static_cast<unsigned>(l.gx), static_cast<unsigned>(l.gy)),
                                         dim3(static_cast<unsigned>(l.threads)), args, static_cast<size_t>(l.lds),
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? OU_OK : hip_fail(e, l.what);
}

[[maybe_unused]] bool wide_rows(const void* p, int64_t stride, int64_t batch_stride, int bytes, int align)
{
    return reinterpret_cast<uintptr_t>(p) % align == 0 && (stride * bytes) % align == 0 &&
           (batch_stride * bytes) % align == 0;
}

[[maybe_unused]] int check_groups(const int32_t* offsets, int32_t groups, int64_t rows)
{
    if (rows > (int64_t(1) << 28)) return fail(OU_EINVAL, "%lld rows by groups: 2^28 at most", (long long)rows);
    if (groups < 0 || groups > kMaxBatch) return fail(OU_EINVAL, "groups = %d is out of range", groups);
    if (!offsets) return fail(OU_EINVAL, "offsets is null");
    if (reinterpret_cast<uintptr_t>(offsets) % 4) return fail(OU_EALIGN, "offsets is not 4-byte aligned");
    return OU_OK;
}

}  // namespace
