// values.hpp -- the storage types of the operators around experts (device):
// one value or a 16-byte piece of a row, to and from binary32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "experts.h"

namespace experts {
namespace {

using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

template <int DT>
struct Value;

template <>
struct Value<kF32> {
    using Elem = float;
    static constexpr int kBytes = 4;
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ float from_float(float x) { return x; }
    static __device__ __forceinline__ float load(const float* p, int64_t i) { return p[i]; }
    static __device__ __forceinline__ void store(float* p, int64_t i, float x) { p[i] = x; }
    // four neighbours, aligned
    static __device__ __forceinline__ void load4(const float* p, float* out)
    {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t d = w[j];   // a bit cast of the vector's element itself takes its first one
            out[j] = __builtin_bit_cast(float, d);
        }
    }
    static __device__ __forceinline__ void store4(float* p, const float* v)
    {
        *reinterpret_cast<u32x4*>(p) = u32x4{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                                             __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
    }
};
template <>
struct Value<kF16> {
    using Elem = uint16_t;
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ float to_float(uint16_t x) { return static_cast<float>(__builtin_bit_cast(_Float16, x)); }
    static __device__ __forceinline__ uint16_t from_float(float x) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x)); }
    static __device__ __forceinline__ float load(const uint16_t* p, int64_t i) { return to_float(p[i]); }
    static __device__ __forceinline__ void store(uint16_t* p, int64_t i, float x) { p[i] = from_float(x); }
    static __device__ __forceinline__ void load4(const uint16_t* p, float* out)
    {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t d = w[j];
            out[2 * j] = to_float(static_cast<uint16_t>(d));
            out[2 * j + 1] = to_float(static_cast<uint16_t>(d >> 16));
        }
    }
    static __device__ __forceinline__ void store4(uint16_t* p, const float* v)
    {
        *reinterpret_cast<u32x2*>(p) = u32x2{from_float(v[0]) | static_cast<uint32_t>(from_float(v[1])) << 16,
                                             from_float(v[2]) | static_cast<uint32_t>(from_float(v[3])) << 16};
    }
};
template <>
struct Value<kBF16> {
    using Elem = uint16_t;
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ float to_float(uint16_t x) { return __builtin_bit_cast(float, static_cast<uint32_t>(x) << 16); }
    static __device__ __forceinline__ uint16_t from_float(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
    static __device__ __forceinline__ float load(const uint16_t* p, int64_t i) { return to_float(p[i]); }
    static __device__ __forceinline__ void store(uint16_t* p, int64_t i, float x) { p[i] = from_float(x); }
    static __device__ __forceinline__ void load4(const uint16_t* p, float* out)
    {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t d = w[j];
            out[2 * j] = to_float(static_cast<uint16_t>(d));
            out[2 * j + 1] = to_float(static_cast<uint16_t>(d >> 16));
        }
    }
    static __device__ __forceinline__ void store4(uint16_t* p, const float* v)
    {
        *reinterpret_cast<u32x2*>(p) = u32x2{from_float(v[0]) | static_cast<uint32_t>(from_float(v[1])) << 16,
                                             from_float(v[2]) | static_cast<uint32_t>(from_float(v[3])) << 16};
    }
};

// The value of bits that were loaded earlier, of a type that is known at run time.
__device__ __forceinline__ float bits_value(uint32_t b, int dtype)
{
    return dtype == kF32   ? __builtin_bit_cast(float, b)
           : dtype == kF16 ? Value<kF16>::to_float(static_cast<uint16_t>(b))
                           : Value<kBF16>::to_float(static_cast<uint16_t>(b));
}

// The value at `i` of an array whose type is known at run time.
__device__ __forceinline__ float load_value(const void* p, int64_t i, int dtype)
{
    if (dtype == kF32) return static_cast<const float*>(p)[i];
    const uint16_t v = static_cast<const uint16_t*>(p)[i];
    return dtype == kF16 ? Value<kF16>::to_float(v) : Value<kBF16>::to_float(v);
}
__device__ __forceinline__ void store_value(void* p, int64_t i, float x, int dtype)
{
    if (dtype == kF32)
        static_cast<float*>(p)[i] = x;
    else
        static_cast<uint16_t*>(p)[i] = dtype == kF16 ? Value<kF16>::from_float(x) : Value<kBF16>::from_float(x);
}

// Neighbouring values of a row that one lane moves: 16 bytes where rows allow
// it, single values elsewhere.
template <int DT, bool WIDE>
struct Piece {
    using V = Value<DT>;
    using Elem = typename V::Elem;
    static constexpr int kValues = WIDE ? 16 / V::kBytes : 1;

    using Raw = std::conditional_t<WIDE, u32x4, Elem>;

    static __device__ __forceinline__ Raw fetch(const void* p, int64_t i)
    {
        return *reinterpret_cast<const Raw*>(static_cast<const Elem*>(p) + i);
    }
    // read once: past the caches
    static __device__ __forceinline__ Raw fetch_once(const void* p, int64_t i)
    {
        return __builtin_nontemporal_load(reinterpret_cast<const Raw*>(static_cast<const Elem*>(p) + i));
    }
    static __device__ __forceinline__ void load(const void* p, int64_t i, float* out) { unpack(fetch(p, i), out); }
    template <class R = Raw, std::enable_if_t<std::is_same_v<R, Elem>, int> = 0>
    static __device__ __forceinline__ void unpack(R x, float* out)
    {
        out[0] = V::to_float(x);
    }
    template <class R = Raw, std::enable_if_t<std::is_same_v<R, u32x4>, int> = 0>
    static __device__ __forceinline__ void unpack(R w, float* out)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t d = w[j];   // a bit cast of the vector's element itself takes its first one
            if constexpr (DT == kF32) {
                out[j] = __builtin_bit_cast(float, d);
            } else {
                out[2 * j] = V::to_float(static_cast<uint16_t>(d));
                out[2 * j + 1] = V::to_float(static_cast<uint16_t>(d >> 16));
            }
        }
    }
    static __device__ __forceinline__ Raw pack(const float* v)
    {
        if constexpr (!WIDE) {
            return V::from_float(v[0]);
        } else {
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DT == kF32)
                    w[j] = __builtin_bit_cast(uint32_t, v[j]);
                else
                    w[j] = static_cast<uint32_t>(V::from_float(v[2 * j])) | static_cast<uint32_t>(V::from_float(v[2 * j + 1])) << 16;
            }
            return w;
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float* v, bool past_caches)
    {
        Raw* const q = reinterpret_cast<Raw*>(static_cast<Elem*>(p) + i);
        if (past_caches)
            __builtin_nontemporal_store(pack(v), q);
        else
            *q = pack(v);
    }
};

}  // namespace
}  // namespace experts
