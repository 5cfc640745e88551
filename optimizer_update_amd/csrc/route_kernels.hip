// route_kernels.hip -- routing to experts (device): scores and choice of the
// experts of a token, their weights and the gradients, the order of rows by
// expert, the dispatch of rows and their weighted combination.
#include <type_traits>

#include "experts.h"
#include "values.hpp"

#pragma clang fp contract(off)

namespace experts {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 64;

using i32x4 = int32_t __attribute__((ext_vector_type(4)));

// What lanes of a wave wrote to LDS is seen by the others behind this.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
    return x;
}
__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int s = 32; s; s >>= 1) x = fmaxf(x, __shfl_xor(x, s));
    return x;
}

// ---- the choice ---------------------------------------------------------------

// Whole numbers in the order of the values: NaN above all, -0 as 0; what is
// absent is 0, below everything.
__device__ __forceinline__ uint64_t order_key(double x)
{
    if (x != x) return ~uint64_t(0);
    const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
    return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}

__device__ __forceinline__ double key_value(uint64_t k)
{
    if (k == ~uint64_t(0)) return __builtin_nan("");
    return __builtin_bit_cast(double, k >> 63 ? k ^ (uint64_t(1) << 63) : ~k);
}

// Larger and smaller of three without the quieting of signalling NaNs that
// fmaxf() adds for every operand (rows with a NaN are seen by their sum).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c)
{
    float r;
    asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Reductions over L neighbouring lanes (16, 32 or 64), the same answer in all
// of them.
template <int L, class F>
__device__ __forceinline__ uint32_t reduce_lanes(uint32_t x, F f)
{
    x = f(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xf, 0xf, true)));    // lane ^ 1
    x = f(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xf, 0xf, true)));    // lane ^ 2
    x = f(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x141, 0xf, 0xf, true)));   // mirrored 8
    x = f(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x140, 0xf, 0xf, true)));   // mirrored 16
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        const uint32_t u = r[0], v = r[1];
        x = f(u, v);
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        const uint32_t u = r[0], v = r[1];
        x = f(u, v);
    }
    return x;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_min_u32(uint32_t x)
{
    return reduce_lanes<L>(x, [](uint32_t u, uint32_t v) { return u < v ? u : v; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float x)
{
    return __builtin_bit_cast(float, reduce_lanes<L>(__builtin_bit_cast(uint32_t, x), [](uint32_t u, uint32_t v) {
        return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, u), __builtin_bit_cast(float, v)));
    }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x)
{
    return __builtin_bit_cast(float, reduce_lanes<L>(__builtin_bit_cast(uint32_t, x), [](uint32_t u, uint32_t v) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) + __builtin_bit_cast(float, v));
    }));
}

// The choice of one token in 64 bits, by a whole wave: the choice `lane` in
// each lane (-1: none).  keys: LDS for one of every expert.
template <int DT>
__device__ int choose_exact(const TopkArgs& p, int64_t token, int lane, uint64_t* keys)
{
    constexpr float kInf = __builtin_inff();
    const typename Value<DT>::Elem* x = static_cast<const typename Value<DT>::Elem*>(p.logits) + token * p.row_stride;
    const bool by_logit = !p.bias && (p.groups == 1 || !p.best_two);
    float top = -kInf;
    double total = 0;
    if (p.scores == kSoftmax && !by_logit) {
        for (int e = lane; e < p.experts; e += kWave) top = fmaxf(top, Value<DT>::load(x, e));
        top = wave_max(top);
        for (int e = lane; e < p.experts; e += kWave) {
            const float v = Value<DT>::load(x, e);
            if (v != -kInf) total += exp(static_cast<double>(v) - top);
        }
#pragma unroll
        for (int s = 32; s; s >>= 1) total += __shfl_xor(total, s);
    }
    for (int e = lane; e < p.experts; e += kWave) {
        const float v = Value<DT>::load(x, e);
        double c = v;
        if (!by_logit) {
            c = p.scores == kSoftmax ? exp(c - top) / total : 1 / (1 + exp(-c));
            if (p.bias) c += p.bias[e];
        }
        keys[e] = v == -kInf ? 0 : order_key(c);
    }
    wave_sync();
    if (p.groups > 1) {
        const int size = p.experts / p.groups;
        uint64_t mine = 0;
        if (lane < p.groups) {
            uint64_t a = 0, b = 0;
            for (int i = 0; i < size; ++i) {
                const uint64_t c = keys[lane * size + i];
                if (c > a) {
                    b = a;
                    a = c;
                } else if (c > b) {
                    b = c;
                }
            }
            mine = !p.best_two || !b ? a : order_key(key_value(a) + key_value(b));
        }
        int ahead = 0;
        for (int g = 0; g < p.groups; ++g) {
            const uint64_t other = __shfl(mine, g);
            ahead += other > mine || (other == mine && g < lane);
        }
        if (lane < p.groups && ahead >= p.top_groups)
            for (int i = 0; i < size; ++i) keys[lane * size + i] = 0;
        wave_sync();
    }
    int chosen = -1;
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        int at = 0;
        for (int e = lane; e < p.experts; e += kWave) {
            const uint64_t c = keys[e];
            if (c > best) {
                best = c;
                at = e;
            }
        }
#pragma unroll
        for (int s = 32; s; s >>= 1) {
            const uint64_t other = __shfl_xor(best, s);
            const int oat = __shfl_xor(at, s);
            if (other > best || (other == best && oat < at)) {
                best = other;
                at = oat;
            }
        }
        if (!best) break;
        if (lane == j) chosen = at;
        if ((at & (kWave - 1)) == lane) keys[at] = 0;
        wave_sync();
    }
    wave_sync();   // the next token's keys come behind this one's last reads
    return chosen;
}

// L lanes a token, V of its experts a lane.  A choice of k out of E by k rounds
// over values and indexes in 64 bits costs 500 us for 32768 x 256; so the
// rounds go over 32-bit keys: the choice's value in 2^22 steps between the
// row's extremes (or the 64 below the largest), then the expert from above, so
// that all keys differ and the next one below `m` is m - 1 less the minimum of
// m - 1 - key in unsigned arithmetic: one subtraction and half a three-way
// minimum a key, nothing to mark as taken.  What this finds is right wherever
// neighbours in the order differ by more than the binary32 scores and the steps
// may be off (`margin`), or are of the same logit and bias.  Otherwise the first
// L in this order are put in the order of 64 bits, a lane each; and where that
// does not settle it (many as near, a NaN, two parts alike) the token goes
// through choose_exact().  The scores' errors: 2^-22 for the logistic function
// (an argument to half a step of itself, exponential and reciprocal to one
// step), 45 half steps of the largest for the softmax (arguments, a sum of 16 +
// 6 terms, the quotient), half a step of c for the bias.  All are taken twice.
// 32768 x 256 fp32 in 8 parts: 29 us, bound by instructions (some 1230 for a
// wave's four tokens, 300 of them the rounds); its 34 MB would take 7.
template <int DT, int L, int V>
__global__ __launch_bounds__(kTopkWaves * kWave) void k_topk(TopkArgs p)
{
    using Elem = typename Value<DT>::Elem;
    constexpr int kTokens = kWave / L, kExperts = L * V;
    constexpr int kIndex = kExperts <= 64 ? 6 : kExperts <= 128 ? 7 : kExperts <= 256 ? 8 : kExperts <= 512 ? 9 : 10;
    constexpr float kSteps = 4194000.0f, kInf = __builtin_inff();
    constexpr int kRoom = kTokens * (kExperts + L) / 2, kWords = kRoom > kExperts ? kRoom : kExperts;
    __shared__ uint64_t lds[kTopkWaves][kWords];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int sub = lane & (L - 1), row = lane / L;
    const int64_t token0 = (static_cast<int64_t>(blockIdx.x) * kTopkWaves + wave) * kTokens, token = token0 + row;
    if (token0 >= p.tokens) return;   // waves do not meet
    const int k = p.k;
    const bool inside = token < p.tokens, live = inside && !(p.mask && !p.mask[token]);
    const Elem* const x = static_cast<const Elem*>(p.logits) + (inside ? token : p.tokens - 1) * p.row_stride;
    const bool by_logit = !p.bias && (p.groups == 1 || !p.best_two);   // scores rise with the logits
    auto expert = [&](int v) { return (v >> 2) * (4 * L) + sub * 4 + (v & 3); };

    float v[V], c[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const int e = expert(i);
        if (p.wide) {
            if (e < p.experts) {
                Value<DT>::load4(x + e, &v[i]);
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) v[i + h] = -kInf;
            }
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) v[i + h] = e + h < p.experts ? Value<DT>::load(x, e + h) : -kInf;
        }
    }
    // Whether every register of the wave holds an expert: absent ones cost two
    // instructions at each step of what follows.
    float lowest = kInf;
#pragma unroll
    for (int i = 0; i < V; i += 2) lowest = min3(lowest, v[i], v[i + 1]);
    const bool full = !__any(lowest == -kInf);
    float top = -kInf, worst = 0.0f;   // worst: a NaN if any is NaN or +inf
    if (p.scores == kSoftmax) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            top = fmaxf(top, v[i]);
            worst += v[i] == -kInf ? 0.0f : v[i] - v[i];
        }
        top = lanes_max<L>(top);
        worst = lanes_sum<L>(worst);
    }
    float error = 0.0f;
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = v[i] == -kInf ? 0.0f : v[i];
    } else if (p.scores == kSigmoid) {
        constexpr float kLog2e = 1.44269504f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v[i]));
        error = 0x1p-21f;
    } else {
        constexpr float kLog2e = 1.44269504f;
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = v[i] == -kInf ? 0.0f : __builtin_amdgcn_exp2f(kLog2e * (v[i] - top));
            all += c[i];
        }
        const float r = __builtin_amdgcn_rcpf(lanes_sum<L>(all));
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] *= r;
        error = r * (90.0f * 0x1p-24f);
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = expert(i);
            float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (p.bias_wide) {
                if (e < p.experts) Value<kF32>::load4(p.bias + e, b);
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (e + h < p.experts) b[h] = p.bias[e + h];
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) c[i + h] += b[h];
        }
    }
    const uint64_t rows = L == 64 ? ~uint64_t(0) : ((uint64_t(1) << (L & 63)) - 1) << (row * L);
    float hi = -kInf, lo = kInf, odd = 0.0f;
    if (full) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            hi = max3(hi, c[i], c[i + 1]);
            lo = min3(lo, c[i], c[i + 1]);
            odd += c[i] + c[i + 1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            hi = max3(hi, v[i] == -kInf ? -kInf : c[i], v[i + 1] == -kInf ? -kInf : c[i + 1]);
            lo = min3(lo, v[i] == -kInf ? kInf : c[i], v[i + 1] == -kInf ? kInf : c[i + 1]);
            odd += c[i] + c[i + 1];
        }
    }
    hi = lanes_max<L>(hi);
    lo = -lanes_max<L>(-lo);
    odd = lanes_sum<L>(odd);
    if (!by_logit) error += fmaxf(fabsf(hi), fabsf(lo)) * 0x1p-23f;
    bool none = hi == -kInf;   // no expert is there, unless there are NaN alone, which the extremes pass over
    if (__any(none)) {
        bool some = false;
#pragma unroll
        for (int i = 0; i < V; ++i) some |= v[i] != -kInf;
        none = !(__ballot(some) & rows);
    }
    bool sure = fabsf(odd) < kInf || none;
    // steps of c from `base` on; a base that is far from 0 is rounded for all
    // alike, by 64 steps at most
    const float base = none ? 0.0f : fmaxf(lo, hi - 64.0f);
    const float range = fmaxf(fmaxf(none ? 1.0f : hi - base, 0x1p-100f), fabsf(base) * 0x1p-8f);
    const float scale = kSteps / range, shift = 65.0f - base * scale;
    const float off = 3.0f + 2.0f * error * scale;
    const uint32_t margin = off < kSteps ? static_cast<uint32_t>(off) + 1 : 1u << 22;

    uint64_t stays = 0;
    uint32_t part = 0;     // an expert's part is expert * part >> 20
    int helpers = 0;       // 2^helpers lanes look at a part
    if (p.groups > 1) {
        // parts one word apart from where they would be, rows L words, for other banks
        const int size = p.experts / p.groups;
        part = ((1u << 20) + size - 1) / size;
        while ((p.groups << helpers) <= L / 2) ++helpers;
        const int team = 1 << helpers;
        float* const room = reinterpret_cast<float*>(lds[wave]) + row * (kExperts + L);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t e = static_cast<uint32_t>(expert(i));
            if (full || e < static_cast<uint32_t>(p.experts)) room[e + (e * part >> 20)] = v[i] == -kInf ? -kInf : c[i];
        }
        wave_sync();
        float a = -kInf, b = -kInf;   // the two largest
        const int g0 = sub >> helpers;
        if (g0 < p.groups) {
            const float* const mine = room + g0 * (size + 1);
#pragma unroll 4
            for (int i = sub & (team - 1); i < size; i += team) {
                const float u = mine[i];
                b = __builtin_amdgcn_fmed3f(a, b, u);   // of a >= b and u the one between
                a = max3(a, u, u);
            }
        }
        for (int w = 1; w < team; w <<= 1) {
            const float oa = __shfl_xor(a, w), ob = __shfl_xor(b, w);
            b = max3(__builtin_amdgcn_fmed3f(a, b, oa), ob, ob);
            a = max3(a, oa, oa);
        }
        const float mine = p.best_two && b != -kInf ? a + b : a;
        int ahead = 0;
        for (int g = 0; g < p.groups; ++g) {
            const float other = __shfl(mine, g << helpers, L);
            ahead += other > mine || (other == mine && g < g0);
        }
        const bool stay = g0 < p.groups && ahead < p.top_groups;
        stays = __ballot(stay) >> (row * L);
        // the smallest that stays and the largest that does not
        const float least = -lanes_max<L>(stay ? -mine : -kInf);
        const float most = lanes_max<L>(g0 < p.groups && !stay ? mine : -kInf);
        // two sums of two, and their own rounding
        if (most != -kInf && !(least - most > 4.0f * error + (fabsf(least) + fabsf(most)) * 0x1p-23f)) sure = false;
        wave_sync();
    }
    uint32_t key[V];
    const uint32_t from = kExperts - 1 - sub * 4;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t q = static_cast<uint32_t>(fmaxf(__builtin_fmaf(c[i], scale, shift), 1.0f));
        key[i] = (q << kIndex) + from - ((i >> 2) * (4 * L) + (i & 3));
    }
    if (!full) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = v[i] == -kInf ? 0 : key[i];
    }
    if (p.groups > 1) {
        // all ones where bit `at` is set
        auto in_part = [&](uint32_t e) {
            const uint32_t at = (e * part >> 20) << helpers;
            return static_cast<uint32_t>(static_cast<int32_t>((L < 64 ? static_cast<uint32_t>(stays) >> (at & 31u)
                                                                      : static_cast<uint32_t>(stays >> (at & 63u))) << 31) >> 31);
        };
        if (p.experts / p.groups % 4 == 0) {   // four neighbours are of one part
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const uint32_t bits = in_part(static_cast<uint32_t>(expert(i)));
#pragma unroll
                for (int h = 0; h < 4; ++h) key[i + h] &= bits;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] &= in_part(static_cast<uint32_t>(expert(i)));
        }
    }
    uint32_t m = ~0u, own = 0;   // own: the key of choice `sub`; choice k is the first one left out
    for (int j = 0; j <= k; ++j) {
        const uint32_t t = m - 1;
        uint32_t r = ~0u;
#pragma unroll
        for (int i = 0; i < V; ++i) r = min(r, t - key[i]);
        r = lanes_min_u32<L>(r);
        m = m && r <= t ? t - r : 0;
        if (sub == j) own = m;
    }
    // Candidates: choice `sub` and, behind the choices, those left out.
    auto index_of = [](uint32_t key) { return static_cast<int>(kExperts - 1 - (key & (kExperts - 1))); };
    bool has = own >> kIndex;
    int chosen = has && sub < k ? index_of(own) : -1;
    float cx = Value<DT>::load(x, has ? index_of(own) : 0);
    {
        const float cb = p.bias ? p.bias[has ? index_of(own) : 0] : 0.0f;
        const uint32_t next = __shfl_down(own, 1, L);
        const float nx = __shfl_down(cx, 1, L), nb = __shfl_down(cb, 1, L);
        const bool near = sub < k && (next >> kIndex) && (own >> kIndex) - (next >> kIndex) < margin;
        const bool same = cx == nx && cb == nb;
        bool open = __ballot(near && !same) & rows;
        // the last choice and the first one left out are alike: so must be all that are as near
        if (__any(near && same && sub == k - 1)) {
            const uint32_t edge = __shfl(own, k - 1, L) >> kIndex;
            const float ex = __shfl(cx, k - 1, L), eb = __shfl(cb, k - 1, L);
            bool other = false;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t q = key[i] >> kIndex;
                if (q && q <= edge && q + margin > edge)
                    other |= !(v[i] == ex && (!p.bias || p.bias[expert(i)] == eb));
            }
            open |= static_cast<bool>(__ballot(other) & rows);
        }
        open = open && live && sure && !p.exact;
        if (__any(open)) {
            // the first L candidates in the order of 64 bits; those behind them are
            // out if the last one is far enough from the last choice
            for (int j = k + 1; j < L; ++j) {
                const uint32_t t = m - 1;
                uint32_t r = ~0u;
#pragma unroll
                for (int i = 0; i < V; ++i) r = min(r, t - key[i]);
                r = lanes_min_u32<L>(r);
                m = m && r <= t ? t - r : 0;
                if (sub == j) own = m;
            }
            has = own >> kIndex;
            const int at = has ? index_of(own) : 0;
            const float ox = Value<DT>::load(x, at);
            double value = ox;
            if (!by_logit && p.scores == kSigmoid) value = 1 / (1 + exp(-value));
            if (!by_logit && p.scores == kSoftmax) {
                double all = 0;
                for (int e = sub; e < p.experts; e += L) {
                    const float u = Value<DT>::load(x, e);
                    all += u == -kInf ? 0 : exp(static_cast<double>(u) - top);
                }
#pragma unroll
                for (int w = 1; w < L; w <<= 1) all += __shfl_xor(all, w);
                value = exp(value - top) / all;
            }
            if (p.bias) value += p.bias[at];
            int ahead = 0;
            for (int j = 0; j < L; ++j) {
                const double other = __shfl(value, j, L);
                const int oat = __shfl(at, j, L), ohas = __shfl(static_cast<int>(has), j, L);
                ahead += ohas && (other > value || (other == value && oat < at));
            }
            if (!has) ahead = sub;   // behind all others
            // to the lane of its rank
            const int to = (row * L + ahead) * 4;
            const int moved = __builtin_amdgcn_ds_permute(to, at);
            const uint32_t there = static_cast<uint32_t>(__builtin_amdgcn_ds_permute(to, static_cast<int>(own)));
            const uint32_t edge = __shfl(there, k - 1, L) >> kIndex, last = __shfl(own, L - 1, L) >> kIndex;
            if (open) {
                chosen = there >> kIndex && sub < k ? moved : -1;
                cx = Value<DT>::load(x, moved);
                if (last && (edge < last || edge - last < margin)) sure = false;
            }
        }
    }
    if (p.exact) sure = false;
    // rows that are not sure, one at a time
    uint64_t open = __ballot(live && !sure);
    while (open) {
        const int which = __builtin_ctzll(open) / L;
        const int found = choose_exact<DT>(p, token0 + which, lane, lds[wave]);
        const int to = __shfl(found, sub);
        if (row == which) {
            chosen = sub < k ? to : -1;
            if (chosen >= 0) cx = Value<DT>::load(x, chosen);
        }
        open &= L == 64 ? 0 : ~(((uint64_t(1) << (L & 63)) - 1) << (which * L));
    }
    // Weights.  Logistic scores are exp(min(x, 0)) / (1 + exp(-|x|)), so that a
    // common factor can leave both sides of a division of them.
    has = live && chosen >= 0;
    if (!has) cx = -kInf;
    float s;
    if (p.scores == kSigmoid) {
        const float low = fminf(cx, 0.0f), most = lanes_max<L>(has ? low : -kInf);
        s = has ? expf(p.renormalize ? low - most : low) / (1.0f + expf(-fabsf(cx))) : 0.0f;
        if (has && cx != cx) s = cx;
    } else {
        const float most = lanes_max<L>(cx);
        s = has ? expf(cx - (p.renormalize ? most : top)) : 0.0f;
        if (!p.renormalize) {
            float all = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) all += v[i] == -kInf ? 0.0f : expf(v[i] - top);
            s /= lanes_sum<L>(all);
        }
        if (worst != worst && has) s = __builtin_nanf("");
    }
    const float whole = lanes_sum<L>(s);
    if (p.renormalize) s /= whole;
    if (inside && sub < k) {
        p.weights[token * k + sub] = has ? p.scale * s : 0.0f;
        p.ids[token * k + sub] = has ? chosen : -1;
    }
}

// L lanes a token, V of its experts a lane, a choice a lane.  Where only the
// chosen have a gradient, a token's logits are read at those alone.  32768 x 256
// fp32: 8.6 us, 3.9 TB/s of stores (18.5 with a wave a token, by its
// instructions).
template <int DT, int L, int V>
__global__ __launch_bounds__(kTopkWaves * kWave) void k_topk_backward(TopkBackwardArgs p)
{
    using Elem = typename Value<DT>::Elem;
    constexpr int kTokens = kWave / L, kExperts = L * V;
    __shared__ __attribute__((aligned(16))) float lds[kTopkWaves][kTokens * kExperts];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int sub = lane & (L - 1), row = lane / L;
    const int64_t token0 = (static_cast<int64_t>(blockIdx.x) * kTopkWaves + wave) * kTokens;
    if (token0 >= p.tokens) return;
    const bool inside = token0 + row < p.tokens;
    const int64_t token = inside ? token0 + row : p.tokens - 1;
    const int k = p.k;
    constexpr float kInf = __builtin_inff();
    const Elem* const x = static_cast<const Elem*>(p.logits) + token * p.row_stride;
    Elem* const dx = static_cast<Elem*>(p.dlogits) + token * p.experts;
    const int id = sub < k ? p.ids[token * k + sub] : -1;
    const bool has = id >= 0 && id < p.experts;
    const float c = has ? Value<DT>::load(x, id) : -kInf;
    const float g = has ? p.dweights[token * k + sub] : 0.0f;
    const bool dense = p.scores == kSoftmax && !p.renormalize;
    auto expert = [&](int v) { return (v >> 2) * (4 * L) + sub * 4 + (v & 3); };
    float* const room = lds[wave] + row * kExperts;
    using f32x4 = float __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<f32x4*>(room + expert(i)) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float v[V], top = -kInf, sum = 0.0f;
    if (dense) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = expert(i);
            if (p.wide && e < p.experts) {
                Value<DT>::load4(x + e, &v[i]);
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) v[i + h] = e + h < p.experts ? Value<DT>::load(x, e + h) : -kInf;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);
        top = lanes_max<L>(top);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = v[i] == -kInf ? 0.0f : expf(v[i] - top);
            sum += v[i];
        }
        sum = lanes_sum<L>(sum);
    }
    float s, d;
    if (p.scores == kSigmoid) {
        const float low = fminf(c, 0.0f), most = lanes_max<L>(has ? low : -kInf);
        const float t = expf(-fabsf(c));
        s = has ? expf(p.renormalize ? low - most : low) / (1.0f + t) : 0.0f;
        const float rest = (c > 0.0f ? t : 1.0f) / (1.0f + t);   // 1 - the score
        const float whole = lanes_sum<L>(s);
        if (p.renormalize) s /= whole;
        const float mean = lanes_sum<L>(g * s);
        d = p.scale * s * rest * (p.renormalize ? g - mean : g);
    } else {
        const float most = lanes_max<L>(c);   // by all lanes
        s = has ? expf(c - (dense ? top : most)) : 0.0f;
        const float whole = lanes_sum<L>(s);
        s /= dense ? sum : whole;
        const float mean = lanes_sum<L>(g * s);
        d = dense ? mean : p.scale * s * (g - mean);   // dense: of the row
    }
    const bool any = __ballot(has) & (L == 64 ? ~uint64_t(0) : ((uint64_t(1) << (L & 63)) - 1) << (row * L));
    wave_sync();
    if (has) room[id] = dense ? g : d;
    wave_sync();
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const int e = expert(i);
        if (e >= p.experts || !inside) continue;
        const f32x4 q = *reinterpret_cast<const f32x4*>(room + e);
        float r[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            r[h] = q[h];
            if (dense) r[h] = !any || v[i + h] == 0.0f ? 0.0f : p.scale * (v[i + h] / sum) * (r[h] - d);
        }
        if (p.dense_wide) {
            Value<DT>::store4(dx + e, r);
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (e + h < p.experts) Value<DT>::store(dx, e + h, r[h]);
        }
    }
}

// ---- the order of rows ----------------------------------------------------------

// Sorting by counting: a block takes a run of slots, its waves parts of it.
// With more than one block, the first kernel counts every block's slots by
// expert, and each block of the second adds up the counts itself: 128 blocks of
// 2048 slots with 257 bins are 17 MB from the L2, in 16-byte pieces of which a
// thread has eight on their way.  262144 slots, 256 experts: 3.6 us of counting
// and 9.2 (41 where a thread read the counts of its bins one by one); up to 4096
// slots 3.0 in one launch.  Bound by latency: counting, the counts' way through
// the L2, then the waves' steps of 64 slots one behind the other.
__device__ __forceinline__ int bin_of(const OrderArgs& p, int32_t id)
{
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(p.experts) ? id : p.experts;
}

__global__ __launch_bounds__(kOrderThreads) void k_order_count(OrderArgs p)
{
    __shared__ int32_t count[kMaxExperts + 4];
    const int t = static_cast<int>(threadIdx.x);
    for (int e = t; e < p.bins; e += kOrderThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * p.chunk, last = first + p.chunk < p.slots ? first + p.chunk : p.slots;
    constexpr int U = 4;
    for (int64_t i = first + t; i < last; i += U * kOrderThreads) {
        int32_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = i + u * kOrderThreads < last ? p.ids[i + u * kOrderThreads] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kOrderThreads < last) atomicAdd(&count[bin_of(p, id[u])], 1);
    }
    __syncthreads();
    for (int e = t; e < p.bins; e += kOrderThreads) p.counts[static_cast<int64_t>(blockIdx.x) * p.bins + e] = count[e];
}

// A slot's row: rows of the experts before its own, rows of its own in earlier
// blocks, in earlier waves of the block, in earlier lanes.
__global__ __launch_bounds__(kOrderThreads) void k_order_place(OrderArgs p)
{
    constexpr int W = kOrderThreads / kWave, U = 8;
    __shared__ int32_t next[W][kMaxExperts + 4];   // slots of each wave, then its next row
    __shared__ int32_t total[kMaxExperts + 4], before[kMaxExperts + 4], sums[W];
    const int t = static_cast<int>(threadIdx.x), lane = t & 63, wave = t >> 6, bins = p.bins;
    for (int e = t; e < bins; e += kOrderThreads) {
        total[e] = before[e] = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) next[w][e] = 0;
    }
    __syncthreads();
    const int64_t part = p.chunk / W, begin = blockIdx.x * p.chunk + wave * part;
    const int64_t end = begin + part < p.slots ? begin + part : p.slots;
    int32_t id[U];
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kWave + lane;
            id[u] = i < end ? p.ids[i] : -1;
        }
    };
    for (int64_t i0 = begin; i0 < end; i0 += U * kWave) {
        load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * kWave + lane < end) atomicAdd(&next[wave][bin_of(p, id[u])], 1);
    }
    if (p.blocks > 1) {
        const int quads = bins / 4, teams = kOrderThreads / quads, team = t / quads, quad = t - team * quads;
        if (team < teams) {
            int32_t all[4] = {}, mine[4] = {};
            const int32_t* const c = p.counts + quad * 4;
            for (int b = team; b < p.blocks; b += teams * U) {
                i32x4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    v[u] = b + u * teams < p.blocks ? *reinterpret_cast<const i32x4*>(c + static_cast<int64_t>(b + u * teams) * bins)
                                                    : i32x4{0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool earlier = b + u * teams < static_cast<int>(blockIdx.x);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        all[h] += v[u][h];
                        mine[h] += earlier ? v[u][h] : 0;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                atomicAdd(&total[quad * 4 + h], all[h]);
                atomicAdd(&before[quad * 4 + h], mine[h]);
            }
        }
    }
    __syncthreads();
    // neighbouring bins to a thread, and the sum over the threads before it
    constexpr int B = (kMaxExperts + 4 + kOrderThreads - 1) / kOrderThreads;
    const int per = bins > 2 * kOrderThreads ? 3 : bins > kOrderThreads ? 2 : 1;
    int32_t all[B], run = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const int e = t * per + i;
        all[i] = 0;
        if (i >= per || e >= bins) continue;
        if (p.blocks == 1) {
#pragma unroll
            for (int w = 0; w < W; ++w) all[i] += next[w][e];
        } else {
            all[i] = total[e];
        }
        run += all[i];
    }
    int32_t scan = run;
    for (int s = 1; s < kWave; s <<= 1) {
        const int32_t up = __shfl_up(scan, s);
        if (lane >= s) scan += up;
    }
    if (lane == kWave - 1) sums[wave] = scan;
    __syncthreads();
    int32_t row = scan - run;
    for (int w = 0; w < wave; ++w) row += sums[w];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const int e = t * per + i;
        if (i >= per || e >= bins) continue;
        if (blockIdx.x == 0 && e <= p.experts) p.offsets[e] = row;
        int32_t at = row + before[e];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int32_t c = next[w][e];
            next[w][e] = at;
            at += c;
        }
        row += all[i];
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) <= p.experts) ++bits;
    const bool once = end - begin <= U * kWave;   // the ids are still there
    for (int64_t i0 = begin; i0 < end; i0 += U * kWave) {
        if (!once) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kWave + lane;
            if (i - lane >= end) break;
            const bool in = i < end;
            const int e = bin_of(p, id[u]);
            uint64_t same = __ballot(in);   // lanes of the same bin
            for (int b = 0; b < bits; ++b) {
                const uint64_t set = __ballot(e >> b & 1);
                same &= e >> b & 1 ? set : ~set;
            }
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int32_t at = in ? next[wave][e] + rank : 0;
            wave_sync();
            if (in && rank == 0) next[wave][e] = at + __popcll(same);
            wave_sync();
            if (in) {
                p.slot_of_row[at] = e < p.experts ? static_cast<int32_t>(i) : -1;
                p.row_of_slot[i] = e < p.experts ? at : -1;
            }
        }
    }
}

__global__ __launch_bounds__(256) void k_balance(const float* bias, const int32_t* offsets, int32_t experts, float rate,
                                                 float* out)
{
    const int64_t all = offsets[experts];
    for (int e = static_cast<int>(threadIdx.x); e < experts; e += 256) {
        const int64_t more = all - static_cast<int64_t>(experts) * (offsets[e + 1] - offsets[e]);
        out[e] = bias[e] + (more > 0 ? rate : more < 0 ? -rate : 0.0f);
    }
}

// ---- rows -----------------------------------------------------------------------

// A block per token.  Lane j of every wave holds the row (and the weight) of
// choice j: taken from there by readlane they are uniform, and no load of them
// stands between those of the rows.
struct Choices {
    int32_t row;      // of choice `lane`, -1: none
    float weight;

    __device__ __forceinline__ Choices(const int32_t* rows, const float* weights, int64_t t, int k, int64_t count)
    {
        const int lane = static_cast<int>(threadIdx.x) & 63;
        row = lane < k ? rows[t * k + lane] : -1;
        if (row >= count) row = -1;
        weight = weights && lane < k ? weights[t * k + lane] : 1.0f;
    }
    __device__ __forceinline__ int64_t row_of(int j) const { return __builtin_amdgcn_readlane(row, j); }
    __device__ __forceinline__ float weight_of(int j) const
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, weight), j));
    }
};

// Each piece of the token's row is read once and written to the rows of its
// slots.  Block t also clears those of rows t * k .. that are of no slot.  Bound
// by memory: 8190 x 8 rows of 2048 bf16 302 MB in 46 us, 6.6 TB/s, nearly all of
// it stores.
template <class U>
__global__ __launch_bounds__(kRowThreads) void k_dispatch(RowsArgs p)
{
    const int64_t t = blockIdx.x;
    const U* const x = reinterpret_cast<const U*>(p.x) + t * p.x_stride;
    U* const out = reinterpret_cast<U*>(p.out);
    const Choices to(p.row_of_slot, nullptr, t, p.k, p.tokens * p.k);
    const Choices of(p.slot_of_row, nullptr, t, p.k, p.tokens * p.k);
    const uint64_t all = p.k == kWave ? ~uint64_t(0) : (uint64_t(1) << p.k) - 1;
    const uint64_t has = __ballot(to.row >= 0) & all, rest = p.zero_rest ? __ballot(of.row < 0) & all : 0;
    for (int64_t c = threadIdx.x; c < p.cols; c += blockDim.x) {
        const U v = __builtin_nontemporal_load(x + c);
        auto put = [&](U* q, U u) {
            if (p.past_caches)
                __builtin_nontemporal_store(u, q);
            else
                *q = u;
        };
        for (uint64_t m = has; m; m &= m - 1) put(out + to.row_of(__builtin_ctzll(m)) * p.out_stride + c, v);
        for (uint64_t m = rest; m; m &= m - 1) put(out + (t * p.k + __builtin_ctzll(m)) * p.out_stride + c, U{});
    }
}

// A lane has the pieces of eight of the token's rows on their way.  They are read
// once, so past the caches: 8190 x 8 rows of 2048 bf16 302 MB in 57 us, 5.3 TB/s
// (88 by cached loads, whatever their number); 16384 x 8 of 4096 with what is
// added 1.34 GB in 240 to 276 us.  Bound by memory.
template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void k_combine(RowsArgs p)
{
    using P = Piece<DT, WIDE>;
    constexpr int U = 8;
    const int64_t t = blockIdx.x;
    const Choices from(p.row_of_slot, p.weights, t, p.k, p.tokens * p.k);
    const uint64_t has = __ballot(from.row >= 0);
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * P::kValues; c < p.cols;
         c += static_cast<int64_t>(blockDim.x) * P::kValues) {
        float acc[P::kValues] = {};
        for (int j0 = 0; j0 < p.k; j0 += U) {
            if (!(has >> j0 & 0xff)) continue;
            typename P::Raw raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = from.row_of(j0 + u);
                raw[u] = P::fetch_once(p.x, (r < 0 ? 0 : r) * p.x_stride + c);   // row 0 for none: no branch between the loads
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // for none 0 times 0: behind a branch the load would be put there too
                float v[P::kValues];
                P::unpack(has >> (j0 + u) & 1 ? raw[u] : typename P::Raw{}, v);
                const float w = has >> (j0 + u) & 1 ? from.weight_of(j0 + u) : 0.0f;
#pragma unroll
                for (int i = 0; i < P::kValues; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
            }
        }
        if (p.add) {
            float v[P::kValues];
            P::load(p.add, t * p.add_stride + c, v);
#pragma unroll
            for (int i = 0; i < P::kValues; ++i) acc[i] += v[i];
        }
        P::store(p.out, t * p.out_stride + c, acc, p.past_caches);
    }
}

// Eight choices at a time: their rows of y are read and their rows of dy
// written beside one another.  16384 x 8 rows of 4096 bf16: 2.28 GB in 428 us,
// 5.3 TB/s, above a copy's rate.
template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void k_combine_backward(RowsArgs p)
{
    using P = Piece<DT, WIDE>;
    constexpr int W = kRowThreads / kWave, U = 8;
    __shared__ float part[W][kMaxChoices];
    const int64_t t = blockIdx.x;
    const int tid = static_cast<int>(threadIdx.x);
    const Choices from(p.row_of_slot, p.out ? p.weights : nullptr, t, p.k, p.tokens * p.k);
    const Choices of(p.slot_of_row, nullptr, t, p.k, p.tokens * p.k);
    const uint64_t has = __ballot(from.row >= 0);
    const uint64_t all = p.k == kWave ? ~uint64_t(0) : (uint64_t(1) << p.k) - 1;
    const uint64_t rest = p.out ? __ballot(of.row < 0) & all : 0;
    for (int j0 = 0; j0 < p.k; j0 += U) {
        float dot[U] = {};
        for (int64_t c = static_cast<int64_t>(tid) * P::kValues; c < p.cols;
             c += static_cast<int64_t>(blockDim.x) * P::kValues) {
            typename P::Raw raw[U];
            if (p.dweights) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t r = from.row_of(j0 + u);
                    raw[u] = P::fetch_once(p.y, (r < 0 ? 0 : r) * p.y_stride + c);
                }
            }
            float g[P::kValues];
            P::load(p.x, t * p.x_stride + c, g);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p.dweights) {
                    float v[P::kValues];
                    P::unpack(has >> (j0 + u) & 1 ? raw[u] : typename P::Raw{}, v);
#pragma unroll
                    for (int i = 0; i < P::kValues; ++i) dot[u] = __builtin_fmaf(g[i], v[i], dot[u]);
                }
                if (p.out && has >> (j0 + u) & 1) {
                    const float w = from.weight_of(j0 + u);
                    float v[P::kValues];
#pragma unroll
                    for (int i = 0; i < P::kValues; ++i) v[i] = w * g[i];
                    P::store(p.out, from.row_of(j0 + u) * p.out_stride + c, v, p.past_caches);
                }
            }
        }
        if (p.dweights) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float sum = wave_sum(dot[u]);
                if ((tid & 63) == 0 && j0 + u < p.k) part[tid >> 6][j0 + u] = sum;
            }
        }
    }
    for (uint64_t m = rest; m; m &= m - 1) {
        const float zero[P::kValues] = {};
        for (int64_t c = static_cast<int64_t>(tid) * P::kValues; c < p.cols;
             c += static_cast<int64_t>(blockDim.x) * P::kValues)
            P::store(p.out, (t * p.k + __builtin_ctzll(m)) * p.out_stride + c, zero, p.past_caches);
    }
    if (!p.dweights) return;
    __syncthreads();
    if (tid < p.k) {
        float sum = 0.0f;
        for (int w = 0; w < static_cast<int>(blockDim.x) / kWave; ++w) sum += part[w][tid];
        p.dweights[t * p.k + tid] = has >> tid & 1 ? sum : 0.0f;   // whatever dout holds
    }
}

}  // namespace

namespace {

template <int DT>
TopkKernel choose_topk(int32_t experts, int32_t k, int32_t groups)
{
    // choices and the first one left out are a lane each, and parts
    if (experts <= 256 && k < 16 && groups <= 16) {
        if (experts <= 64) return {reinterpret_cast<const void*>(k_topk<DT, 16, 4>), 4};
        if (experts <= 128) return {reinterpret_cast<const void*>(k_topk<DT, 16, 8>), 4};
        return {reinterpret_cast<const void*>(k_topk<DT, 16, 16>), 4};
    }
    if (experts <= 512 && k < 32 && groups <= 32) return {reinterpret_cast<const void*>(k_topk<DT, 32, 16>), 2};
    return {reinterpret_cast<const void*>(k_topk<DT, 64, 16>), 1};
}

}  // namespace

TopkKernel topk_kernel(int dtype, int32_t experts, int32_t k, int32_t groups)
{
    return dtype == kF32   ? choose_topk<kF32>(experts, k, groups)
           : dtype == kF16 ? choose_topk<kF16>(experts, k, groups)
                           : choose_topk<kBF16>(experts, k, groups);
}
namespace {

template <int DT>
TopkKernel choose_topk_backward(int32_t experts, int32_t k)
{
    if (experts <= 256 && k <= 16) {
        if (experts <= 64) return {reinterpret_cast<const void*>(k_topk_backward<DT, 16, 4>), 4};
        if (experts <= 128) return {reinterpret_cast<const void*>(k_topk_backward<DT, 16, 8>), 4};
        return {reinterpret_cast<const void*>(k_topk_backward<DT, 16, 16>), 4};
    }
    if (experts <= 512 && k <= 32) return {reinterpret_cast<const void*>(k_topk_backward<DT, 32, 16>), 2};
    return {reinterpret_cast<const void*>(k_topk_backward<DT, 64, 16>), 1};
}

}  // namespace

TopkKernel topk_backward_kernel(int dtype, int32_t experts, int32_t k)
{
    return dtype == kF32   ? choose_topk_backward<kF32>(experts, k)
           : dtype == kF16 ? choose_topk_backward<kF16>(experts, k)
                           : choose_topk_backward<kBF16>(experts, k);
}
const void* order_count_kernel() { return reinterpret_cast<const void*>(k_order_count); }
const void* order_place_kernel() { return reinterpret_cast<const void*>(k_order_place); }
const void* balance_kernel() { return reinterpret_cast<const void*>(k_balance); }

const void* dispatch_kernel(int bytes, bool wide)
{
    return wide         ? reinterpret_cast<const void*>(k_dispatch<u32x4>)
           : bytes == 4 ? reinterpret_cast<const void*>(k_dispatch<uint32_t>)
                        : reinterpret_cast<const void*>(k_dispatch<uint16_t>);
}
const void* combine_kernel(int dtype, bool wide)
{
    static const void* const fn[3][2] = {
        {reinterpret_cast<const void*>(k_combine<kF32, false>), reinterpret_cast<const void*>(k_combine<kF32, true>)},
        {reinterpret_cast<const void*>(k_combine<kF16, false>), reinterpret_cast<const void*>(k_combine<kF16, true>)},
        {reinterpret_cast<const void*>(k_combine<kBF16, false>), reinterpret_cast<const void*>(k_combine<kBF16, true>)}};
    return fn[dtype][wide];
}
const void* combine_backward_kernel(int dtype, bool wide)
{
    static const void* const fn[3][2] = {{reinterpret_cast<const void*>(k_combine_backward<kF32, false>),
                                          reinterpret_cast<const void*>(k_combine_backward<kF32, true>)},
                                         {reinterpret_cast<const void*>(k_combine_backward<kF16, false>),
                                          reinterpret_cast<const void*>(k_combine_backward<kF16, true>)},
                                         {reinterpret_cast<const void*>(k_combine_backward<kBF16, false>),
                                          reinterpret_cast<const void*>(k_combine_backward<kBF16, true>)}};
    return fn[dtype][wide];
}

}  // namespace experts
