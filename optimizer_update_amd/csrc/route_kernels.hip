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

// One wave per token, expert v * 64 + lane in register v: scores in 64 bits,
// one round of the wave for each choice.
template <int DT>
__global__ __launch_bounds__(kTopkWaves * kWave) void k_topk(TopkArgs p)
{
    constexpr int V = kMaxExperts / kWave;
    __shared__ uint64_t lds[kTopkWaves][kMaxExperts];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kTopkWaves + wave;
    if (token >= p.tokens) return;   // waves do not meet
    const int k = p.k;
    float* const weights = p.weights + token * k;
    int32_t* const ids = p.ids + token * k;
    if (p.mask && !p.mask[token]) {
        if (lane < k) {
            weights[lane] = 0.0f;
            ids[lane] = -1;
        }
        return;
    }
    const typename Value<DT>::Elem* x = static_cast<const typename Value<DT>::Elem*>(p.logits) + token * p.row_stride;
    constexpr float kInf = __builtin_inff();
    const bool by_logit = !p.bias && (p.groups == 1 || !p.best_two);   // scores rise with the logits
    float v[V], top = -kInf;
    bool bad = false;                                                  // a NaN or +inf among the logits
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        v[i] = e < p.experts ? Value<DT>::load(x, e) : -kInf;
        top = fmaxf(top, v[i]);
        bad |= !(v[i] < kInf);
    }
    top = wave_max(top);
    bad = __any(bad);
    double total = 0;
    if (p.scores == kSoftmax && !by_logit) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (v[i] != -kInf) total += exp(static_cast<double>(v[i]) - top);
#pragma unroll
        for (int s = 32; s; s >>= 1) total += __shfl_xor(total, s);
    }
    uint64_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        key[i] = 0;
        if (e >= p.experts || v[i] == -kInf) continue;
        double c = v[i];
        if (!by_logit) {
            c = p.scores == kSoftmax ? exp(c - top) / total : 1 / (1 + exp(-c));
            if (p.bias) c += p.bias[e];
        }
        key[i] = order_key(c);
    }
    if (p.groups > 1) {
        const int size = p.experts / p.groups;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * kWave + lane < p.experts) lds[wave][i * kWave + lane] = key[i];
        wave_sync();
        uint64_t mine = 0;
        if (lane < p.groups) {
            uint64_t a = 0, b = 0;
            for (int i = 0; i < size; ++i) {
                const uint64_t c = lds[wave][lane * size + i];
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
        const uint64_t stays = __ballot(lane < p.groups && ahead < p.top_groups);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * kWave + lane;
            if (e < p.experts && !(stays >> (e / size) & 1)) key[i] = 0;
        }
    }
    int chosen = -1;   // of choice `lane`
    for (int j = 0; j < k; ++j) {
        uint64_t best = key[0];
        int at = lane;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            if (key[i] > best) {
                best = key[i];
                at = i * kWave + lane;
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
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * kWave + lane == at) key[i] = 0;
    }
    // Weights.  Logistic scores are exp(min(x, 0)) / (1 + exp(-|x|)), so that a
    // common factor can leave both sides of a division of them.
    const bool has = lane < k && chosen >= 0;
    const float c = has ? Value<DT>::load(x, chosen) : -kInf;
    float s;
    if (p.scores == kSigmoid) {
        const float low = fminf(c, 0.0f), most = p.renormalize ? wave_max(has ? low : -kInf) : 0.0f;
        s = has ? expf(low - most) / (1.0f + expf(-fabsf(c))) : 0.0f;
        if (has && c != c) s = c;
    } else {
        const float most = p.renormalize ? wave_max(c) : top;
        s = has ? expf(c - most) : 0.0f;
        if (!p.renormalize) {
            float sum = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[i] == -kInf ? 0.0f : expf(v[i] - top);
            s /= wave_sum(sum);
        }
        if (bad && has) s = __builtin_nanf("");
    }
    if (p.renormalize) s /= wave_sum(s);
    if (lane < k) {
        weights[lane] = has ? p.scale * s : 0.0f;
        ids[lane] = chosen;
    }
}

// One wave per token.
template <int DT>
__global__ __launch_bounds__(kTopkWaves * kWave) void k_topk_backward(TopkBackwardArgs p)
{
    constexpr int V = kMaxExperts / kWave;
    __shared__ float lds[kTopkWaves][kMaxExperts];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int64_t token = static_cast<int64_t>(blockIdx.x) * kTopkWaves + wave;
    if (token >= p.tokens) return;
    const int k = p.k;
    constexpr float kInf = __builtin_inff();
    const typename Value<DT>::Elem* x = static_cast<const typename Value<DT>::Elem*>(p.logits) + token * p.row_stride;
    typename Value<DT>::Elem* dx = static_cast<typename Value<DT>::Elem*>(p.dlogits) + token * p.experts;
    const int id = lane < k ? p.ids[token * k + lane] : -1;
    const bool has = id >= 0 && id < p.experts;
    const float c = has ? Value<DT>::load(x, id) : -kInf;
    const float g = has ? p.dweights[token * k + lane] : 0.0f;
    const bool dense = p.scores == kSoftmax && !p.renormalize && __any(has);
    float v[V], top = -kInf, sum = 0.0f;
    if (dense) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * kWave + lane;
            v[i] = e < p.experts ? Value<DT>::load(x, e) : -kInf;
            top = fmaxf(top, v[i]);
        }
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < V; ++i) sum += v[i] == -kInf ? 0.0f : expf(v[i] - top);
        sum = wave_sum(sum);
    }
    float s, d;
    if (p.scores == kSigmoid) {
        const float low = fminf(c, 0.0f), most = p.renormalize ? wave_max(has ? low : -kInf) : 0.0f;
        const float t = expf(-fabsf(c));
        s = has ? expf(low - most) / (1.0f + t) : 0.0f;
        const float rest = (c > 0.0f ? t : 1.0f) / (1.0f + t);   // 1 - the score
        if (p.renormalize) {
            s /= wave_sum(s);
            d = p.scale * s * rest * (g - wave_sum(g * s));
        } else {
            d = p.scale * s * rest * g;
        }
    } else if (p.renormalize) {
        const float most = wave_max(c);   // by all lanes
        s = has ? expf(c - most) : 0.0f;
        s /= wave_sum(s);
        d = p.scale * s * (g - wave_sum(g * s));
    } else {
        s = has ? expf(c - top) / sum : 0.0f;
        d = wave_sum(g * s);   // of the row
    }
    float* row = lds[wave];
    for (int e = lane; e < p.experts; e += kWave) row[e] = 0.0f;
    wave_sync();
    if (has) row[id] = dense ? g : d;
    wave_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * kWave + lane;
        if (e >= p.experts) continue;
        float r = row[e];
        if (dense) r = v[i] == -kInf ? 0.0f : p.scale * (expf(v[i] - top) / sum) * (r - d);
        Value<DT>::store(dx, e, r);
    }
}

// ---- the order of rows ----------------------------------------------------------

// Sorting by counting: a block takes a run of slots, its waves parts of it.
__device__ __forceinline__ int bin_of(const OrderArgs& p, int64_t slot)
{
    const int32_t id = p.ids[slot];
    return id >= 0 && id < p.experts ? id : p.experts;
}

__global__ __launch_bounds__(kOrderThreads) void k_order_count(OrderArgs p)
{
    __shared__ int32_t count[kMaxExperts + 1];
    const int t = static_cast<int>(threadIdx.x), bins = p.experts + 1;
    for (int e = t; e < bins; e += kOrderThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * p.chunk, last = first + p.chunk < p.slots ? first + p.chunk : p.slots;
    for (int64_t i = first + t; i < last; i += kOrderThreads) atomicAdd(&count[bin_of(p, i)], 1);
    __syncthreads();
    for (int e = t; e < bins; e += kOrderThreads) p.counts[static_cast<int64_t>(blockIdx.x) * bins + e] = count[e];
}

// A slot's row: rows of the experts before its own, rows of its own in earlier
// blocks, in earlier waves of the block, in earlier lanes.
__global__ __launch_bounds__(kOrderThreads) void k_order_place(OrderArgs p)
{
    constexpr int W = kOrderThreads / kWave;
    __shared__ int32_t next[W][kMaxExperts + 1];   // the next row of each wave
    __shared__ int32_t sums[W];
    const int t = static_cast<int>(threadIdx.x), lane = t & 63, wave = t >> 6, bins = p.experts + 1;
    for (int e = t; e < W * (kMaxExperts + 1); e += kOrderThreads) (&next[0][0])[e] = 0;
    __syncthreads();
    const int64_t part = p.chunk / W, begin = blockIdx.x * p.chunk + wave * part;
    const int64_t end = begin + part < p.slots ? begin + part : p.slots;
    for (int64_t i = begin + lane; i < end; i += kWave) atomicAdd(&next[wave][bin_of(p, i)], 1);
    __syncthreads();
    // two bins a thread at most: a thread's are neighbours
    constexpr int B = (kMaxExperts + kOrderThreads) / kOrderThreads;
    int32_t all[B], before[B], run = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const int e = t * B + i;
        all[i] = before[i] = 0;
        if (e >= bins) continue;
        if (p.blocks == 1) {
            for (int w = 0; w < W; ++w) all[i] += next[w][e];
        } else {
            for (int b = 0; b < p.blocks; ++b) {
                const int32_t c = p.counts[static_cast<int64_t>(b) * bins + e];
                all[i] += c;
                if (b < static_cast<int>(blockIdx.x)) before[i] += c;
            }
        }
        run += all[i];
    }
    // sum over the threads before this one
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
        const int e = t * B + i;
        if (e >= bins) continue;
        if (blockIdx.x == 0) p.offsets[e] = row;
        int32_t at = row + before[i];
        for (int w = 0; w < W; ++w) {
            const int32_t c = next[w][e];
            next[w][e] = at;
            at += c;
        }
        row += all[i];
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < bins) ++bits;
    for (int64_t i0 = begin; i0 < end; i0 += kWave) {
        const int64_t i = i0 + lane;
        const bool in = i < end;
        const int e = in ? bin_of(p, i) : 0;
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

// A block per token: each piece of its row is read once and written to the rows
// of its slots.  Block t also clears those of rows t * k .. that are of no slot.
template <class U>
__global__ __launch_bounds__(kRowThreads) void k_dispatch(RowsArgs p)
{
    const int64_t t = blockIdx.x, rows = p.tokens * p.k;
    const U* x = reinterpret_cast<const U*>(p.x) + t * p.x_stride;
    U* out = reinterpret_cast<U*>(p.out);
    const int32_t* to = p.row_of_slot + t * p.k;
    const int32_t* of = p.slot_of_row + t * p.k;
    for (int64_t c = threadIdx.x; c < p.cols; c += kRowThreads) {
        const U v = x[c];
        for (int j = 0; j < p.k; ++j) {
            const int64_t r = to[j];
            if (r >= 0 && r < rows) out[r * p.out_stride + c] = v;
        }
        if (p.zero_rest)
            for (int j = 0; j < p.k; ++j)
                if (of[j] < 0) out[(t * p.k + j) * p.out_stride + c] = U{};
    }
}

template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void k_combine(RowsArgs p)
{
    using P = Piece<DT, WIDE>;
    const int64_t t = blockIdx.x, rows = p.tokens * p.k;
    const int32_t* from = p.row_of_slot + t * p.k;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * P::kValues; c < p.cols;
         c += static_cast<int64_t>(kRowThreads) * P::kValues) {
        float acc[P::kValues] = {};
        for (int j = 0; j < p.k; ++j) {
            const int64_t r = from[j];
            if (r < 0 || r >= rows) continue;
            float v[P::kValues];
            P::load(p.x, r * p.x_stride + c, v);
            const float w = p.weights ? p.weights[t * p.k + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < P::kValues; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
        }
        if (p.add) {
            float v[P::kValues];
            P::load(p.add, t * p.add_stride + c, v);
#pragma unroll
            for (int i = 0; i < P::kValues; ++i) acc[i] += v[i];
        }
        P::store(p.out, t * p.out_stride + c, acc);
    }
}

template <int DT, bool WIDE>
__global__ __launch_bounds__(kRowThreads) void k_combine_backward(RowsArgs p)
{
    using P = Piece<DT, WIDE>;
    constexpr int W = kRowThreads / kWave;
    __shared__ float part[W][kMaxChoices];
    const int64_t t = blockIdx.x, rows = p.tokens * p.k;
    const int tid = static_cast<int>(threadIdx.x);
    const int32_t* from = p.row_of_slot + t * p.k;
    const int32_t* of = p.slot_of_row + t * p.k;
    for (int j = 0; j < p.k; ++j) {
        const int64_t r = from[j];
        const bool has = r >= 0 && r < rows, rest = p.out && of[j] < 0;
        const float w = has && p.out ? p.weights[t * p.k + j] : 0.0f;
        float dot = 0.0f;
        for (int64_t c = static_cast<int64_t>(tid) * P::kValues; c < p.cols;
             c += static_cast<int64_t>(kRowThreads) * P::kValues) {
            float g[P::kValues], v[P::kValues];
            if (has) {
                P::load(p.x, t * p.x_stride + c, g);
                if (p.dweights) {
                    P::load(p.y, r * p.y_stride + c, v);
#pragma unroll
                    for (int i = 0; i < P::kValues; ++i) dot = __builtin_fmaf(g[i], v[i], dot);
                }
                if (p.out) {
#pragma unroll
                    for (int i = 0; i < P::kValues; ++i) g[i] *= w;
                    P::store(p.out, r * p.out_stride + c, g);
                }
            }
            if (rest) {
#pragma unroll
                for (int i = 0; i < P::kValues; ++i) v[i] = 0.0f;
                P::store(p.out, (t * p.k + j) * p.out_stride + c, v);
            }
        }
        dot = wave_sum(dot);
        if ((tid & 63) == 0) part[tid >> 6][j] = dot;
    }
    if (!p.dweights) return;
    __syncthreads();
    if (tid < p.k) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += part[w][tid];
        p.dweights[t * p.k + tid] = sum;
    }
}

}  // namespace

const void* topk_kernel(int dtype)
{
    return dtype == kF32   ? reinterpret_cast<const void*>(k_topk<kF32>)
           : dtype == kF16 ? reinterpret_cast<const void*>(k_topk<kF16>)
                           : reinterpret_cast<const void*>(k_topk<kBF16>);
}
const void* topk_backward_kernel(int dtype)
{
    return dtype == kF32   ? reinterpret_cast<const void*>(k_topk_backward<kF32>)
           : dtype == kF16 ? reinterpret_cast<const void*>(k_topk_backward<kF16>)
                           : reinterpret_cast<const void*>(k_topk_backward<kBF16>);
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
