// zc_moe.hip -- expert routing, and token rows into and out of the per-expert
// chunks that the codec sends (zc_route, zc_expert_slots, zc_dispatch,
// zc_combine and their gradients; the definitions are in zc_ops.h).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "zc_ops.h"
#include "zc_device.h"

namespace {

using namespace zcd;

constexpr int kBlock = 256;
constexpr int kXcds = 8;                           // workgroups go to them in turn
constexpr size_t kLine = 128;                      // bytes of a cache line
constexpr double kKeepBytes = 256 << 20;           // the last-level cache
constexpr uint32_t kMaxGrid = 1u << 20;            // workgroups of a launch; the rest in a loop

// ------------------------------------------------------------------ routing

struct RouteArgs {
    int32_t experts, k, groups, top_groups, per_group;
    uint32_t magic;                                // ceil(2^32 / per_group), 0 for per_group 1
    int32_t softmax, top2, renorm;
    float scale;
};

// e / per_group: the product with the rounded-up reciprocal is exact while
// e per_group < 2^32.
__device__ inline int group_of(const RouteArgs& a, int e)
{
    return a.magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(e), a.magic)) : e;
}

// Keys as unsigned numbers of the same order: 0 is "not to be chosen", 1 a
// NaN, and every number is above them.
__device__ inline uint32_t ordered(float f)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, f);
    const uint32_t u = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return f != f ? 1u : u;
}

__device__ inline float unordered(uint32_t u)
{
    if (u == 1u)
        return __builtin_nanf("");
    return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

template <class T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Run {
    T v[V];
};

// The lane's V logits, -inf past the last expert.
template <class T, int V>
__device__ inline void load_logits(const T* row, int e0, int experts, float (&x)[V])
{
    if (e0 + V <= experts) {
        const Run<T, V> r = *reinterpret_cast<const Run<T, V>*>(row + e0);
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = widen(r.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = e0 + i < experts ? widen(row[e0 + i]) : -__builtin_inff();
    }
}

__device__ inline float sigmoid(float x)
{
    return 1.0f / (1.0f + expf(-x));
}

// What the renormalised weights of a softmax are made of: the exponentials of
// the chosen logits less the largest of them.  The softmax over the chosen
// ones is the chosen scores divided by their sum, but does not vanish with
// them (a bias can choose experts that are far below the token's best).  x is
// -inf for a lane without a choice; one where all are has zeros.
template <int LT, int JN>
__device__ inline void chosen_exponentials(float (&x)[JN])
{
    float top = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < JN; ++q)
        top = fmaxf(top, x[q]);
    top = reduce_max<LT>(top);
#pragma unroll
    for (int q = 0; q < JN; ++q)
        x[q] = x[q] == -__builtin_inff() ? 0.0f : expf(x[q] - top);
}

// Largest logit and fp32-rounded fp64 sum of exponentials of one token, over
// its LT lanes; x becomes the exponentials.
template <int LT, int V>
__device__ inline void softmax_parts(float (&x)[V], float& top, float& sum)
{
    top = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i)
        top = fmaxf(top, x[i]);
    top = reduce_max<LT>(top);
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = expf(x[i] - top);
        d += static_cast<double>(x[i]);
    }
    sum = static_cast<float>(reduce_sum<LT>(d));
}

// Largest and second largest of two such pairs.
__device__ inline void merge_two(uint32_t& first, uint32_t& second, uint32_t f, uint32_t s)
{
    const uint32_t less = first < f ? first : f;
    first = first > f ? first : f;
    second = second > s ? second : s;
    second = second > less ? second : less;
}

// Score of a group from its two largest keys (0 and 0 where it has none).
__device__ inline uint32_t group_score(const RouteArgs& a, uint32_t first, uint32_t second)
{
    return a.top2 && second ? ordered(unordered(first) + unordered(second)) : first;
}

// Changes two keys and their indices round where the second key is larger.
// (By value: a choice between array elements becomes an indexed read.)
__device__ inline void in_order(uint32_t& u0, uint32_t& u1, uint32_t& a0, uint32_t& a1)
{
    const uint32_t ku = u0, kv = u1, ia = a0, ib = a1;
    const bool later = kv > ku;
    u0 = later ? kv : ku;
    u1 = later ? ku : kv;
    a0 = later ? ib : ia;
    a1 = later ? ia : ib;
}

// Lowest set lane of a ballot among the LT lanes from `base` on, from there.
template <int LT>
__device__ inline int lowest_lane(uint64_t b, int base)
{
    if constexpr (LT == 64)
        return __builtin_ctzll(b);
    uint32_t half = base & 32 ? static_cast<uint32_t>(b >> 32) : static_cast<uint32_t>(b);
    if constexpr (LT == 16)
        half = half >> (base & 16) & 0xFFFFu;
    return __builtin_ctz(half);
}

// One token per LT lanes, V neighbouring experts per lane, so that equal keys
// meet in index order: the lowest lane, then its lowest value.  A lane first
// sorts its min(k, V) largest keys to its front (neighbours change places
// only where the later key is larger: equal ones keep their order); each of
// the k rounds is then a maximum over the lanes' first keys and a ballot, and
// the winning lane moves its next key up.
// Bound by its instructions: 880 vector ones per wave of two tokens at 256
// experts, 8 groups and k = 8 (200 of them the exact sigmoids), whose issue
// takes 12.1 us of the 12.5 to 13 that 16384 tokens take; their 17.8 MB would
// take 3.  Softmax without groups takes 12.3 us, at 64 experts and k = 2 4.8,
// at 1024 and k = 8 45.  Four tokens per wave with 16 values per lane: 14.9
// us.  A single token takes 2.6 us at 8 experts, the least a launch takes, and
// 4.2 at 256, for the instructions that it is the first to fetch.  GROUPS: 0
// for none, 1 where a group is a power of two of whole lanes (its two largest
// keys meet in registers), 2 for any other size (through LDS; 23 us where 1
// took 15, 16.9 for 250 experts in 10 groups).
template <class T, int LT, int V, int GROUPS>
__global__ __launch_bounds__(kBlock) void zc_route_kernel(
    const T* __restrict__ logits, int64_t tokens, int64_t stride, RouteArgs a, const float* __restrict__ bias,
    const uint8_t* __restrict__ valid, int32_t* __restrict__ experts, float* __restrict__ weights)
{
    constexpr int TB = kBlock / LT;
    constexpr int JN = (ZC_MAX_TOPK + LT - 1) / LT;
    __shared__ float s_val[TB][LT * V];
    __shared__ uint32_t s_key[GROUPS == 2 ? TB : 1][GROUPS == 2 ? LT * V : 1];
    __shared__ __align__(16) uint32_t s_score[GROUPS ? TB : 1][64];
    __shared__ uint32_t s_allow[GROUPS == 2 ? TB : 1][64];
    __shared__ int32_t s_sel[TB][ZC_MAX_TOPK];

    const int l = threadIdx.x & (LT - 1);
    const int tb = threadIdx.x / LT;
    const int base = threadIdx.x & (kLanes - 1) & ~(LT - 1);   // first lane of the token in its wave
    const int e0 = l * V;

    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB; t0 < tokens;
         t0 += static_cast<int64_t>(gridDim.x) * TB) {
        const bool real = t0 + tb < tokens;
        const int64_t t = real ? t0 + tb : tokens - 1;
        const bool live = real && (!valid || valid[t]);

        float x[V];
        load_logits<T, V>(logits + t * stride, e0, a.experts, x);
        uint32_t out = 0;                                      // bit i: value i may not be chosen
#pragma unroll
        for (int i = 0; i < V; ++i)
            out |= x[i] == -__builtin_inff() ? 1u << i : 0u;
        const bool over_chosen = a.softmax && a.renorm;        // then s_val holds the logits, not the scores
        float sum = 0.0f;
        if (over_chosen)
#pragma unroll
            for (int i = 0; i < V; ++i)
                s_val[tb][e0 + i] = x[i];
        if (a.softmax) {
            float top;
            softmax_parts<LT, V>(x, top, sum);
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = x[i] / sum;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = sigmoid(x[i]);
        }
        if (!over_chosen)
#pragma unroll
            for (int i = 0; i < V; ++i)
                s_val[tb][e0 + i] = x[i];
        if (bias) {
            float b[V];
            load_logits<float, V>(bias, e0, a.experts, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                out |= b[i] == -__builtin_inff() ? 1u << i : 0u;
                x[i] = x[i] + b[i];
            }
        }
        uint32_t u[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            u[i] = out >> i & 1u ? 0u : ordered(x[i]);

        if constexpr (GROUPS == 1) {
            uint32_t first = u[0], second = 0;
#pragma unroll
            for (int i = 1; i < V; ++i)
                merge_two(first, second, u[i], 0);
            const int gl = a.per_group / V;                    // lanes of a group, at most half the token's
            if (gl > 1)
                merge_two(first, second, dpp<kDppXor1>(first), dpp<kDppXor1>(second));
            if (gl > 2)
                merge_two(first, second, dpp<kDppXor2>(first), dpp<kDppXor2>(second));
            if (gl > 4)
                merge_two(first, second, dpp<kDppHalfMirror>(first), dpp<kDppHalfMirror>(second));
            if constexpr (LT > 16)
                if (gl > 8)
                    merge_two(first, second, dpp<kDppMirror>(first), dpp<kDppMirror>(second));
            if constexpr (LT > 32)
                if (gl > 16) {
                    const auto f = __builtin_amdgcn_permlane16_swap(first, first, false, false);
                    const auto s = __builtin_amdgcn_permlane16_swap(second, second, false, false);
                    first = f[0];
                    second = s[0];
                    merge_two(first, second, f[1], s[1]);
                }
            const uint32_t mine = group_score(a, first, second);
            const int g = group_of(a, e0);
            if (l < 4 && a.groups + l < 64)
                s_score[tb][a.groups + l] = 0;                 // the rest of the last four
            if (e0 < a.experts)
                s_score[tb][g] = mine;                         // the group's lanes write one value
            wave_lds_order();
            int rank = 0;
            for (int h = 0; h < a.groups; h += 4) {
                const u32x4 other = *reinterpret_cast<const u32x4*>(&s_score[tb][h]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    rank += other[c] > mine || (other[c] == mine && h + c < g);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                u[i] = rank < a.top_groups ? u[i] : 0u;
        } else if constexpr (GROUPS == 2) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                s_key[tb][e0 + i] = u[i];
            wave_lds_order();
            for (int g = l; g < a.groups; g += LT) {
                uint32_t first = 0, second = 0;
                int i = g % a.per_group;                       // lanes start apart in the banks
                for (int c = 0; c < a.per_group; ++c) {
                    merge_two(first, second, s_key[tb][g * a.per_group + i], 0);
                    i = i + 1 == a.per_group ? 0 : i + 1;
                }
                s_score[tb][g] = group_score(a, first, second);
            }
            wave_lds_order();
            for (int g = l; g < a.groups; g += LT) {
                const uint32_t mine = s_score[tb][g];
                int rank = 0;
                for (int h = 0; h < a.groups; ++h) {
                    const uint32_t other = s_score[tb][h];
                    rank += other > mine || (other == mine && h < g);
                }
                s_allow[tb][g] = rank < a.top_groups;
            }
            wave_lds_order();
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < a.experts && !s_allow[tb][group_of(a, e0 + i)])
                    u[i] = 0;
        }

        uint32_t at[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            at[i] = i;
        // loops of V - 1 steps each, not unrolled further: a wave runs this
        // once, and instructions it has to fetch cost more than a few it need
        // not run
        if (2 * a.k >= V) {
#pragma unroll 1
            for (int p = 0; p < (V + 1) / 2; ++p) {            // odd and even neighbours: sorts all V
#pragma unroll
                for (int i = 0; i + 1 < V; i += 2)
                    in_order(u[i], u[i + 1], at[i], at[i + 1]);
#pragma unroll
                for (int i = 1; i + 1 < V; i += 2)
                    in_order(u[i], u[i + 1], at[i], at[i + 1]);
            }
        } else {
#pragma unroll 1
            for (int p = 0; p < a.k; ++p) {                    // the largest of the rest comes to the front
#pragma unroll
                for (int i = V - 2; i >= 0; --i)
                    in_order(u[i], u[i + 1], at[i], at[i + 1]);
            }
        }
        using Order = std::conditional_t<(V > 8), uint64_t, uint32_t>;
        Order order = 0;                                       // at[], 4 bits each
#pragma unroll
        for (int i = 0; i < V; ++i)
            order |= static_cast<Order>(at[i]) << 4 * i;

        for (int j = 0; j < a.k; ++j) {
            const uint32_t best = reduce_max_u32<LT>(u[0]);
            const int lane = lowest_lane<LT>(__ballot(u[0] == best), base);
            if (l == lane) {
                s_sel[tb][j] = best ? e0 + static_cast<int>(order & 15) : -1;
#pragma unroll
                for (int i = 0; i + 1 < V; ++i)
                    u[i] = u[i + 1];
                u[V - 1] = 0;
                order >>= 4;
            }
        }
        wave_lds_order();

        int32_t e[JN];
        float w[JN];
        float total = 0.0f;
#pragma unroll
        for (int q = 0; q < JN; ++q) {
            const int j = q * LT + l;
            e[q] = j < a.k ? s_sel[tb][j] : -1;
            w[q] = e[q] >= 0 ? s_val[tb][e[q]] : over_chosen ? -__builtin_inff() : 0.0f;
        }
        if (over_chosen)
            chosen_exponentials<LT, JN>(w);
        if (a.renorm) {
#pragma unroll
            for (int q = 0; q < JN; ++q)
                total += w[q];
            total = reduce_sum<LT>(total);
            if (sum != sum)                                    // a NaN or +inf logit, chosen or not
                total = sum;
#pragma unroll
            for (int q = 0; q < JN; ++q)
                w[q] = total == 0.0f || e[q] < 0 ? 0.0f : w[q] / total;
        }
#pragma unroll
        for (int q = 0; q < JN; ++q) {
            const int j = q * LT + l;
            if (real && j < a.k) {
                experts[t * a.k + j] = live ? e[q] : -1;
                weights[t * a.k + j] = live ? a.scale * w[q] : 0.0f;
            }
        }
        wave_lds_order();
    }
}

// Gradient of the weights: the chosen experts' terms, one lane each, go
// through an LDS row to the lanes that store the token's V neighbouring
// values.  Only softmax without renormalisation reads the whole row; with it
// the weights are the softmax over the chosen logits alone.
template <class T, int LT, int V>
__global__ __launch_bounds__(kBlock) void zc_route_grad_kernel(
    const T* __restrict__ logits, int64_t tokens, int64_t stride, RouteArgs a, const int32_t* __restrict__ experts,
    const float* __restrict__ grad, T* __restrict__ out)
{
    constexpr int TB = kBlock / LT;
    constexpr int JN = (ZC_MAX_TOPK + LT - 1) / LT;
    __shared__ float s_row[TB][LT * V];

    const int l = threadIdx.x & (LT - 1);
    const int tb = threadIdx.x / LT;
    const int e0 = l * V;

    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB; t0 < tokens;
         t0 += static_cast<int64_t>(gridDim.x) * TB) {
        const bool real = t0 + tb < tokens;
        const int64_t t = real ? t0 + tb : tokens - 1;
        const T* row = logits + t * stride;

#pragma unroll
        for (int i = 0; i < V; ++i)
            s_row[tb][e0 + i] = 0.0f;
        int32_t e[JN];
        float v[JN], g[JN];
#pragma unroll
        for (int q = 0; q < JN; ++q) {
            const int j = q * LT + l;
            e[q] = j < a.k ? experts[t * a.k + j] : -1;
            if (e[q] >= a.experts)
                e[q] = -1;
            v[q] = e[q] >= 0 ? widen(row[e[q]]) : -__builtin_inff();
            g[q] = e[q] >= 0 ? grad[t * a.k + j] : 0.0f;
        }

        float p[V];
        float dot = 0.0f;
        bool none = false;
        if (a.softmax && !a.renorm) {
            load_logits<T, V>(row, e0, a.experts, p);
            float top, sum;
            softmax_parts<LT, V>(p, top, sum);
            // no gradient where every expert is masked, nor for a token of
            // which none was chosen: its logits may be anything
            uint32_t any = 0;
#pragma unroll
            for (int q = 0; q < JN; ++q)
                any |= e[q] >= 0 ? 1u : 0u;
            none = top == -__builtin_inff() || !reduce_max_u32<LT>(any);
#pragma unroll
            for (int i = 0; i < V; ++i)
                p[i] = p[i] / sum;
#pragma unroll
            for (int q = 0; q < JN; ++q)
                if (e[q] >= 0 && !none)
                    dot += g[q] * (expf(v[q] - top) / sum);
            dot = reduce_sum<LT>(dot);
        } else if (a.softmax) {
            chosen_exponentials<LT, JN>(v);
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < JN; ++q)
                sum += v[q];
            sum = reduce_sum<LT>(sum);
#pragma unroll
            for (int q = 0; q < JN; ++q) {
                v[q] = sum == 0.0f ? 0.0f : v[q] / sum;
                dot += g[q] * v[q];
            }
            dot = reduce_sum<LT>(dot);
#pragma unroll
            for (int q = 0; q < JN; ++q)
                g[q] = v[q] * (g[q] - dot);
        } else {
            // renormalised, ds (1 - s) s is p (1 - s) (g - sum g p) with p = s
            // / S: S may be as small as a number can be, and 1 / S too large
            float rest[JN];                                    // 1 - s, without cancellation
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < JN; ++q) {
                rest[q] = sigmoid(-v[q]);
                v[q] = sigmoid(v[q]);
                sum += v[q];
            }
            if (a.renorm) {
                sum = reduce_sum<LT>(sum);
#pragma unroll
                for (int q = 0; q < JN; ++q) {
                    v[q] = sum == 0.0f ? 0.0f : v[q] / sum;
                    dot += g[q] * v[q];
                }
                dot = reduce_sum<LT>(dot);
            }
#pragma unroll
            for (int q = 0; q < JN; ++q)
                g[q] = v[q] * rest[q] * (g[q] - dot);
        }
        wave_lds_order();
#pragma unroll
        for (int q = 0; q < JN; ++q)
            if (e[q] >= 0)
                s_row[tb][e[q]] = a.scale * g[q];
        wave_lds_order();

        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            d[i] = s_row[tb][e0 + i];
        if (a.softmax && !a.renorm) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                d[i] = none ? 0.0f : p[i] * (d[i] - a.scale * dot);
        }
        if (real) {
            T* to = out + t * a.experts;
            if (e0 + V <= a.experts) {
                Run<T, V> r;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    r.v[i] = static_cast<T>(d[i]);
                *reinterpret_cast<Run<T, V>*>(to + e0) = r;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + i < a.experts)
                        to[e0 + i] = static_cast<T>(d[i]);
            }
        }
        wave_lds_order();
    }
}

// -------------------------------------------------------------------- slots

constexpr int kSlotBlock = 512;
constexpr int kSlotWaves = kSlotBlock / kLanes;
constexpr int kSlotAhead = 4;                      // pairs of a thread loaded at once
// Pairs that one workgroup places alone: 64 experts, 4096 pairs 7.6 us alone
// and in two launches (and 4.5 us less of the host), 2048 4.7 and 7.2, 8192
// 12.8 and 7.9; 1024 experts, 4096 pairs 10.5 and 16.2, 8192 17.1 and 17.6.
constexpr int64_t kSlotOne = 4096;
constexpr int kMaxBins = ZC_MAX_EXPERTS + 1;       // the last bin: pairs without an expert

// Pairs per workgroup, a multiple of its threads, for at most 256 workgroups
// (each reads every other's histogram).
inline int64_t slot_segment(int64_t pairs)
{
    if (pairs <= kSlotOne)
        return (pairs + kSlotBlock - 1) / kSlotBlock * kSlotBlock;
    int64_t s = (pairs + 255) / 256;
    s = s < 2048 ? 2048 : s;
    return (s + kSlotBlock - 1) / kSlotBlock * kSlotBlock;
}

__device__ inline uint32_t bin_of(int32_t e, int32_t experts)
{
    return static_cast<uint32_t>(e) < static_cast<uint32_t>(experts) ? static_cast<uint32_t>(e)
                                                                     : static_cast<uint32_t>(experts);
}

// The bins of up to kSlotAhead pairs per thread, STEP apart, loaded at once
// (~0 past the end).
template <int STEP>
__device__ inline void load_bins(const int32_t* experts, int64_t i, int64_t end, int32_t num,
                                 uint32_t (&bin)[kSlotAhead])
{
    int32_t e[kSlotAhead];
#pragma unroll
    for (int c = 0; c < kSlotAhead; ++c)
        e[c] = i + c * STEP < end ? experts[i + c * STEP] : 0;
#pragma unroll
    for (int c = 0; c < kSlotAhead; ++c)
        bin[c] = i + c * STEP < end ? bin_of(e[c], num) : ~0u;
}

__global__ __launch_bounds__(kSlotBlock) void zc_slot_count_kernel(const int32_t* __restrict__ experts, int64_t pairs,
                                                                   int32_t num, int64_t segment,
                                                                   uint32_t* __restrict__ hist)
{
    __shared__ uint32_t s_hist[kMaxBins];
    const int64_t begin = blockIdx.x * segment;
    const int64_t end = begin + segment < pairs ? begin + segment : pairs;
    uint32_t bin[kSlotAhead];
    load_bins<kSlotBlock>(experts, begin + threadIdx.x, end, num, bin);
    for (int e = threadIdx.x; e <= num; e += kSlotBlock)
        s_hist[e] = 0;
    __syncthreads();
    for (int64_t i = begin + threadIdx.x; i < end;) {
#pragma unroll
        for (int c = 0; c < kSlotAhead; ++c)
            if (bin[c] != ~0u)
                atomicAdd(&s_hist[bin[c]], 1u);
        i += kSlotAhead * kSlotBlock;
        if (i < end)
            load_bins<kSlotBlock>(experts, i, end, num, bin);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= num; e += kSlotBlock)
        hist[static_cast<int64_t>(blockIdx.x) * (num + 1) + e] = s_hist[e];
}

// Stable placement: a workgroup owns a segment of the pairs and a wave a part
// of it, both in order.  A pair's row is the rows of smaller bins, plus those
// of its bin in earlier workgroups (their histograms), in earlier waves, in
// earlier steps of this wave, and in lower lanes (bit-wise ballots of the
// bin).  Integer counts only: the LDS atomics' order cannot show.  Bound by
// its chain of loads, not their size: 65536 pairs take 6.2 us here and 4.7 us
// in the count, 26 pairs 2.8 us.
__global__ __launch_bounds__(kSlotBlock) void zc_slot_place_kernel(const int32_t* __restrict__ experts, int64_t pairs,
                                                                   int32_t num, int64_t segment,
                                                                   const uint32_t* __restrict__ hist,
                                                                   int64_t row_values, int32_t* __restrict__ slots,
                                                                   int64_t* __restrict__ counts)
{
    __shared__ uint32_t s_count[kSlotWaves][kMaxBins];
    __shared__ uint32_t s_before[kMaxBins];        // rows of the bin in earlier workgroups
    __shared__ uint32_t s_base[kMaxBins];          // all rows of the bin, then those of smaller bins
    const int bins = num + 1;
    const int lane = threadIdx.x & (kLanes - 1);
    const int wave = threadIdx.x / kLanes;
    const int64_t part = segment / kSlotWaves;
    const int64_t begin = blockIdx.x * segment + wave * part;
    const int64_t end = begin + part < pairs ? begin + part : pairs;
    uint32_t bin[kSlotAhead];
    load_bins<kLanes>(experts, begin + lane, end, num, bin);

    for (int e = threadIdx.x; e < bins; e += kSlotBlock) {
#pragma unroll
        for (int w = 0; w < kSlotWaves; ++w)
            s_count[w][e] = 0;
        s_before[e] = s_base[e] = 0;
    }
    __syncthreads();
    if (hist) {
        // a wave sums every kSlotWaves-th workgroup's histogram
        for (int e = lane; e < bins; e += kLanes) {
            uint32_t before = 0, total = 0;
            for (uint32_t b0 = wave; b0 < gridDim.x; b0 += 4 * kSlotWaves) {
                uint32_t h[4];
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) {
                    const uint32_t b = b0 + c * kSlotWaves;
                    h[c] = b < gridDim.x ? hist[static_cast<int64_t>(b) * bins + e] : 0u;
                }
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) {
                    before += b0 + c * kSlotWaves < blockIdx.x ? h[c] : 0u;
                    total += h[c];
                }
            }
            if (total) {
                atomicAdd(&s_before[e], before);
                atomicAdd(&s_base[e], total);
            }
        }
    }
    for (int64_t i = begin + lane; i < end;) {
#pragma unroll
        for (int c = 0; c < kSlotAhead; ++c)
            if (bin[c] != ~0u)
                atomicAdd(&s_count[wave][bin[c]], 1u);
        i += kSlotAhead * kLanes;
        if (i < end)
            load_bins<kLanes>(experts, i, end, num, bin);
    }
    __syncthreads();

    for (int e = threadIdx.x; e < bins; e += kSlotBlock) {
        uint32_t run = s_before[e];
#pragma unroll
        for (int w = 0; w < kSlotWaves; ++w) {
            const uint32_t c = s_count[w][e];
            s_count[w][e] = run;
            run += c;
        }
        const uint32_t total = hist ? s_base[e] : run;
        s_base[e] = total;
        if (blockIdx.x == 0)
            counts[e] = static_cast<int64_t>(total) * row_values;
    }
    __syncthreads();

    if (wave == 0) {                               // exclusive scan of the bins' totals
        const int per = (bins + kLanes - 1) / kLanes;
        uint32_t sum = 0;
        for (int i = 0; i < per; ++i)
            sum += lane * per + i < bins ? s_base[lane * per + i] : 0u;
        uint32_t incl = sum;
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) {
            const uint32_t up = __shfl_up(incl, d);
            incl += lane >= d ? up : 0u;
        }
        uint32_t run = incl - sum;
        for (int i = 0; i < per; ++i)
            if (lane * per + i < bins) {
                const uint32_t c = s_base[lane * per + i];
                s_base[lane * per + i] = run;
                run += c;
            }
    }
    __syncthreads();

    const int bits = 32 - __builtin_clz(static_cast<uint32_t>(num));
    if (part > kSlotAhead * kLanes)                // else the bins are still at hand
        load_bins<kLanes>(experts, begin + lane, end, num, bin);
    for (int64_t i0 = begin; i0 < end;) {
#pragma unroll
        for (int c = 0; c < kSlotAhead; ++c) {
            if (i0 + c * kLanes >= end)
                break;
            const uint32_t e = bin[c];
            const bool live = e != ~0u;
            uint64_t same = __ballot(live);
            for (int b = 0; b < bits; ++b) {
                const uint64_t set = __ballot(e >> b & 1u);
                same &= e >> b & 1u ? set : ~set;
            }
            if (live) {
                const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
                const uint32_t at = s_count[wave][e];
                const int32_t row = static_cast<int32_t>(s_base[e] + at + rank);
                slots[i0 + c * kLanes + lane] = e < static_cast<uint32_t>(num) ? row : ~row;
                wave_lds_order();
                if (rank == 0)
                    s_count[wave][e] = at + __popcll(same);
            }
            wave_lds_order();
        }
        i0 += kSlotAhead * kLanes;
        if (i0 < end)
            load_bins<kLanes>(experts, i0 + lane, end, num, bin);
    }
}

// ------------------------------------------------------------- row movement

// Dispatch and combine: a workgroup is one wave, and takes 64 neighbouring
// 16-byte words of one token's row (`parts` of them cover a row, the part
// running fastest).  FLAT: of all rows, a short row's words following the
// last one's (`parts` is then the words of a row), so that no lane is left
// over.  The waves then
// walk through memory in order, which is worth more than long ones: 16384
// rows of 7168 bf16 to 4 slots each take 217 us in waves of one word per
// lane, 236 us in workgroups of 256 threads with the part as the slow index;
// joined again, 190 us against 212 us (in waves of seven words 225 and 214;
// all on one card: others take 211 and 197 in the order that a router gives,
// 224 and 201 over random slots).
// XCD: the parts of a row go to one XCD, whose L2 then holds both halves of
// a cache line that two waves share (workgroups are dealt to the XCDs in
// turn).  A row's last word begins early, in its neighbour's, so that rows of
// any length are moved in whole words.
template <bool FLAT, bool XCD>
struct Place {
    int64_t token, at;                             // token, and the lane's first value of the row
    int skip;                                      // values of the word that its neighbour has
    bool none, whole;                              // nothing to do; the row has a whole word
    __device__ Place(int64_t first, uint32_t parts, int64_t tokens, int64_t values, int n)
    {
        if constexpr (FLAT) {
            const uint32_t block = XCD ? blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds : blockIdx.x;
            const uint32_t word = block * kLanes + threadIdx.x;
            const uint32_t row = word / parts;
            token = first + row;
            at = static_cast<int64_t>(word - row * parts) * n;
        } else {
            const uint32_t seq = XCD ? blockIdx.x / kXcds : blockIdx.x;
            const uint32_t round = seq / parts;
            token = first + (XCD ? round * kXcds + blockIdx.x % kXcds : round);
            at = (static_cast<int64_t>(seq - round * parts) * kLanes + threadIdx.x) * n;
        }
        none = token >= tokens || at >= values;
        whole = values >= n;
        skip = 0;
        if (whole && at + n > values) {
            skip = static_cast<int>(at + n - values);
            at = values - n;
        }
    }
};

// The row a slot names, or -1 where it lies outside the buffer; a negative
// slot is the row of a pair without an expert.
__device__ inline int64_t row_of(int32_t slot, int64_t rows)
{
    const int64_t r = slot < 0 ? ~slot : slot;
    return r < rows ? r : -1;
}

// A row is read once and written k times.  Bound by the writes: 1.17 GB at
// 5.3 TB/s for 16384 rows of 7168 bf16 to 4 random slots each, 5.6 in the
// order that a router gives.  Rows of whole cache lines are written in the order of
// memory, many of them past the L2 (40000 x 1024 to 3 slots: 50 us against 61;
// 24 MB through it 5.8 us, by XCD 6.2); lines that two rows or waves share are
// joined in one L2 first (30000 x 2056 to 6: 185 us against 239, written in
// order past it).
template <class T, bool FLAT, int K, bool XCD, bool STREAM>
__global__ __launch_bounds__(kLanes) void zc_dispatch_kernel(const T* __restrict__ x, int64_t first, int64_t tokens,
                                                             int64_t values, int64_t stride, uint32_t parts,
                                                             const int32_t* __restrict__ slots, int32_t k,
                                                             T* __restrict__ rows)
{
    constexpr int N = Word<T>::N;
    const Place<FLAT, XCD> p(first, parts, tokens, values, N);
    const int64_t t = p.token, at = p.at;
    if (p.none)
        return;
    const T* from = x + t * stride + at;
    if (p.whole) {
        const u32x4 w = load16<false>(from);
        const u32x4 zero = {0, 0, 0, 0};
        for (int j0 = 0; j0 < k; j0 += K) {
            int32_t s[K];
#pragma unroll
            for (int q = 0; q < K; ++q)
                s[q] = slots[t * k + (j0 + q < k ? j0 + q : k - 1)];
#pragma unroll
            for (int q = 0; q < K; ++q) {
                const int64_t r = row_of(s[q], tokens * k);
                if (r >= 0 && j0 + q < k)
                    store16<STREAM>(rows + r * values + at, s[q] < 0 ? zero : w);
            }
        }
    } else {
        for (int j = 0; j < k; ++j) {
            const int32_t s = slots[t * k + j];
            const int64_t r = row_of(s, tokens * k);
            for (int64_t i = 0; r >= 0 && at + i < values; ++i)
                rows[r * values + at + i] = s < 0 ? static_cast<T>(0.0f) : from[i];
        }
    }
}

// K choices at a time: their K loads are issued together.  Bound by the
// reads: 1.17 GB at 5.8 to 6.0 TB/s for 16384 tokens' 4 rows of 7168 bf16 (a
// copy reaches 6.1 to 6.5); rows that end inside a cache line 5.4 (5.1 where
// a row's parts go to different XCDs).
template <class T, bool FLAT, int K, bool STREAM>
__global__ __launch_bounds__(kLanes) void zc_combine_kernel(const T* __restrict__ rows, int64_t first, int64_t tokens,
                                                            int64_t values, uint32_t parts,
                                                            const int32_t* __restrict__ slots, int32_t k,
                                                            const float* __restrict__ weights, const T* base,
                                                            int64_t base_stride, T* out)
{
    constexpr int N = Word<T>::N;
    const Place<FLAT, true> p(first, parts, tokens, values, N);
    const int64_t t = p.token, at = p.at;
    if (p.none)
        return;
    if (p.whole) {
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[i] = 0.0f;
        if (base)
            Word<T>::unpack(load16<STREAM>(base + t * base_stride + at), acc);
        for (int j0 = 0; j0 < k; j0 += K) {
            u32x4 w[K];
            float f[K];
            int32_t slot[K];
            bool has[K];
#pragma unroll
            for (int q = 0; q < K; ++q) {
                const int64_t i = t * k + (j0 + q < k ? j0 + q : k - 1);
                slot[q] = slots[i];
                f[q] = weights ? weights[i] : 1.0f;
            }
#pragma unroll
            for (int q = 0; q < K; ++q) {
                // a pair that adds nothing reads row 0 instead: no load waits
                // for a branch
                has[q] = j0 + q < k && slot[q] >= 0 && slot[q] < tokens * k;
                w[q] = load16<STREAM>(rows + (has[q] ? slot[q] : 0) * values + at);
            }
#pragma unroll
            for (int q = 0; q < K; ++q) {
                float y[N];
                Word<T>::unpack(has[q] ? w[q] : u32x4{0, 0, 0, 0}, y);
                f[q] = has[q] ? f[q] : 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[i] = fmaf(f[q], y[i], acc[i]);
            }
        }
        if (p.skip && out == base) {
            // the neighbour may have written its part of this base already
#pragma unroll
            for (int i = 1; i < N; ++i)
                if (i >= p.skip)
                    out[t * values + at + i] = static_cast<T>(acc[i]);
        } else {
            store16<STREAM>(out + t * values + at, Word<T>::pack(acc));
        }
    } else {
        for (int i = 0; at + i < values; ++i) {
            float sum = base ? widen(base[t * base_stride + at + i]) : 0.0f;
            for (int j = 0; j < k; ++j) {
                const int32_t s = slots[t * k + j];
                if (s >= 0 && s < tokens * k)
                    sum = fmaf(weights ? weights[t * k + j] : 1.0f, widen(rows[s * values + at + i]), sum);
            }
            out[t * values + at + i] = static_cast<T>(sum);
        }
    }
}

// One token per TX threads over its whole row: the token's gradient is read
// once, and its K products with the expert rows stay in registers to the
// row's end.  TX is near the row's words, at most 512 (16384 rows of 7168
// bf16 and 2 choices, in the order that a router gives: 218 us with 512
// threads, 235 us with 1024; over random slots 229 with 512; 30000 rows of
// 2049 and 6 choices: 364 us with 256, 368 us with 512, 405 us with 64).
// KEEP: the rows' gradients are written through the caches.  Loads through
// them too, loads past them, and both past them, in us, by the rows' size:
//               200 values, 3     1024 values, 3    2049 values, 6
//    26 MB       15   18   18      13   14   14      16   18   19
//    90 MB       44   45   58      36   36   40      40   41   50
//   260 MB      147  120  161     113   95  108     124  105  135
//   350 MB      194  205  218     151  150  143     164  175  181
//   700 MB      385  458  438     303  311  293     325  358  360
// Stores past them pay for whole cache lines beyond the 256 MB last-level
// cache alone; the rule below takes them there for all rows.
template <class T, int TX, int K, bool STREAM, bool KEEP>
__global__ __launch_bounds__(TX < kLanes ? kLanes : TX) void zc_combine_grad_kernel(
    const T* __restrict__ grad, int64_t tokens, int64_t values, int64_t stride, const T* __restrict__ rows,
    const int32_t* __restrict__ slots, int32_t k, const float* __restrict__ weights, T* __restrict__ rows_grad,
    float* __restrict__ weights_grad)
{
    constexpr int N = Word<T>::N;
    constexpr int TB = TX < kLanes ? kLanes / TX : 1;
    constexpr int L = TX < kLanes ? TX : kLanes;
    __shared__ float s_part[TX > kLanes ? TX / kLanes : 1][K];
    const int l = threadIdx.x & (TX - 1);
    // every thread of a workgroup takes the same number of turns
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB; t0 < tokens;
         t0 += static_cast<int64_t>(gridDim.x) * TB) {
        const int64_t t = t0 + (TB > 1 ? threadIdx.x / TX : 0);
        const bool real = t < tokens;
        for (int j0 = 0; j0 < k; j0 += K) {
            float dot[K], f[K];
            int32_t slot[K];
            int64_t to[K];                                     // row, -1 for none
            bool has[K];
#pragma unroll
            for (int q = 0; q < K; ++q) {
                const int64_t i = (real ? t : tokens - 1) * k + (j0 + q < k ? j0 + q : k - 1);
                slot[q] = slots[i];
                f[q] = weights[i];
            }
#pragma unroll
            for (int q = 0; q < K; ++q) {
                // a pair without a row reads row 0: no load waits for a branch
                to[q] = real && j0 + q < k ? row_of(slot[q], tokens * k) : -1;
                has[q] = to[q] >= 0 && slot[q] >= 0;
                dot[q] = 0.0f;
            }
            if (real)
                for (int64_t at0 = static_cast<int64_t>(l) * N; at0 < values; at0 += TX * N) {
                    // a row's last word begins early, in its neighbour's
                    const bool over = values >= N && at0 + N > values;
                    const int64_t at = over ? values - N : at0;
                    const T* g = grad + t * stride + at;
                    if (values >= N) {
                        float d[N];
                        u32x4 w[K];
                        const u32x4 gw = load16<STREAM>(g);
#pragma unroll
                        for (int q = 0; q < K; ++q)
                            w[q] = load16<STREAM>(rows + (has[q] ? to[q] : 0) * values + at);
                        Word<T>::unpack(gw, d);
#pragma unroll
                        for (int q = 0; q < K; ++q) {
                            float y[N], o[N];
                            Word<T>::unpack(w[q], y);
#pragma unroll
                            for (int i = 0; i < N; ++i) {
                                dot[q] = !over || at + i >= at0 ? fmaf(d[i], y[i], dot[q]) : dot[q];
                                o[i] = f[q] * d[i];
                            }
                            if (to[q] >= 0)
                                store16<!KEEP>(rows_grad + to[q] * values + at,
                                                has[q] ? Word<T>::pack(o) : u32x4{0, 0, 0, 0});
                        }
                    } else {
                        for (int i = 0; at + i < values; ++i) {
                            const float d = widen(g[i]);
#pragma unroll
                            for (int q = 0; q < K; ++q) {
                                if (has[q])
                                    dot[q] = fmaf(d, widen(rows[to[q] * values + at + i]), dot[q]);
                                if (to[q] >= 0)
                                    rows_grad[to[q] * values + at + i] = static_cast<T>(has[q] ? f[q] * d : 0.0f);
                            }
                        }
                    }
                }
#pragma unroll
            for (int q = 0; q < K; ++q)
                dot[q] = reduce_sum<L>(has[q] ? dot[q] : 0.0f);
            if constexpr (TX > kLanes) {
                __syncthreads();
#pragma unroll
                for (int q = 0; q < K; ++q)
                    if ((threadIdx.x & (kLanes - 1)) == 0)
                        s_part[threadIdx.x / kLanes][q] = dot[q];
                __syncthreads();
                if (threadIdx.x < K) {
                    float sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < TX / kLanes; ++w)
                        sum += s_part[w][threadIdx.x];
                    if (j0 + threadIdx.x < static_cast<unsigned>(k))
                        weights_grad[t * k + j0 + threadIdx.x] = sum;
                }
            } else {
#pragma unroll
                for (int q = 0; q < K; ++q)
                    if (real && j0 + q < k && l == q)
                        weights_grad[t * k + j0 + q] = dot[q];
            }
        }
    }
}

// ---------------------------------------------------------------- launching

int done()
{
    return hipGetLastError() == hipSuccess ? ZC_OK : ZC_EHIP;
}

bool logits_ok(const void* p, int32_t dtype, int64_t tokens, int64_t stride, const zc_router* r)
{
    return elem_bytes(dtype) && tokens >= 0 && r && r->experts >= 1 && r->experts <= ZC_MAX_EXPERTS && r->k >= 1
        && r->k <= ZC_MAX_TOPK && r->k <= r->experts && stride >= 0
        && (r->score == ZC_SCORE_SOFTMAX || r->score == ZC_SCORE_SIGMOID) && (r->renorm == 0 || r->renorm == 1)
        && (tokens == 0 || (p && !misaligned(p, elem_bytes(dtype))));
}

uint32_t grid_for(int64_t tokens, int per_block)
{
    const int64_t b = (tokens + per_block - 1) / per_block;
    return static_cast<uint32_t>(b < kMaxGrid ? b : kMaxGrid);
}

// Rows that dispatch takes FLAT: short ones that leave lanes over (50000 x
// 520 bf16 to 4 slots 45 us against 72 in waves of one row, 768 60 against 65,
// 2000 equal).
bool flat_copies(int64_t words)
{
    return words < 4 * kLanes && words % kLanes != 0;
}

// Rows that combine takes FLAT, where each lane reads its own slots and
// weights: those that leave two lanes in five over or more (50000 x 520 48 us
// against 65, 100000 x 200 with 8 rows 74 against 84; 768 72 against 67).
bool flat_sums(int64_t words)
{
    return words < 4 * kLanes && 5 * words <= 3 * ((words + kLanes - 1) / kLanes * kLanes);
}

// Launches of dispatch and combine: f(first token, workgroups, parts) for as
// many tokens at a time as a grid (and a 32-bit word number) takes.
template <class F>
void over_tokens(int64_t tokens, int64_t words, bool flat, F f)
{
    if (flat) {
        constexpr int64_t kTurn = kXcds * kLanes;              // a multiple of it fills whole turns
        const int64_t most = (1ll << 31) / words / kTurn * kTurn - kTurn;
        for (int64_t t = 0; t < tokens; t += most) {
            const int64_t here = tokens - t < most ? tokens - t : most;
            f(t, static_cast<uint32_t>((here * words + kTurn - 1) / kTurn * kXcds), static_cast<uint32_t>(words));
        }
        return;
    }
    const int64_t parts = (words + kLanes - 1) / kLanes;       // at most 2^20
    const int64_t most = (1ll << 25) / parts / kXcds * kXcds + kXcds;
    for (int64_t t = 0; t < tokens; t += most) {
        const int64_t here = tokens - t < most ? tokens - t : most;
        f(t, static_cast<uint32_t>((here + kXcds - 1) / kXcds * kXcds * parts), static_cast<uint32_t>(parts));
    }
}

// Calls f with a null pointer of the element type.
template <class F>
void with_type(int32_t dtype, F f)
{
    if (dtype == ZC_BF16)
        f(static_cast<__bf16*>(nullptr));
    else if (dtype == ZC_F16)
        f(static_cast<_Float16*>(nullptr));
    else
        f(static_cast<float*>(nullptr));
}

template <int N>
struct Int {
    static constexpr int value = N;
};

// Lanes per token and experts per lane: at least 16 lanes, up to 8 values
// each while the lanes last.
template <class F>
void with_lanes(int32_t experts, F f)
{
    if (experts <= 16)
        f(Int<16>{}, Int<1>{});
    else if (experts <= 32)
        f(Int<16>{}, Int<2>{});
    else if (experts <= 64)
        f(Int<16>{}, Int<4>{});
    else if (experts <= 128)
        f(Int<16>{}, Int<8>{});
    else if (experts <= 256)
        f(Int<32>{}, Int<8>{});
    else if (experts <= 512)
        f(Int<64>{}, Int<8>{});
    else
        f(Int<64>{}, Int<16>{});
}

// Threads per row of combine_grad: the power of two next to its words (see
// there), from 64 to 512, or 16 or 32 lanes where that is enough.
template <class F>
void with_threads(int64_t words, F f)
{
    if (words <= 16)
        f(Int<16>{});
    else if (words <= 32)
        f(Int<32>{});
    else if (5 * words <= 7 * 64)
        f(Int<64>{});
    else if (5 * words <= 7 * 128)
        f(Int<128>{});
    else if (5 * words <= 7 * 256)
        f(Int<256>{});
    else
        f(Int<512>{});
}

template <class F>
void with_bool(bool b, F f)
{
    if (b)
        f(std::true_type{});
    else
        f(std::false_type{});
}

template <class F>
void with_choices(int32_t k, F f)
{
    if (k == 1)
        f(Int<1>{});
    else if (k == 2)
        f(Int<2>{});
    else if (k <= 4)
        f(Int<4>{});
    else
        f(Int<8>{});
}

// What dispatch, combine and their gradients ask of their sizes.
bool rows_ok(int32_t dtype, int64_t tokens, int64_t values, int32_t k)
{
    return elem_bytes(dtype) && tokens >= 0 && values >= 0 && values <= ZC_MAX_ROW_VALUES && k >= 1
        && k <= ZC_MAX_TOPK && tokens * static_cast<__int128>(k) <= 0x7FFFFFFF;
}

// Whether a call that moves `rows` rows per token streams past the caches.
bool stream_past(int64_t tokens, int64_t values, int rows, size_t bytes)
{
    return static_cast<double>(tokens) * values * rows * bytes > kStreamBytes;
}

}  // namespace

extern "C" {

int zc_route(const void* d_logits, int32_t dtype, int64_t tokens, int64_t row_stride, const zc_router* router,
             const float* d_bias, const uint8_t* d_valid, int32_t* d_experts, float* d_weights, void* stream)
{
    if (!logits_ok(d_logits, dtype, tokens, row_stride, router))
        return ZC_EINVAL;
    const zc_router& r = *router;
    if (r.groups < 1 || r.groups > 64 || r.experts % r.groups || r.top_groups < 1 || r.top_groups > r.groups
        || r.k > r.top_groups * (r.experts / r.groups)
        || (r.group_score != ZC_GROUP_MAX && r.group_score != ZC_GROUP_TOP2))
        return ZC_EINVAL;
    if (misaligned(d_bias, 4) || misaligned(d_experts, 4) || misaligned(d_weights, 4))
        return ZC_EINVAL;
    if (tokens == 0)
        return ZC_OK;
    if (!d_experts || !d_weights)
        return ZC_EINVAL;
    RouteArgs a;
    a.experts = r.experts;
    a.k = r.k;
    a.groups = r.groups;
    a.top_groups = r.top_groups;
    a.per_group = r.experts / r.groups;
    a.magic = static_cast<uint32_t>((0xFFFFFFFFull + a.per_group) / a.per_group);   // 2^32 wraps to 0
    a.softmax = r.score == ZC_SCORE_SOFTMAX;
    a.top2 = r.group_score == ZC_GROUP_TOP2;
    a.renorm = r.renorm;
    a.scale = r.scale;
    // every group taking part is the same as no groups
    const bool groups = r.top_groups < r.groups;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        with_lanes(r.experts, [&](auto lanes, auto each) {
            constexpr int LT = decltype(lanes)::value, V = decltype(each)::value;
            const dim3 grid(grid_for(tokens, kBlock / LT));
            const T* x = static_cast<const T*>(d_logits);
            const int gl = a.per_group / V;
            if (!groups)
                hipLaunchKernelGGL((zc_route_kernel<T, LT, V, 0>), grid, dim3(kBlock), 0, s, x, tokens, row_stride, a,
                                   d_bias, d_valid, d_experts, d_weights);
            else if (a.per_group % V == 0 && (gl & (gl - 1)) == 0)
                hipLaunchKernelGGL((zc_route_kernel<T, LT, V, 1>), grid, dim3(kBlock), 0, s, x, tokens, row_stride, a,
                                   d_bias, d_valid, d_experts, d_weights);
            else
                hipLaunchKernelGGL((zc_route_kernel<T, LT, V, 2>), grid, dim3(kBlock), 0, s, x, tokens, row_stride, a,
                                   d_bias, d_valid, d_experts, d_weights);
        });
    });
    return done();
}

int zc_route_grad(const void* d_logits, int32_t dtype, int64_t tokens, int64_t row_stride, const zc_router* router,
                  const int32_t* d_experts, const float* d_weights_grad, void* d_logits_grad, void* stream)
{
    if (!logits_ok(d_logits, dtype, tokens, row_stride, router) || misaligned(d_experts, 4)
        || misaligned(d_weights_grad, 4) || misaligned(d_logits_grad, elem_bytes(dtype)))
        return ZC_EINVAL;
    if (tokens == 0)
        return ZC_OK;
    if (!d_experts || !d_weights_grad || !d_logits_grad)
        return ZC_EINVAL;
    const zc_router& r = *router;
    RouteArgs a{};
    a.experts = r.experts;
    a.k = r.k;
    a.softmax = r.score == ZC_SCORE_SOFTMAX;
    a.renorm = r.renorm;
    a.scale = r.scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        with_lanes(r.experts, [&](auto lanes, auto each) {
            constexpr int LT = decltype(lanes)::value, V = decltype(each)::value;
            hipLaunchKernelGGL((zc_route_grad_kernel<T, LT, V>), dim3(grid_for(tokens, kBlock / LT)), dim3(kBlock), 0,
                               s, static_cast<const T*>(d_logits), tokens, row_stride, a, d_experts, d_weights_grad,
                               static_cast<T*>(d_logits_grad));
        });
    });
    return done();
}

size_t zc_slots_workspace_bytes(int64_t pairs, int32_t experts)
{
    if (pairs < 0 || pairs > 0x7FFFFFFF || experts < 1 || experts > ZC_MAX_EXPERTS || pairs <= kSlotOne)
        return 0;
    const int64_t seg = slot_segment(pairs);
    return static_cast<size_t>((pairs + seg - 1) / seg) * (experts + 1) * 4;
}

int zc_expert_slots(const int32_t* d_experts, int64_t pairs, int32_t experts, int64_t row_values, int32_t* d_slots,
                    int64_t* d_counts, void* d_ws, size_t ws_bytes, void* stream)
{
    if (pairs < 0 || pairs > 0x7FFFFFFF || experts < 1 || experts > ZC_MAX_EXPERTS || row_values < 0
        || row_values > ZC_MAX_CHUNK_VALUES || !d_counts || (pairs && (!d_experts || !d_slots)))
        return ZC_EINVAL;
    const size_t need = zc_slots_workspace_bytes(pairs, experts);
    if (misaligned(d_experts, 4) || misaligned(d_slots, 4) || misaligned(d_counts, 8) || misaligned(d_ws, 4)
        || (need && !d_ws))
        return ZC_EINVAL;
    if (ws_bytes < need)
        return ZC_ENOSPC;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t seg = pairs ? slot_segment(pairs) : kSlotBlock;
    const uint32_t blocks = pairs ? static_cast<uint32_t>((pairs + seg - 1) / seg) : 1u;
    uint32_t* hist = need ? static_cast<uint32_t*>(d_ws) : nullptr;
    if (hist) {
        hipLaunchKernelGGL(zc_slot_count_kernel, dim3(blocks), dim3(kSlotBlock), 0, s, d_experts, pairs, experts, seg,
                           hist);
        if (hipGetLastError() != hipSuccess)
            return ZC_EHIP;
    }
    hipLaunchKernelGGL(zc_slot_place_kernel, dim3(blocks), dim3(kSlotBlock), 0, s, d_experts, pairs, experts, seg,
                       hist, row_values, d_slots, d_counts);
    return done();
}

int zc_dispatch(const void* d_x, int32_t dtype, int64_t tokens, int64_t row_values, int64_t row_stride,
                const int32_t* d_slots, int32_t k, void* d_rows, void* stream)
{
    if (!rows_ok(dtype, tokens, row_values, k) || row_stride < 0)
        return ZC_EINVAL;
    const size_t b = elem_bytes(dtype);
    if (misaligned(d_x, b) || misaligned(d_rows, b) || misaligned(d_slots, 4))
        return ZC_EINVAL;
    if (tokens == 0 || row_values == 0)
        return ZC_OK;
    if (!d_x || !d_slots || !d_rows)
        return ZC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        const int64_t words = (row_values + Word<T>::N - 1) / Word<T>::N;
        const bool lines = (row_values * b) % kLine == 0 && !misaligned(d_rows, kLine);
        const bool past = lines && stream_past(tokens, row_values, k + 1, b);
        with_bool(flat_copies(words), [&](auto flat) {
            with_choices(k, [&](auto choices) {
                constexpr bool F = decltype(flat)::value;
                constexpr int K = decltype(choices)::value;
                over_tokens(tokens, words, F, [&](int64_t first, uint32_t blocks, uint32_t parts) {
                    const auto launch = [&](auto kernel) {
                        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kLanes), 0, s, static_cast<const T*>(d_x),
                                           first, tokens, row_values, row_stride, parts, d_slots, k,
                                           static_cast<T*>(d_rows));
                    };
                    if (past)
                        launch(zc_dispatch_kernel<T, F, K, false, true>);
                    else if (lines)
                        launch(zc_dispatch_kernel<T, F, K, false, false>);
                    else
                        launch(zc_dispatch_kernel<T, F, K, true, false>);
                });
            });
        });
    });
    return done();
}

int zc_combine(const void* d_rows, int32_t dtype, int64_t tokens, int64_t row_values, const int32_t* d_slots,
               int32_t k, const float* d_weights, const void* d_base, int64_t base_stride, void* d_out, void* stream)
{
    if (!rows_ok(dtype, tokens, row_values, k) || (d_base && base_stride < 0))
        return ZC_EINVAL;
    const size_t b = elem_bytes(dtype);
    if (misaligned(d_rows, b) || misaligned(d_base, b) || misaligned(d_out, b) || misaligned(d_slots, 4)
        || misaligned(d_weights, 4))
        return ZC_EINVAL;
    if (tokens == 0 || row_values == 0)
        return ZC_OK;
    if (!d_rows || !d_slots || !d_out)
        return ZC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        const int64_t words = (row_values + Word<T>::N - 1) / Word<T>::N;
        with_bool(flat_sums(words), [&](auto flat) {
            with_choices(k, [&](auto choices) {
                with_bool(stream_past(tokens, row_values, k + (d_base ? 2 : 1), b), [&](auto past) {
                    constexpr bool F = decltype(flat)::value;
                    constexpr int K = decltype(choices)::value;
                    over_tokens(tokens, words, F, [&](int64_t first, uint32_t blocks, uint32_t parts) {
                        hipLaunchKernelGGL((zc_combine_kernel<T, F, K, decltype(past)::value>), dim3(blocks),
                                           dim3(kLanes), 0, s, static_cast<const T*>(d_rows), first, tokens,
                                           row_values, parts, d_slots, k, d_weights,
                                           static_cast<const T*>(d_base), base_stride, static_cast<T*>(d_out));
                    });
                });
            });
        });
    });
    return done();
}

int zc_combine_grad(const void* d_out_grad, int32_t dtype, int64_t tokens, int64_t row_values, int64_t row_stride,
                    const void* d_rows, const int32_t* d_slots, int32_t k, const float* d_weights, void* d_rows_grad,
                    float* d_weights_grad, void* stream)
{
    if (!rows_ok(dtype, tokens, row_values, k) || row_stride < 0)
        return ZC_EINVAL;
    const size_t b = elem_bytes(dtype);
    if (misaligned(d_out_grad, b) || misaligned(d_rows, b) || misaligned(d_rows_grad, b) || misaligned(d_slots, 4)
        || misaligned(d_weights, 4) || misaligned(d_weights_grad, 4))
        return ZC_EINVAL;
    if (tokens == 0)
        return ZC_OK;
    if (!d_slots || !d_weights || !d_weights_grad || (row_values && (!d_out_grad || !d_rows || !d_rows_grad)))
        return ZC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        const int64_t words = (row_values + Word<T>::N - 1) / Word<T>::N;
        const bool keep = static_cast<double>(tokens) * k * row_values * b <= kKeepBytes;
        with_threads(words, [&](auto threads) {
            with_choices(k, [&](auto choices) {
                with_bool(stream_past(tokens, row_values, 2 * k + 1, b), [&](auto past) {
                    constexpr int TX = decltype(threads)::value, K = decltype(choices)::value;
                    constexpr int BL = TX < kLanes ? kLanes : TX;
                    constexpr bool P = decltype(past)::value;
                    const auto launch = [&](auto kernel) {
                        hipLaunchKernelGGL(kernel, dim3(grid_for(tokens, BL / TX)), dim3(BL), 0, s,
                                           static_cast<const T*>(d_out_grad), tokens, row_values, row_stride,
                                           static_cast<const T*>(d_rows), d_slots, k, d_weights,
                                           static_cast<T*>(d_rows_grad), d_weights_grad);
                    };
                    if (P && !keep)
                        launch(zc_combine_grad_kernel<T, TX, K, P, !P>);
                    else
                        launch(zc_combine_grad_kernel<T, TX, K, P, true>);
                });
            });
        });
    });
    return done();
}

}  // extern "C"
