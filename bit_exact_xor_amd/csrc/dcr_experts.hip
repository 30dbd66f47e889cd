// dcr_experts.hip -- the choice of experts, its gradient, and the order of the
// chosen (token, expert) pairs.
//
// A row of logits lies in the registers of 8 to 64 lanes of a wave, eight
// consecutive ones (or twice eight) a lane, so several rows share a wave and
// nothing of a row leaves it but what is written.  The choice is made as in 64
// bits: the scores of experts next to one another often differ by less than
// the rounding of 32, and a choice that depended on it would differ from one
// program to the next.
#include <algorithm>

#include "dcr_step.h"

namespace dcr {
namespace {

constexpr uint32_t kET = 256;                     // threads of a workgroup

struct SelectArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    const float* dweights;    // gradient
    void* dlogits;
    uint64_t stride, d_stride;
    uint32_t rows, experts, k, groups, top_groups, sigmoid, renormalize;
    uint32_t wide, group_log2;      // the choice in 64 bits at once; else a group is 8 << group_log2 experts
    float scale;
};

// order of numbers as that of unsigned integers; NaN in front of all, and
// 0 for what may not be chosen
__device__ __forceinline__ uint64_t rank_of(double c) {
    if (c != c) return ~uint64_t(0);
    const uint64_t b = uint64_t(__double_as_longlong(c + 0.0));
    return b ^ (uint64_t(int64_t(b) >> 63) | (uint64_t(1) << 63));
}
__device__ __forceinline__ uint32_t rank_of(float c) {
    if (c != c) return ~0u;
    const uint32_t b = __float_as_uint(c + 0.0f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_rank(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// LDS of one wave: its accesses are in order, the compiler has to keep them so
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int LANES, typename T>
__device__ __forceinline__ T lanes_max(T v) {
    return lanes_all<LANES>(v, [](T a, T b) { return (b > a || b != b) ? b : a; });     // (a NaN stays)
}

// A lane's logits: element 8 * (lane + LANES * r) + i of the row is v[8 r + i];
// -infinity behind the end.
template <typename T, int LANES, int R>
__device__ __forceinline__ void load_row(const T* row, uint32_t lane, uint32_t n, float* v) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t c = 8 * (lane + LANES * r);
        const int some = c < n ? int(min(8u, n - c)) : 0;
        Raw8<T> raw;
        if (some == 8)
            raw.load(row + c);
        else
            raw.load_some(row + c, some, kBf16MinusInf);
        raw.get(v + 8 * r);
    }
}
template <int LANES>
__device__ __forceinline__ uint32_t expert_of(uint32_t lane, int i) {
    return 8 * (lane + LANES * (i / 8)) + i % 8;
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// The k largest ranks of a row, one after the other, 0 taking no part; a lane
// keeps every LANES-th.  `seen` gets each round's rank, then that of what would
// come next.
template <int LANES, int N, typename U, typename F>
__device__ __forceinline__ void take_best(U* rank, uint32_t lane, uint32_t k, int32_t* id, F&& seen) {
    constexpr int KEEP = DCR_EXPERTS_MAX_K / LANES;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) id[q] = -1;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        for (uint32_t j = q * LANES; j < min(k, uint32_t(q + 1) * LANES); ++j) {
            U mine = rank[0];
#pragma unroll
            for (int i = 1; i < N; ++i) mine = max(mine, rank[i]);
            const U best = lanes_all<LANES>(mine, [](U a, U b) { return max(a, b); });
            seen(best);
            uint32_t at = ~0u;
#pragma unroll
            for (int i = N - 1; i >= 0; --i) at = rank[i] == best ? expert_of<LANES>(lane, i) : at;
            at = lanes_all<LANES>(at, [](uint32_t a, uint32_t b) { return min(a, b); });
#pragma unroll
            for (int i = 0; i < N; ++i) rank[i] = expert_of<LANES>(lane, i) == at ? U(0) : rank[i];
            if (j - q * LANES == lane) id[q] = best ? int32_t(at) : -1;
        }
    }
    U mine = rank[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mine = max(mine, rank[i]);
    seen(lanes_all<LANES>(mine, [](U a, U b) { return max(a, b); }));
}

// The same where each lane first sorts its eight (28 steps of neighbours, which
// leave equals in their order): a round then is a maximum and a minimum over the
// heads of the lanes' lists, and the lane that had the best moves up.  About 30
// instructions a round where searching eight took 79.
template <int LANES, typename F>
__device__ __forceinline__ void take_sorted(uint32_t* rank, uint32_t lane, uint32_t k, int32_t* id, F&& seen) {
    constexpr int KEEP = DCR_EXPERTS_MAX_K / LANES;
    uint32_t at[8], order = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) at[i] = uint32_t(i);
#pragma unroll
    for (int last = 7; last > 0; --last) {
#pragma unroll
        for (int i = 0; i < last; ++i) {
            const bool swap = rank[i] < rank[i + 1];
            const uint32_t x = rank[i], y = at[i];
            rank[i] = max(x, rank[i + 1]);
            rank[i + 1] = min(x, rank[i + 1]);
            at[i] = swap ? at[i + 1] : y;
            at[i + 1] = swap ? y : at[i + 1];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) order |= at[i] << (4 * i);
#pragma unroll
    for (int q = 0; q < KEEP; ++q) id[q] = -1;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        for (uint32_t j = q * LANES; j < min(k, uint32_t(q + 1) * LANES); ++j) {
            const uint32_t best = lanes_all<LANES>(rank[0], [](uint32_t a, uint32_t b) { return max(a, b); });
            seen(best);
            const uint32_t mine = 8 * lane + (order & 7u);
            const uint32_t e = lanes_all<LANES>(rank[0] == best ? mine : ~0u, [](uint32_t a, uint32_t b) { return min(a, b); });
            const bool won = e == mine;
#pragma unroll
            for (int i = 0; i < 7; ++i) rank[i] = won ? rank[i + 1] : rank[i];
            rank[7] = won ? 0 : rank[7];
            order = won ? order >> 4 : order;
            if (j - q * LANES == lane) id[q] = best ? int32_t(e) : -1;
        }
    }
    seen(lanes_all<LANES>(rank[0], [](uint32_t a, uint32_t b) { return max(a, b); }));
}

// The choice in 64 bits, through LDS where there are groups (the row's values
// and its groups' ranks).
template <int LANES, int N>
__device__ __forceinline__ void choose64(const SelectArgs& a, const float* v, const float* bias, float top, double* lds,
                                         uint32_t lane, int32_t* id) {
    const bool grouped = a.top_groups < a.groups;
    double sum = 1.0;
    if (!a.sigmoid) {
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) z += exp(double(v[i]) - double(top));
        sum = lanes_sum<LANES>(z);
        if (sum == 0.0) sum = 1.0;
    }
    uint64_t rank[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t e = expert_of<LANES>(lane, i);
        double c = double(v[i]);               // without a bias the logits have the order of the scores
        if (a.bias || grouped) {
            c = a.sigmoid ? sigmoid64(c) : exp(c - double(top)) / sum;
            c += double(bias[i]);
            if (grouped && e < a.experts) lds[e] = v[i] == -INFINITY ? -INFINITY : c;
            if (!a.bias) c = double(v[i]);
        }
        rank[i] = v[i] == -INFINITY ? 0 : rank_of(c);
    }
    if (grouped) {
        uint64_t* of_group = reinterpret_cast<uint64_t*>(lds + a.experts);
        const uint32_t size = a.experts / a.groups;
        wave_sync();
        for (uint32_t g = lane; g < a.groups; g += LANES) {
            double first = -INFINITY, second = -INFINITY;
            bool odd = false;
            for (uint32_t i = 0; i < size; ++i) {
                const double c = lds[g * size + i];
                odd |= c != c;
                second = c > first ? first : c > second ? c : second;
                first = c > first ? c : first;
            }
            of_group[g] = odd ? ~uint64_t(0) : first == -INFINITY ? 0 : rank_of(second == -INFINITY ? first : first + second);
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t e = expert_of<LANES>(lane, i);
            if (e >= a.experts) continue;
            const uint32_t mine = e / size;
            const uint64_t r = of_group[mine];
            uint32_t ahead = 0;
            for (uint32_t g = 0; g < a.groups; ++g) ahead += (of_group[g] > r || (of_group[g] == r && g < mine)) ? 1u : 0u;
            if (ahead >= a.top_groups) rank[i] = 0;
        }
    }
    take_best<LANES, N>(rank, lane, a.k, id, [](uint64_t) {});
}

// The same in 32 bits, for groups of a power of two of lanes; false where two
// values that decide are closer than they are certain.  A sigmoid by the
// hardware's exponential and reciprocal (one step off each) is off by less than
// 2.3 * 2^-23 and a sum with the bias by 2^-24 of itself; a softmax's sum of up
// to 1024 terms adds less than 2^-20 of a score.  So `off` bounds a value's error,
// and two values 2 `off` apart (groups: sums of two, 5 `off`) are in order.
template <int LANES, int N>
__device__ __forceinline__ bool choose32(const SelectArgs& a, const float* v, const float* bias, float top, uint32_t lane,
                                         int32_t* id) {
    constexpr float kLog2e = 1.44269504088896340736f;
    const bool grouped = a.top_groups < a.groups;
    float c[N];
    uint32_t rank[N];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < N; ++i) odd |= v[i] != v[i];
    const float off = a.sigmoid ? 0x1p-21f : 0x1p-20f;
    const auto apart = [](uint32_t hi, uint32_t lo, float by) {
        const float x = of_rank(hi), y = of_rank(lo);
        return lo == 0 || x - y > by * fmaxf(1.0f, fabsf(x));
    };
    if (a.bias || grouped) {
        float inv = 1.0f;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v[i]));
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) z += c[i] = __builtin_amdgcn_exp2f((v[i] - top) * kLog2e);
            z = lanes_sum<LANES>(z);
            inv = z == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(z);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            c[i] = v[i] == -INFINITY ? -INFINITY : __fmaf_rn(c[i], inv, bias[i]);
            odd |= c[i] != c[i];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) rank[i] = v[i] == -INFINITY ? 0 : rank_of(a.bias ? c[i] : v[i]);
    if (grouped) {
        float first = -INFINITY, second = -INFINITY;
        const auto meet = [&](float f, float s) {
            second = fmaxf(fminf(first, f), fmaxf(second, s));
            first = fmaxf(first, f);
        };
#pragma unroll
        for (int i = 0; i < N; ++i) meet(c[i], -INFINITY);
        const auto fold = [&](auto step) {
            constexpr int S = decltype(step)::value;
            if constexpr (S < LANES) {
                if ((1u << a.group_log2) > S) {
                    float f[2], s[2];
                    partners_of<S>(first, &f[0], &f[1]);
                    partners_of<S>(second, &s[0], &s[1]);
                    first = f[0], second = s[0];
                    meet(f[1], s[1]);
                }
            }
        };
        fold(std::integral_constant<int, 1>()), fold(std::integral_constant<int, 2>()), fold(std::integral_constant<int, 4>());
        fold(std::integral_constant<int, 8>()), fold(std::integral_constant<int, 16>()), fold(std::integral_constant<int, 32>());
        const uint32_t of = first == -INFINITY ? 0 : rank_of(second == -INFINITY ? first : first + second);
        const uint32_t mine = lane >> a.group_log2, base = threadIdx.x & 63u & ~uint32_t(LANES - 1);
        uint32_t ahead = 0;
        for (uint32_t g = 0; g < a.groups; ++g) {
            const uint32_t o = uint32_t(__shfl(int(of), int(base + (g << a.group_log2)), 64));
            ahead += (o > of || (o == of && g < mine)) ? 1u : 0u;
        }
        const bool in = ahead < a.top_groups;      // (lanes behind the last group are shut, and last)
        const uint32_t least = lanes_all<LANES>(in && mine < a.groups ? of : ~0u, [](uint32_t x, uint32_t y) { return min(x, y); });
        const uint32_t most = lanes_all<LANES>(in ? 0u : of, [](uint32_t x, uint32_t y) { return max(x, y); });
        odd |= !apart(least, most, 5 * off);
#pragma unroll
        for (int i = 0; i < N; ++i) rank[i] = in ? rank[i] : 0;
    }
    uint32_t before = 0;
    bool sure = true;
    const auto seen = [&](uint32_t best) {
        if (a.bias && before) sure &= apart(before, best, 2 * off);
        before = best;
    };
    if constexpr (N == 8)
        take_sorted<LANES>(rank, lane, a.k, id, seen);
    else
        take_best<LANES, N>(rank, lane, a.k, id, seen);
    return sure && !odd;
}

template <typename T, int LANES, int R>
__global__ void __launch_bounds__(kET) experts_select_kernel(SelectArgs a) {
    constexpr int N = 8 * R, ROWS = kET / LANES, KEEP = DCR_EXPERTS_MAX_K / LANES;
    extern __shared__ double values[];         // with groups: a row's values, then its groups' ranks
    const uint32_t lane = threadIdx.x % LANES, in_wg = threadIdx.x / LANES;
    const uint32_t at = blockIdx.x * ROWS + in_wg;
    const bool live = at < a.rows;
    const T* row = static_cast<const T*>(a.logits) + uint64_t(live ? at : 0) * a.stride;
    float v[N], bias[N];
    load_row<T, LANES, R>(row, lane, a.experts, v);
    if (a.bias) {
        load_row<float, LANES, R>(a.bias, lane, a.experts, bias);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) bias[i] = 0.0f;
    }
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = (v[i] > top || v[i] != v[i]) ? v[i] : top;
    top = lanes_max<LANES>(top);
    if (top == -INFINITY) top = 0.0f;          // every expert is shut
    int32_t id[KEEP];
    const bool sure = !a.wide && choose32<LANES, N>(a, v, bias, top, lane, id);
    if (__any(!sure)) choose64<LANES, N>(a, v, bias, top, values + in_wg * (a.experts + a.groups), lane, id);

    // the weights in 64 bits: a few exponentials a row
    double sum = 1.0;
    if (!a.sigmoid && !a.renormalize) {
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) z += exp(double(v[i]) - double(top));
        sum = lanes_sum<LANES>(z);
        if (sum == 0.0) sum = 1.0;
    }
    double w[KEEP], all = 0.0;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        w[q] = 0.0;
        if (id[q] >= 0) {
            const double l = double(wide(row[id[q]]));
            w[q] = a.sigmoid ? sigmoid64(l) : exp(l - double(top));
        }
        all += w[q];
    }
    if (a.renormalize) {
        sum = lanes_sum<LANES>(all);
        if (sum == 0.0) sum = 1.0;
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        const uint32_t j = q * LANES + lane;
        if (j >= a.k) continue;
        a.ids[uint64_t(at) * a.k + j] = id[q];
        a.weights[uint64_t(at) * a.k + j] = float(w[q] / sum * double(a.scale));
    }
}

// The gradient.  With w_j = scale s_j / W (W: the chosen scores' sum, or 1)
//   ds_j = scale (dw_j - [renormalised] sum dw s / W) / W
//   dl   = s (1 - s) ds  or, of a softmax, s (ds - sum ds s), a sum that is
//          zero where the weights are renormalised
// A lane has the pairs j = lane, lane + LANES, ..., whose logits it fetches.
template <typename T, int LANES, int R>
__global__ void __launch_bounds__(kET) experts_select_grad_kernel(SelectArgs a) {
    constexpr int N = 8 * R, ROWS = kET / LANES, KEEP = DCR_EXPERTS_MAX_K / LANES;
    const uint32_t lane = threadIdx.x % LANES, at = blockIdx.x * ROWS + threadIdx.x / LANES;
    const bool live = at < a.rows;
    const uint64_t safe = live ? at : 0;
    const T* row = static_cast<const T*>(a.logits) + safe * a.stride;
    float v[N], d[N];
    load_row<T, LANES, R>(row, lane, a.experts, v);
    uint32_t id[KEEP];
    float dw[KEEP], s[KEEP];
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        const uint32_t j = q * LANES + lane;
        id[q] = ~0u, dw[q] = s[q] = 0.0f;
        if (j < a.k) {
            const uint32_t e = uint32_t(a.ids[safe * a.k + j]);
            if (e < a.experts) id[q] = e, dw[q] = a.dweights[safe * a.k + j], s[q] = wide(row[e]);
        }
    }
    float top = 0.0f, inv = 1.0f;
    if (!a.sigmoid) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = (v[i] > top || v[i] != v[i]) ? v[i] : top;
        top = lanes_max<LANES>(top);
        if (top == -INFINITY) top = 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) z += d[i] = expf(v[i] - top);
        z = lanes_sum<LANES>(z);
        inv = z == 0.0f ? 0.0f : 1.0f / z;
    }
    // the row's scalars in 64 bits: dw and its mean are often nearly the same
    double all = 0.0, dot = 0.0;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        if (id[q] == ~0u) continue;
        s[q] = a.sigmoid ? 1.0f / (1.0f + expf(-s[q])) : expf(s[q] - top) * inv;
        all += double(s[q]);
        dot += double(dw[q]) * double(s[q]);
    }
    dot = lanes_sum<LANES>(dot);
    double over = double(a.scale), mean = 0.0;     // scale / W, and what the renormalisation takes off dw
    if (a.renormalize) {
        all = lanes_sum<LANES>(all);
        if (all == 0.0) all = 1.0;
        over /= all;
        mean = dot / all;
    }
    const float off = a.sigmoid || a.renormalize ? 0.0f : float(dot * over);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (a.sigmoid) {
            const float q = expf(-fabsf(v[i]));    // s (1 - s) = q / (1 + q)^2
            v[i] = q / ((1.0f + q) * (1.0f + q));
        } else {
            v[i] = d[i] * inv;
        }
        d[i] = -off;
    }
    const int base = int(threadIdx.x & 63u & ~uint32_t(LANES - 1));
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        if (uint32_t(q) * LANES >= a.k) break;
        const float ds = float((double(dw[q]) - mean) * over);
        for (uint32_t j = 0; j < min(uint32_t(LANES), a.k - q * LANES); ++j) {
            const uint32_t e = uint32_t(__shfl(int(id[q]), base + int(j), 64));
            const float of = __shfl(ds, base + int(j), 64);
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] += expert_of<LANES>(lane, i) == e ? of : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] *= v[i];
    if (!live) return;
    T* out = static_cast<T*>(a.dlogits) + uint64_t(at) * a.d_stride;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t c = 8 * (lane + LANES * r);
        if (c >= a.experts) continue;
        const int n = int(min(8u, a.experts - c));
        n == 8 ? store8(out + c, d + 8 * r) : store_some(out + c, d + 8 * r, n);
    }
}

// ------------------------------------------------------------------- order
//
// A counting sort by expert that keeps the order of pairs.  Each workgroup has
// a run of pairs; the first launch counts each run's experts, the second adds
// the runs in front, and every wave places its part of a run by ranks among
// 64 pairs at a time (ballots over the bits of the expert).  No atomics decide
// anything, so slots depend on the ids alone.

constexpr uint32_t kOT = 512, kOWaves = kOT / 64;
constexpr uint32_t kOrderRuns = 128;              // at most

struct OrderArgs {
    const int32_t* ids;
    int32_t* offsets;
    int32_t* slots;
    uint32_t* counts;         // [runs][experts]
    uint32_t n, experts, bits, runs, per_wave;    // pairs of a wave: a multiple of 64
};

__global__ void __launch_bounds__(kOT) experts_count_kernel(OrderArgs a) {
    extern __shared__ uint32_t cnt[];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kOT) cnt[e] = 0;
    __syncthreads();
    const uint64_t from = uint64_t(blockIdx.x) * a.per_wave * kOWaves;
    const uint64_t to = min(uint64_t(a.n), from + a.per_wave * kOWaves);
    for (uint64_t i = from + threadIdx.x; i < to; i += kOT) {
        const uint32_t e = uint32_t(a.ids[i]);
        if (e < a.experts) atomicAdd(&cnt[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kOT) a.counts[blockIdx.x * a.experts + e] = cnt[e];
}

// lanes of the wave with the same expert (bit by bit); `e` below 2^bits where `has`
__device__ __forceinline__ uint64_t same_expert(uint32_t e, bool has, uint32_t bits) {
    uint64_t peers = __ballot(has);
    for (uint32_t b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((e >> b) & 1u);
        peers &= ((e >> b) & 1u) ? one : ~one;
    }
    return peers;
}

__global__ void __launch_bounds__(kOT) experts_place_kernel(OrderArgs a) {
    extern __shared__ uint32_t shared[];
    uint32_t* cnt = shared;                          // [kOWaves][experts]
    uint32_t* base = shared + kOWaves * a.experts;   // [experts]: where the run's pairs of an expert begin
    uint32_t* sums = base + a.experts;            // [experts]: pairs in all runs
    uint32_t* part = sums + a.experts;            // [kOWaves]
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    for (uint32_t i = threadIdx.x; i < (kOWaves + 2) * a.experts; i += kOT) cnt[i] = 0;
    __syncthreads();
    const uint64_t from = (uint64_t(blockIdx.x) * kOWaves + wave) * a.per_wave;
    const uint64_t to = min(uint64_t(a.n), from + a.per_wave);
    for (uint64_t i = from + lane; i < to; i += 64) {
        const uint32_t e = uint32_t(a.ids[i]);
        if (e < a.experts) atomicAdd(&cnt[wave * a.experts + e], 1u);
    }
    __syncthreads();
    // the experts' pairs in all runs and in the runs in front: each wave adds up
    // some of the runs (so that the loads are on their way together)
    if (a.runs > 1) {
        for (uint32_t e = lane; e < a.experts; e += 64) {
            uint32_t all = 0, front = 0;
#pragma unroll 8
            for (uint32_t r = wave; r < a.runs; r += kOWaves) {
                const uint32_t c = a.counts[r * a.experts + e];
                all += c;
                front += r < blockIdx.x ? c : 0;
            }
            atomicAdd(&sums[e], all);
            atomicAdd(&base[e], front);
        }
        __syncthreads();
    }
    uint32_t all[2] = {}, front[2] = {};          // two experts a thread
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t e = 2 * threadIdx.x + h;
        if (e >= a.experts) continue;
        if (a.runs > 1)
            all[h] = sums[e], front[h] = base[e];
        else
            for (uint32_t w = 0; w < kOWaves; ++w) all[h] += cnt[w * a.experts + e];
    }
    // pairs of the experts below: prefix over lanes, then waves
    uint32_t sum = all[0] + all[1];
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(sum, d, 64);
        if (lane >= d) sum += o;
    }
    if (lane == 63) part[wave] = sum;
    __syncthreads();
    uint32_t below = sum - all[0] - all[1];
    for (uint32_t w = 0; w < wave; ++w) below += part[w];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t e = 2 * threadIdx.x + h;
        if (e >= a.experts) continue;
        const uint32_t start = below + (h ? all[0] : 0);
        base[e] = start + front[h];
        if (blockIdx.x == 0) {
            a.offsets[e] = int32_t(start);
            if (e + 1 == a.experts) a.offsets[a.experts] = int32_t(start + all[h]);
        }
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kOT) {
        uint32_t at = base[e];
        for (uint32_t w = 0; w < kOWaves; ++w) {
            const uint32_t c = cnt[w * a.experts + e];
            cnt[w * a.experts + e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (uint64_t i0 = from; i0 < to; i0 += 64) {
        const uint64_t i = i0 + lane;
        const uint32_t e = i < to ? uint32_t(a.ids[i]) : ~0u;
        const bool has = e < a.experts;
        const uint64_t peers = same_expert(e, has, a.bits);
        uint32_t* mine = &cnt[wave * a.experts + (has ? e : 0)];
        const uint32_t rank = uint32_t(__popcll(peers & ((uint64_t(1) << lane) - 1)));
        const uint32_t start = has ? *mine : 0;
        __builtin_amdgcn_wave_barrier();
        if (has && rank == 0) *mine = start + uint32_t(__popcll(peers));
        __builtin_amdgcn_wave_barrier();
        if (i < to) a.slots[i] = has ? int32_t(start + rank) : -1;
    }
}

// -------------------------------------------------------------------- host

// f(lanes, registers of eight) for a row of n elements
template <typename F>
void with_lanes(uint32_t n, F&& f) {
    const std::integral_constant<int, 1> one;
    if (n <= 64) f(std::integral_constant<int, 8>(), one);
    else if (n <= 128) f(std::integral_constant<int, 16>(), one);
    else if (n <= 256) f(std::integral_constant<int, 32>(), one);
    else if (n <= 512) f(std::integral_constant<int, 64>(), one);
    else f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
}

int32_t check_select(uint64_t rows, uint32_t experts, uint32_t k, uint32_t score, uint32_t options, float scale) {
    if (rows >= (uint64_t(1) << 31) || rows * k >= (uint64_t(1) << 31)) return step_fail(DCR_E_INVAL, "2^31 rows or pairs or more");
    if (!experts || experts > DCR_EXPERTS_MAX) return step_fail(DCR_E_INVAL, "experts are not 1 .. 1024");
    if (!k || k > DCR_EXPERTS_MAX_K || k > experts) return step_fail(DCR_E_INVAL, "k is not 1 .. 64 and at most the experts");
    if (score != DCR_SCORE_SOFTMAX && score != DCR_SCORE_SIGMOID) return step_fail(DCR_E_INVAL, "unknown score");
    if (options & ~uint32_t(DCR_EXPERTS_RENORMALIZE)) return step_fail(DCR_E_INVAL, "unknown option");
    if (!(scale > -INFINITY && scale < INFINITY)) return step_fail(DCR_E_INVAL, "scale is not finite");
    return DCR_OK;
}

int32_t select(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint32_t experts, const float* bias,
               uint32_t score, uint32_t groups, uint32_t top_groups, uint32_t options, float scale, uint32_t k, int32_t* ids,
               float* weights, hipStream_t st) {
    int32_t rc;
    if ((rc = check_select(rows, experts, k, score, options, scale)) ||
        (rc = check_matrix(logits, type, rows, experts, stride, "logits")))
        return rc;
    if (!groups || groups > DCR_EXPERTS_MAX_GROUPS || experts % groups)
        return step_fail(DCR_E_INVAL, "groups are not 1 .. 64 or do not divide the experts");
    if (!top_groups || top_groups > groups) return step_fail(DCR_E_INVAL, "top_groups is not 1 .. groups");
    if (!rows) return DCR_OK;
    if ((bias && (rc = check_array(bias, "bias"))) || (rc = check_array(ids, "ids")) || (rc = check_array(weights, "weights")))
        return rc;
    SelectArgs a{};
    a.logits = logits, a.bias = bias, a.ids = ids, a.weights = weights, a.stride = stride;
    a.rows = uint32_t(rows), a.experts = experts, a.k = k, a.groups = groups, a.top_groups = top_groups;
    a.sigmoid = score == DCR_SCORE_SIGMOID, a.renormalize = options & DCR_EXPERTS_RENORMALIZE, a.scale = scale;
    if (top_groups < groups) {
        const uint32_t size = experts / groups;
        while ((8u << a.group_log2) < size) ++a.group_log2;
        a.wide = experts > 512 || (8u << a.group_log2) != size;
    }
    with_type(type, [&](auto t) {
        with_lanes(experts, [&](auto lanes, auto r) {
            constexpr int L = decltype(lanes)::value, ROWS = kET / L;
            const uint32_t lds = top_groups < groups ? ROWS * (experts + groups) * 8 : 0;
            const uint32_t grid = uint32_t((rows + ROWS - 1) / ROWS);
            hipLaunchKernelGGL((experts_select_kernel<decltype(t), L, decltype(r)::value>), dim3(grid), dim3(kET), lds, st, a);
        });
    });
    return step_launched();
}

int32_t select_grad(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint32_t experts, const int32_t* ids,
                    const float* dweights, uint32_t k, uint32_t score, uint32_t options, float scale, void* dlogits,
                    uint64_t d_stride, hipStream_t st) {
    int32_t rc;
    if ((rc = check_select(rows, experts, k, score, options, scale)) ||
        (rc = check_matrix(logits, type, rows, experts, stride, "logits")) ||
        (rc = check_matrix(dlogits, type, rows, experts, d_stride, "dlogits")))
        return rc;
    if (!rows) return DCR_OK;
    if ((rc = check_array(ids, "ids")) || (rc = check_array(dweights, "dweights"))) return rc;
    SelectArgs a{};
    a.logits = logits, a.ids = const_cast<int32_t*>(ids), a.dweights = dweights, a.dlogits = dlogits;
    a.stride = stride, a.d_stride = d_stride, a.rows = uint32_t(rows), a.experts = experts, a.k = k;
    a.sigmoid = score == DCR_SCORE_SIGMOID, a.renormalize = options & DCR_EXPERTS_RENORMALIZE, a.scale = scale;
    with_type(type, [&](auto t) {
        with_lanes(experts, [&](auto lanes, auto r) {
            constexpr int L = decltype(lanes)::value, ROWS = kET / L;
            const uint32_t grid = uint32_t((rows + ROWS - 1) / ROWS);
            hipLaunchKernelGGL((experts_select_grad_kernel<decltype(t), L, decltype(r)::value>), dim3(grid), dim3(kET), 0, st, a);
        });
    });
    return step_launched();
}

int32_t order(const int32_t* ids, uint64_t n, uint32_t experts, int32_t* offsets, int32_t* slots, void* ws, uint64_t ws_bytes,
              hipStream_t st) {
    int32_t rc;
    if (n >= (uint64_t(1) << 31)) return step_fail(DCR_E_INVAL, "2^31 pairs or more");
    if (!experts || experts > DCR_EXPERTS_MAX) return step_fail(DCR_E_INVAL, "experts are not 1 .. 1024");
    if ((n && ((rc = check_array(ids, "ids")) || (rc = check_array(slots, "slots")))) || (rc = check_array(offsets, "offsets")) ||
        (rc = check_step_workspace(ws, ws_bytes)))
        return rc;
    OrderArgs a{};
    a.ids = ids, a.offsets = offsets, a.slots = slots, a.counts = static_cast<uint32_t*>(ws);
    a.n = uint32_t(n), a.experts = experts;
    while ((1u << a.bits) < experts) ++a.bits;
    a.runs = uint32_t(std::min<uint64_t>(kOrderRuns, std::max<uint64_t>(1, (n + 2047) / 2048)));
    a.per_wave = uint32_t(((n + a.runs * kOWaves - 1) / (a.runs * kOWaves) + 63) / 64 * 64);
    if (a.runs > 1)
        hipLaunchKernelGGL(experts_count_kernel, dim3(a.runs), dim3(kOT), experts * 4, st, a);
    hipLaunchKernelGGL(experts_place_kernel, dim3(a.runs), dim3(kOT), ((kOWaves + 2) * experts + kOWaves) * 4, st, a);
    return step_launched();
}

}  // namespace
}  // namespace dcr

extern "C" {

int32_t dcr_experts_select(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint32_t experts,
                           const float* bias, uint32_t score, uint32_t groups, uint32_t top_groups, uint32_t options,
                           float scale, uint32_t k, int32_t* ids, float* weights, void* stream) try {
    dcr::set_error("");
    return dcr::select(logits, type, stride, rows, experts, bias, score, groups, top_groups, options, scale, k, ids, weights,
                       static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_experts_select_grad(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint32_t experts,
                                const int32_t* ids, const float* dweights, uint32_t k, uint32_t score, uint32_t options,
                                float scale, void* dlogits, uint64_t dlogits_stride, void* stream) try {
    dcr::set_error("");
    return dcr::select_grad(logits, type, stride, rows, experts, ids, dweights, k, score, options, scale, dlogits,
                            dlogits_stride, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_experts_order(const int32_t* ids, uint64_t n, uint32_t experts, int32_t* offsets, int32_t* slots,
                          void* workspace_dev, uint64_t ws_bytes, void* stream) try {
    dcr::set_error("");
    return dcr::order(ids, n, experts, offsets, slots, workspace_dev, ws_bytes, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

}  // extern "C"
