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
    float scale;
};

// order of numbers as that of unsigned integers; NaN in front of all, and
// 0 for what may not be chosen
__device__ __forceinline__ uint64_t rank_of(double c) {
    if (c != c) return ~uint64_t(0);
    const uint64_t b = uint64_t(__double_as_longlong(c + 0.0));
    return b ^ (uint64_t(int64_t(b) >> 63) | (uint64_t(1) << 63));
}

struct Best {
    uint64_t rank;
    uint32_t at;
};
__device__ __forceinline__ Best better(Best a, Best b) {
    return (b.rank > a.rank || (b.rank == a.rank && b.at < a.at)) ? b : a;
}
template <int LANES>
__device__ __forceinline__ Best best_of(Best b) {
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) {
        const Best o = {uint64_t(__shfl_xor((unsigned long long)b.rank, d, 64)), uint32_t(__shfl_xor(int(b.at), d, 64))};
        b = better(b, o);
    }
    return b;
}
template <int LANES, typename T>
__device__ __forceinline__ T lanes_max(T v) {
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) {
        const T o = __shfl_xor(v, d, 64);
        v = (o > v || o != o) ? o : v;         // (a NaN stays)
    }
    return v;
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

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// scores of a lane's logits in 64 bits; top and sum are those of the softmax
template <int LANES, int N>
__device__ __forceinline__ void softmax_sums(const float* v, float* top, double* sum) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = (v[i] > m || v[i] != v[i]) ? v[i] : m;
    m = lanes_max<LANES>(m);
    if (m == -INFINITY) m = 0.0f;              // every expert is shut
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) z += exp(double(v[i]) - double(m));
    *top = m;
    *sum = lanes_sum<LANES>(z);
}

template <typename T, int LANES, int R>
__global__ void __launch_bounds__(kET) experts_select_kernel(SelectArgs a) {
    constexpr int N = 8 * R, ROWS = kET / LANES;
    extern __shared__ double values[];         // with groups: the row's values, then its groups' ranks
    const uint32_t lane = threadIdx.x % LANES, in_wg = threadIdx.x / LANES;
    const uint32_t at = blockIdx.x * ROWS + in_wg;
    const bool live = at < a.rows;
    const T* row = static_cast<const T*>(a.logits) + uint64_t(live ? at : 0) * a.stride;
    float v[N];
    load_row<T, LANES, R>(row, lane, a.experts, v);
    const bool grouped = a.top_groups < a.groups;
    float top = 0.0f;
    double sum = 1.0;
    if (!a.sigmoid) softmax_sums<LANES, N>(v, &top, &sum);
    if (sum == 0.0) sum = 1.0;

    uint64_t rank[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t e = 8 * (lane + LANES * (i / 8)) + i % 8;
        double c = double(v[i]);               // without a bias the logits have the order of the scores
        if (a.bias || grouped) {
            c = a.sigmoid ? sigmoid64(c) : exp(c - double(top)) / sum;
            if (a.bias && e < a.experts) c += double(a.bias[e]);
            if (grouped && e < a.experts) values[in_wg * a.experts + e] = v[i] == -INFINITY ? -INFINITY : c;
            if (!a.bias) c = double(v[i]);
        }
        rank[i] = v[i] == -INFINITY ? 0 : rank_of(c);
    }
    if (grouped) {
        uint64_t* of_group = reinterpret_cast<uint64_t*>(values + ROWS * a.experts) + in_wg * a.groups;
        const uint32_t size = a.experts / a.groups;
        __syncthreads();
        for (uint32_t g = lane; g < a.groups; g += LANES) {
            double first = -INFINITY, second = -INFINITY;
            bool odd = false;
            for (uint32_t i = 0; i < size; ++i) {
                const double c = values[in_wg * a.experts + g * size + i];
                odd |= c != c;
                second = c > first ? first : c > second ? c : second;
                first = c > first ? c : first;
            }
            of_group[g] = odd ? ~uint64_t(0) : first == -INFINITY ? 0 : rank_of(second == -INFINITY ? first : first + second);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t e = 8 * (lane + LANES * (i / 8)) + i % 8;
            if (e >= a.experts) continue;
            const uint32_t mine = e / size;
            const uint64_t r = of_group[mine];
            uint32_t ahead = 0;
            for (uint32_t g = 0; g < a.groups; ++g) ahead += (of_group[g] > r || (of_group[g] == r && g < mine)) ? 1u : 0u;
            if (ahead >= a.top_groups) rank[i] = 0;
        }
    }
    // the k best, one after the other; a lane keeps every LANES-th
    constexpr int KEEP = DCR_EXPERTS_MAX_K / LANES;
    int32_t id[KEEP];
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        id[q] = -1;
        for (uint32_t j = q * LANES; j < min(a.k, uint32_t(q + 1) * LANES); ++j) {
            Best b = {0, ~0u};
#pragma unroll
            for (int i = 0; i < N; ++i) b = better(b, Best{rank[i], 8 * (lane + LANES * (i / 8)) + i % 8});
            b = best_of<LANES>(b);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (8 * (lane + LANES * (i / 8)) + i % 8 == b.at) rank[i] = 0;
            if (j % LANES == lane) id[q] = b.rank ? int32_t(b.at) : -1;
        }
    }
    double w[KEEP], all = 0.0;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        w[q] = 0.0;
        if (id[q] >= 0) {
            const double l = double(wide(row[id[q]]));
            w[q] = a.sigmoid ? sigmoid64(l) : exp(l - double(top)) / sum;
        }
        all += w[q];
    }
    if (a.renormalize) {
        all = lanes_sum<LANES>(all);
        if (all == 0.0) all = 1.0;
    } else {
        all = 1.0;
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        const uint32_t j = q * LANES + lane;
        if (j >= a.k) continue;
        a.ids[uint64_t(at) * a.k + j] = id[q];
        a.weights[uint64_t(at) * a.k + j] = float(w[q] / all * double(a.scale));
    }
}

// The gradient.  With w_j = scale s_j / W (W: the chosen scores' sum, or 1)
//   ds_j = scale (dw_j - [renormalised] sum dw s / W) / W
//   dl   = s (1 - s) ds  or, of a softmax, s (ds - sum ds s), a sum that is
//          zero where the weights are renormalised
template <typename T, int LANES, int R>
__global__ void __launch_bounds__(kET) experts_select_grad_kernel(SelectArgs a) {
    constexpr int N = 8 * R, ROWS = kET / LANES;
    const uint32_t lane = threadIdx.x % LANES, at = blockIdx.x * ROWS + threadIdx.x / LANES;
    const bool live = at < a.rows;
    const uint64_t safe = live ? at : 0;
    const T* row = static_cast<const T*>(a.logits) + safe * a.stride;
    const int32_t* ids = a.ids + safe * a.k;
    const float* dw = a.dweights + safe * a.k;
    float v[N], d[N];
    load_row<T, LANES, R>(row, lane, a.experts, v);
    float top = 0.0f, inv = 1.0f;
    if (!a.sigmoid) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = (v[i] > top || v[i] != v[i]) ? v[i] : top;
        top = lanes_max<LANES>(top);
        if (top == -INFINITY) top = 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) z += expf(v[i] - top);
        z = lanes_sum<LANES>(z);
        inv = z == 0.0f ? 0.0f : 1.0f / z;
    }
    auto score = [&](float l) { return a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) * inv; };
    // the row's scalars in 64 bits: dw and its mean are often nearly the same
    double all = 0.0, dot = 0.0;
    for (uint32_t j = 0; j < a.k; ++j) {
        const uint32_t e = uint32_t(ids[j]);
        if (e >= a.experts) continue;
        const double s = double(score(wide(row[e])));
        all += s;
        dot += double(dw[j]) * s;
    }
    double over = double(a.scale), mean = 0.0;     // scale / W, and what the renormalisation takes off dw
    if (a.renormalize) {
        if (all == 0.0) all = 1.0;
        over /= all;
        mean = dot / all;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = 0.0f;
    for (uint32_t j = 0; j < a.k; ++j) {
        const uint32_t e = uint32_t(ids[j]);
        if (e >= a.experts) continue;
        const float ds = float((double(dw[j]) - mean) * over);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (8 * (lane + LANES * (i / 8)) + i % 8 == e) d[i] += ds;
    }
    const float off = a.renormalize ? 0.0f : float(dot * over);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (a.sigmoid) {
            const float q = expf(-fabsf(v[i]));    // s (1 - s) = q / (1 + q)^2
            d[i] *= q / ((1.0f + q) * (1.0f + q));
        } else {
            d[i] = expf(v[i] - top) * inv * (d[i] - off);
        }
    }
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
    uint32_t* part = base + a.experts;            // [kOWaves + 1]
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    for (uint32_t i = threadIdx.x; i < kOWaves * a.experts; i += kOT) cnt[i] = 0;
    __syncthreads();
    const uint64_t from = (uint64_t(blockIdx.x) * kOWaves + wave) * a.per_wave;
    const uint64_t to = min(uint64_t(a.n), from + a.per_wave);
    for (uint64_t i = from + lane; i < to; i += 64) {
        const uint32_t e = uint32_t(a.ids[i]);
        if (e < a.experts) atomicAdd(&cnt[wave * a.experts + e], 1u);
    }
    __syncthreads();
    // the experts' pairs in all runs, and in the runs in front; two experts a thread
    uint32_t all[2] = {}, front[2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t e = 2 * threadIdx.x + h;
        if (e >= a.experts) continue;
        if (a.runs == 1) {
            for (uint32_t w = 0; w < kOWaves; ++w) all[h] += cnt[w * a.experts + e];
        } else {
            for (uint32_t r = 0; r < a.runs; ++r) {
                const uint32_t c = a.counts[r * a.experts + e];
                all[h] += c;
                front[h] += r < blockIdx.x ? c : 0;
            }
        }
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
    hipLaunchKernelGGL(experts_place_kernel, dim3(a.runs), dim3(kOT), ((kOWaves + 1) * experts + kOWaves) * 4, st, a);
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
