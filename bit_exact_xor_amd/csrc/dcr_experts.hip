// dcr_experts.hip -- the choice of experts, its gradient, and the order of the
// chosen (token, expert) pairs.
//
// A row of logits lies in the registers of 8 to 64 lanes of a wave, eight
// consecutive ones (or twice eight) a lane, so several rows share a wave and
// nothing of a row leaves it but what is written.
//
// The choice is that of 64 bits: the values of experts next to one another often
// differ by less than the rounding of 32, and a choice that depended on it would
// differ from one program to the next.  32 bits decide what they can: a bound
// that the k best values surely reach (the k-th of the largest of the lanes'
// halves; of whole lanes' largest 24 of 128 took 39 us for 16000 rows, so 15)
// leaves little more than k candidates a row, and those alone, one a lane, are
// computed and ranked in 64.  (All experts in 64 bits took 20 us for 16384 rows of
// 256 where this takes 11; 32 bits with a second look at close rows 13 to 18, since a
// launch waits for its few second looks.)
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
    uint32_t group_log2;      // a group is looked at by 1 << group_log2 lanes
    uint32_t whole;           // its experts are theirs
    float scale;
};

// order of numbers as that of unsigned integers, NaN in front of all; above 0
__device__ __forceinline__ uint64_t rank_of(double c) {
    if (c != c) return ~uint64_t(0);
    const uint64_t b = uint64_t(__double_as_longlong(c + 0.0));
    return b ^ (uint64_t(int64_t(b) >> 63) | (uint64_t(1) << 63));
}
__device__ __forceinline__ uint64_t rank_of(float c) {
    if (c != c) return ~uint64_t(0);
    const uint32_t b = __float_as_uint(c + 0.0f);
    return uint64_t(b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u)) << 32;
}
// A rank with an index in its last ten bits, the lowest index first: no two
// alike, so one comparison decides.  (Of a sum in 64 bits that leaves 42 bits
// behind the leading one.)
static_assert(DCR_EXPERTS_MAX <= 1024 && DCR_EXPERTS_MAX_GROUPS <= 64, "ten bits of a key, 64 bits of groups");
__device__ __forceinline__ uint64_t key_of(uint64_t rank, uint32_t at) { return (rank | 1023u) - at; }
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 1023u - uint32_t(key & 1023u); }

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

// e^x for the comparisons, 2^-51 off: x as a multiple of log 2 and a rest below
// 0.35, of which the power series to the 12th power.  Held to +-700, where
// everything is 0 or 1 beside a bias.
__device__ __forceinline__ double exp_near(double x) {
    x = fmin(fmax(x, -700.0), 700.0);
    const double n = rint(x * 1.44269504088896340736);
    const double r = __fma_rn(n, -2.3190468138462996e-17, __fma_rn(n, -0.69314718055994530942, x));
    double p = 1.0 / 479001600;
    p = __fma_rn(p, r, 1.0 / 39916800), p = __fma_rn(p, r, 1.0 / 3628800), p = __fma_rn(p, r, 1.0 / 362880);
    p = __fma_rn(p, r, 1.0 / 40320), p = __fma_rn(p, r, 1.0 / 5040), p = __fma_rn(p, r, 1.0 / 720);
    p = __fma_rn(p, r, 1.0 / 120), p = __fma_rn(p, r, 1.0 / 24), p = __fma_rn(p, r, 1.0 / 6);
    p = __fma_rn(p, r, 0.5), p = __fma_rn(p, r, 1.0), p = __fma_rn(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, int(n));
}
// 1 / x: the hardware's estimate and two steps of Newton's iteration
__device__ __forceinline__ double inverse_near(double x) {
    double y = __builtin_amdgcn_rcp(x);
    y = __fma_rn(__fma_rn(-x, y, 1.0), y, y);
    return __fma_rn(__fma_rn(-x, y, 1.0), y, y);
}

// LDS of one wave: its accesses are in order, the compiler has to keep them so
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// order of 32-bit values as that of unsigned integers, NaN in front of all;
// above 0
__device__ __forceinline__ uint32_t rank32(float c) { return uint32_t(rank_of(c) >> 32); }
__device__ __forceinline__ float of_rank32(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// sum over the lanes of a row up to and with this one
template <int LANES>
__device__ __forceinline__ uint32_t lanes_upto(uint32_t v, uint32_t lane) {
    const auto add = [&](auto shift) {
        constexpr int D = decltype(shift)::value;
        const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x110 + D, 0xF, 0xF, true));   // D lanes up in a row of 16
        v += (LANES >= 16 || lane >= D) ? o : 0;
    };
    add(std::integral_constant<int, 1>()), add(std::integral_constant<int, 2>()), add(std::integral_constant<int, 4>());
    if constexpr (LANES >= 16) add(std::integral_constant<int, 8>());
    if constexpr (LANES >= 32) v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false));  // row 0 to 1, 2 to 3
    if constexpr (LANES >= 64) v += uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false));  // half to half
    return v;
}

// The two largest values of a lane's part of a group, and over STEP lanes more.
template <typename V>
struct Two {
    V first, second;
    __device__ __forceinline__ void meet(V f, V s) {
        second = fmax(fmin(first, f), fmax(second, s));
        first = fmax(first, f);
    }
    template <int STEP, int LANES>
    __device__ __forceinline__ void fold(uint32_t lanes) {
        if constexpr (STEP < LANES) {
            if (lanes > STEP) {
                V f[2], s[2];
                partners_of<STEP>(first, &f[0], &f[1]);
                partners_of<STEP>(second, &s[0], &s[1]);
                first = f[0], second = s[0];
                meet(f[1], s[1]);
            }
            fold<2 * STEP, LANES>(lanes);
        }
    }
    __device__ __forceinline__ bool none() const { return first == -INFINITY; }      // nothing is open
    __device__ __forceinline__ V value() const { return second == -INFINITY ? first : first + second; }
};

// The two largest of each group, in all of its lanes, from values c of the lane's
// experts (-infinity where shut).  Groups that are not whole lanes go through LDS.
// odd: there is a NaN among what the lane has seen.
template <int LANES, int N, typename V>
__device__ __forceinline__ Two<V> two_of_groups(const SelectArgs& a, const V* c, uint32_t lane, V* lds, bool* odd) {
    Two<V> two = {-INFINITY, -INFINITY};
    *odd = false;
    if (a.whole) {
#pragma unroll
        for (int i = 0; i < N; ++i) two.meet(c[i], -INFINITY), *odd |= c[i] != c[i];
    } else {
        const uint32_t size = a.experts / a.groups, mine = lane >> a.group_log2, share = 1u << a.group_log2;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (expert_of<LANES>(lane, i) < a.experts) lds[expert_of<LANES>(lane, i)] = c[i];
        wave_sync();
        if (mine < a.groups) {
            for (uint32_t i = lane & (share - 1); i < size; i += share) {
                const V x = lds[mine * size + i];
                two.meet(x, -INFINITY), *odd |= x != x;
            }
        }
        wave_sync();
    }
    two.template fold<1, LANES>(1u << a.group_log2);
    return two;
}

// Ranks to 0 outside the groups that are `in` (a group's lanes say the same).
template <int LANES, int N>
__device__ __forceinline__ void shut_groups(const SelectArgs& a, uint32_t lane, bool in, uint32_t* rank) {
    if (a.whole) {
#pragma unroll
        for (int i = 0; i < N; ++i) rank[i] = in ? rank[i] : 0;
        return;
    }
    const uint64_t taken = __ballot(in) >> (threadIdx.x & 63u & ~uint32_t(LANES - 1));
    const float inv = 1.0f / float(a.experts / a.groups);      // (e + 1/2 over the size is further from a whole number than its rounding)
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t e = expert_of<LANES>(lane, i), g = uint32_t((float(e) + 0.5f) * inv);
        rank[i] = e < a.experts && (taken >> (g << a.group_log2) & 1) ? rank[i] : 0;
    }
}

// The groups' choice in 32 bits.  Shuts experts (ranks to 0) and returns whether
// what decides is certain.  A value is off by `off` and 2^-24 of itself, and so
// is a sum of two once more: values 4 `off` and 2^-21 of the largest among them
// apart are in order.  Without a bias also those 2^-16 of themselves apart: a
// score is off by 2^-17 of itself at most (where its logit is 87 away from the
// others, by the rounding of its exponent) but for what all have in common, and
// has fewer bits only near 2^-126.
template <int LANES, int N>
__device__ __forceinline__ bool take_groups32(const SelectArgs& a, const float* c, uint32_t lane, float off, float* lds,
                                              uint32_t* rank) {
    bool odd;
    const Two<float> two = two_of_groups<LANES, N>(a, c, lane, lds, &odd);
    const uint32_t of = two.none() ? 0 : rank32(two.value());
    const uint32_t mine = lane >> a.group_log2, base = threadIdx.x & 63u & ~uint32_t(LANES - 1);
    uint32_t ahead = 0;
    for (uint32_t g = 0; g < a.groups; ++g) {
        const uint32_t o = uint32_t(__shfl(int(of), int(base + (g << a.group_log2)), 64));
        ahead += (o > of || (o == of && g < mine)) ? 1u : 0u;
    }
    const bool in = mine < a.groups && ahead < a.top_groups;
    const auto of_lanes = [](auto v, auto f) { return lanes_all<LANES>(v, f); };
    const float x = of_rank32(of_lanes(in ? of : ~0u, [](uint32_t p, uint32_t q) { return min(p, q); }));      // least taken
    const uint32_t most = of_lanes(in || mine >= a.groups ? 0u : of, [](uint32_t p, uint32_t q) { return max(p, q); });
    const float far = fmaxf(two.first == -INFINITY ? 0.0f : fabsf(two.first), two.second == -INFINITY ? 0.0f : fabsf(two.second));
    float apart = fmaf(0x1p-20f, of_lanes(far, [](float p, float q) { return fmaxf(p, q); }), 5 * off);
    if (!a.bias) apart = fminf(apart, fmaf(0x1p-15f, x, 0x1p-120f));
    shut_groups<LANES, N>(a, lane, in, rank);
    return !odd && (most == 0 || x - of_rank32(most) > apart);
}

// The same in 64 bits; a NaN's group goes first.  Groups without a value come
// behind all, the lowest index first, in both: their experts at a bias of
// -infinity may be taken yet.
template <int LANES, int N>
__device__ __forceinline__ void take_groups(const SelectArgs& a, const double* c, uint32_t lane, double* lds, uint32_t* rank) {
    bool odd;
    const Two<double> two = two_of_groups<LANES, N>(a, c, lane, lds, &odd);
    const uint32_t mine = lane >> a.group_log2, base = threadIdx.x & 63u & ~uint32_t(LANES - 1);
    uint64_t of = two.none() ? key_of(0, mine) : key_of(rank_of(two.value()), mine);      // (a rank is above 0)
    const uint64_t odds = __ballot(odd) >> (base + (mine << a.group_log2));
    if (odds & ((uint64_t(2) << ((1u << a.group_log2) - 1)) - 1)) of = key_of(~uint64_t(0), mine);
    uint32_t ahead = 0;
    for (uint32_t g = 0; g < a.groups; ++g)
        ahead += uint64_t(__shfl((unsigned long long)of, int(base + (g << a.group_log2)), 64)) > of ? 1u : 0u;
    shut_groups<LANES, N>(a, lane, mine < a.groups && ahead < a.top_groups, rank);
}

// scores of a row in 64 bits for the comparisons
template <int LANES, int N>
__device__ __forceinline__ double softmax_inverse(const float* v, float top) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) z += v[i] == -INFINITY ? 0.0 : exp_near(double(v[i]) - double(top));
    z = lanes_sum<LANES>(z);
    return z == 0.0 ? 0.0 : 1.0 / z;
}

// LDS of a row: its candidates, the chosen ones
__host__ __device__ inline uint32_t select_lds(uint32_t experts, uint32_t k) { return (8 * experts + 12 * k + 7) / 8 * 8; }

// (Held to the registers of eight waves a SIMD: 16384 x 256 in groups 14.0 us, with
// seven 14.9; 8 bytes of LDS an expert, not 12, so that they fit: 16000 x 1024 20
// us for 24.)
template <typename T, int LANES, int R>
__global__ void __launch_bounds__(kET, R == 1 ? 8 : 4) experts_select_kernel(SelectArgs a) {
    constexpr int N = 8 * R, ROWS = kET / LANES;
    constexpr float kLog2e = 1.44269504088896340736f;
    extern __shared__ uint64_t lds[];
    const uint32_t lane = threadIdx.x % LANES, in_wg = threadIdx.x / LANES;
    uint64_t* keys = lds + in_wg * (select_lds(a.experts, a.k) / 8);
    double* weights = reinterpret_cast<double*>(keys + a.experts);
    int32_t* ids = reinterpret_cast<int32_t*>(weights + a.k);
    const uint32_t at = blockIdx.x * ROWS + in_wg;
    const bool live = at < a.rows;
    const T* row = static_cast<const T*>(a.logits) + uint64_t(live ? at : 0) * a.stride;
    const bool grouped = a.top_groups < a.groups;
    float v[N], bias[N];
    load_row<T, LANES, R>(row, lane, a.experts, v);
    if (a.bias) {
        load_row<float, LANES, R>(a.bias, lane, a.experts, bias);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) bias[i] = 0.0f;
    }
    for (uint32_t j = lane; j < a.k; j += LANES) ids[j] = -1, weights[j] = 0.0;
    float top = 0.0f;
    if (!a.sigmoid) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = (v[i] > top || v[i] != v[i]) ? v[i] : top;
        top = lanes_max<LANES>(top);
        if (top == -INFINITY) top = 0.0f;      // every expert is shut
        if (top == INFINITY) top = NAN;        // infinity less itself: no score of the row is a number, as with a NaN
    }
    // Ranks in 32 bits.  A sigmoid by the hardware's exponential and reciprocal
    // (one step off each) is off by less than 2.3 * 2^-23 and a sum with the bias
    // by 2^-24 of itself.  A softmax's sum of a lane's 8 terms and 64 lanes' is off by
    // less than 26 * 2^-24: 13 additions, a term's 2 steps, and its exponent's
    // rounding, 2.3 times its distance from the largest, of which the terms' mean is
    // below 4.5 for 1024 of them; of a lane's 16 by 34 * 2^-24, eight additions more.
    // A score has its reciprocal's 2 and its own term's 2 steps besides: 30 and 38.
    // Without a bias the logits themselves have the scores' order.
    float off = 0x1p-21f;
    uint32_t rank[N];
    double inverse = 1.0;                      // of the softmax's sum
    if (!a.sigmoid && (a.bias || !a.renormalize)) inverse = softmax_inverse<LANES, N>(v, top);
    if (a.bias || grouped) {
        float c[N], inv = 1.0f;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v[i]));
        } else {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) z += c[i] = __builtin_amdgcn_exp2f((v[i] - top) * kLog2e);
            z = lanes_sum<LANES>(z);
            inv = z == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(z);
            off = (R == 2 ? 0x1p-18f : 0x1p-19f) * inv;      // (the largest score is inv)
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            c[i] = v[i] == -INFINITY ? -INFINITY : __fmaf_rn(c[i], inv, bias[i]);
            rank[i] = v[i] == -INFINITY ? 0 : rank32(a.bias ? c[i] : v[i]);
        }
        if (grouped) {
            uint32_t all[N];
#pragma unroll
            for (int i = 0; i < N; ++i) all[i] = rank[i];
            if (__any(!take_groups32<LANES, N>(a, c, lane, off, reinterpret_cast<float*>(keys), rank))) {
                double d[N];
                double z = inverse;
                if (!a.sigmoid && !a.bias && a.renormalize) z = softmax_inverse<LANES, N>(v, top);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    rank[i] = all[i];
                    d[i] = a.sigmoid ? inverse_near(1.0 + exp_near(-double(v[i]))) : exp_near(double(v[i]) - double(top)) * z;
                    d[i] = v[i] == -INFINITY ? -INFINITY : (v[i] != v[i] || top != top) ? NAN : d[i] + double(bias[i]);
                }
                take_groups<LANES, N>(a, d, lane, reinterpret_cast<double*>(keys), rank);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) rank[i] = v[i] == -INFINITY ? 0 : rank32(v[i]);
    }
    // the k-th largest of the largest ranks of the lanes' halves (or, with equals
    // among them, one below): at least k experts reach it
    uint32_t bound = 0;
    if (a.k <= 2 * LANES) {
        uint32_t mine = rank[0], next = rank[N / 2];
#pragma unroll
        for (int i = 1; i < N / 2; ++i) mine = max(mine, rank[i]), next = max(next, rank[N / 2 + i]);
        if (mine < next) {
            const uint32_t less = mine;
            mine = next, next = less;
        }
        for (uint32_t j = 0; j < a.k; ++j) {
            bound = lanes_all<LANES>(mine, [](uint32_t x, uint32_t y) { return max(x, y); });
            const bool out = mine == bound;
            mine = out ? next : mine, next = out ? 0 : next;
        }
        if (a.bias && bound && bound != ~0u) {     // and in 64 bits at least this
            const float x = of_rank32(bound);
            if (x < INFINITY) bound = rank32(x - 2 * fmaf(0x1p-22f, fabsf(x), off));
        }
    }
    bound = max(bound, 1u);
    // the candidates, one behind the other
    uint32_t count = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) count += rank[i] >= bound ? 1u : 0u;
    const uint32_t upto = lanes_upto<LANES>(count, lane);
    const uint32_t n = uint32_t(__shfl(int(upto), int((threadIdx.x & 63u) | (LANES - 1)), 64));
    uint32_t to = upto - count;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (rank[i] >= bound) keys[to] = uint64_t(__float_as_uint(v[i])) << 32 | expert_of<LANES>(lane, i);
        to += rank[i] >= bound ? 1u : 0u;
    }
    wave_sync();
    float first = 0.0f;                        // the logit of the lane's first candidate (there are seldom more)
    for (uint32_t i = lane; i < n; i += LANES) {
        const uint32_t e = uint32_t(keys[i]);
        const float l = __uint_as_float(uint32_t(keys[i] >> 32));
        first = i == lane ? l : first;
        uint64_t key;
        if (a.bias) {
            double c = a.sigmoid ? inverse_near(1.0 + exp_near(-double(l))) : exp_near(double(l) - double(top)) * inverse;
            if (l != l || top != top) c = NAN;
            key = rank_of(c + double(a.bias[e]));
        } else {
            key = rank_of(l);
        }
        keys[i] = key_of(key, e);
    }
    wave_sync();
    for (uint32_t i = lane; i < n; i += LANES) {
        const uint64_t mine = keys[i];
        uint32_t ahead = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < n; ++j) ahead += keys[j] > mine ? 1u : 0u;
        if (ahead < a.k) {
            const double l = double(i == lane ? first : wide(row[index_of(mine)]));
            ids[ahead] = int32_t(index_of(mine));
            weights[ahead] = a.sigmoid ? sigmoid64(l) : exp(l - double(top)) * (a.renormalize ? 1.0 : inverse);
        }
    }
    wave_sync();
    double all = 1.0;
    if (a.renormalize) {
        double sum = 0.0;
        for (uint32_t j = lane; j < a.k; j += LANES) sum += weights[j];
        sum = lanes_sum<LANES>(sum);
        if (sum != 0.0) all = sum;
    }
    if (!live) return;
    for (uint32_t j = lane; j < a.k; j += LANES) {
        a.ids[uint64_t(at) * a.k + j] = ids[j];
        a.weights[uint64_t(at) * a.k + j] = ids[j] < 0 ? 0.0f : float(weights[j] / all * double(a.scale));      // (`all` may be NaN)
    }
}

// The gradient, with ds_j = scale dw_j added up over the pairs of an expert:
//   dl = s (1 - s) ds  or, of a softmax, s (ds - sum ds s)
// and of renormalised weights, with r_j = s_j over the sum of the chosen scores:
//   dl = scale r_j (dw_j - sum dw r)  times 1 - s_j for a sigmoid
// of the chosen experts alone.  There the scores as such do not occur: r is taken
// from the chosen logits by their largest, so that scores of any size (at -104 all
// are 0 in 32 bits, the weights are not) give derivatives of the weights' size.
// Only where the scores of the forward call vanish, in 64 bits, do these.
// A lane has the pairs j = lane, lane + LANES, ..., whose logits it fetches.
constexpr float kGoneSigmoid = -709.7828f, kGoneSoftmax = -745.1332f;      // below these e^x overflows, or is 0, in 64 bits
template <typename T, int LANES, int R, bool RENORM>
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
        if (top == INFINITY) top = NAN;        // (as in the choice)
        if (!RENORM) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) z += d[i] = expf(v[i] - top);
            z = lanes_sum<LANES>(z);
            inv = z == 0.0f ? 0.0f : 1.0f / z;
        }
    }
    // the row's scalars in 64 bits: dw and its mean are often nearly the same
    double all = 0.0, dot = 0.0;
    float most = -INFINITY, rest[KEEP];        // largest of the chosen logits (a sigmoid's up to 0); 1 - s
    if (RENORM) {
#pragma unroll
        for (int q = 0; q < KEEP; ++q) {
            if (id[q] == ~0u) continue;
            const float l = a.sigmoid && s[q] > 0.0f ? 0.0f : s[q];
            most = (l > most || l != l) ? l : most;
        }
        most = lanes_max<LANES>(most);
    }
    const bool gone = a.sigmoid ? most < kGoneSigmoid : most - top < kGoneSoftmax;
#pragma unroll
    for (int q = 0; q < KEEP; ++q) {
        rest[q] = 1.0f;
        if (id[q] == ~0u) continue;
        const float l = s[q];
        if (!RENORM) {
            s[q] = a.sigmoid ? 1.0f : expf(l - top) * inv;
        } else if (a.sigmoid) {
            const float e = expf(-fabsf(l));
            s[q] = expf((l > 0.0f ? 0.0f : l) - most) / (1.0f + e);
            rest[q] = (l > 0.0f ? e : 1.0f) / (1.0f + e);
        } else {
            s[q] = expf(l - most);
        }
        if (RENORM && gone) s[q] = 0.0f;
        all += double(s[q]);
        dot += double(dw[q]) * double(s[q]);
    }
    dot = lanes_sum<LANES>(dot);
    double mean = 0.0;                         // what the renormalisation takes off dw
    if (RENORM) {
        all = lanes_sum<LANES>(all);
        if (all == 0.0) all = 1.0;
        mean = dot / all;
    }
    const float off = a.sigmoid || RENORM ? 0.0f : float(dot * double(a.scale));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (RENORM) {
            v[i] = top == top ? 1.0f : NAN;
        } else if (a.sigmoid) {
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
        float ds = dw[q] * a.scale;
        if (RENORM) ds = float((double(dw[q]) - mean) * double(a.scale) * (double(s[q]) / all * double(rest[q])));
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
    const uint64_t from = (uint64_t(blockIdx.x) * kOWaves + wave) * a.per_wave;
    const uint64_t to = min(uint64_t(a.n), from + a.per_wave);
    // the wave's first pairs, on their way while the runs are added up
    constexpr int AHEAD = 4;
    uint32_t ahead[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        const uint64_t i = from + 64 * u + lane;
        ahead[u] = i < to ? uint32_t(a.ids[i]) : ~0u;
    }
    for (uint32_t i = threadIdx.x; i < (kOWaves + 2) * a.experts; i += kOT) cnt[i] = 0;
    __syncthreads();
    // the experts' pairs in all runs and in the runs in front: each wave adds up
    // some of the runs (so that the loads are on their way together)
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        if (ahead[u] < a.experts) atomicAdd(&cnt[wave * a.experts + ahead[u]], 1u);
    for (uint64_t i = from + 64 * AHEAD + lane; i < to; i += 64) {
        const uint32_t e = uint32_t(a.ids[i]);
        if (e < a.experts) atomicAdd(&cnt[wave * a.experts + e], 1u);
    }
    if (a.runs > 1) {
        // (two experts and eight runs on their way together, as far as there are some)
        for (uint32_t e0 = lane; e0 < a.experts; e0 += 128) {
            uint32_t all[2] = {}, front[2] = {};
            for (uint32_t r0 = wave; r0 < a.runs; r0 += 8 * kOWaves) {
                uint32_t c[2][8];
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u) {
                    const uint32_t r = r0 + u * kOWaves;
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h)
                        c[h][u] = r < a.runs && e0 + 64 * h < a.experts ? a.counts[r * a.experts + e0 + 64 * h] : 0;
                }
#pragma unroll
                for (uint32_t u = 0; u < 8; ++u) {
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        all[h] += c[h][u];
                        front[h] += r0 + u * kOWaves < blockIdx.x ? c[h][u] : 0;
                    }
                }
            }
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                if (e0 + 64 * h >= a.experts) continue;
                atomicAdd(&sums[e0 + 64 * h], all[h]);
                atomicAdd(&base[e0 + 64 * h], front[h]);
            }
        }
    }
    __syncthreads();
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
    const auto place = [&](uint64_t i, uint32_t e) {
        const bool has = e < a.experts;
        const uint64_t peers = same_expert(e, has, a.bits);
        uint32_t* mine = &cnt[wave * a.experts + (has ? e : 0)];
        const uint32_t rank = uint32_t(__popcll(peers & ((uint64_t(1) << lane) - 1)));
        const uint32_t start = has ? *mine : 0;
        __builtin_amdgcn_wave_barrier();
        if (has && rank == 0) *mine = start + uint32_t(__popcll(peers));
        __builtin_amdgcn_wave_barrier();
        if (i < to) a.slots[i] = has ? int32_t(start + rank) : -1;
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
        if (from + 64 * u < to) place(from + 64 * u + lane, ahead[u]);
    for (uint64_t i0 = from + 64 * AHEAD; i0 < to; i0 += 64) place(i0 + lane, i0 + lane < to ? uint32_t(a.ids[i0 + lane]) : ~0u);
}

// -------------------------------------------------------------------- host

// f(lanes, registers of eight) for rows of n elements, of which k are taken: the
// fewest lanes that hold a row, or one for each that is taken while the rows leave
// lanes without work (24 of 128 for 1000 rows 7.8 us, with the 16 lanes that hold
// them 10.5 us; 16000 rows 15 us with either)
template <typename F>
void with_lanes(uint32_t n, uint32_t k, uint64_t rows, F&& f) {
    const std::integral_constant<int, 1> one;
    uint32_t lanes = 8;
    while (lanes < 64 && (lanes * 8 < n || (lanes < k && rows * lanes * 2 <= 262144))) lanes *= 2;
    if (n > 512) f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    else if (lanes == 8) f(std::integral_constant<int, 8>(), one);
    else if (lanes == 16) f(std::integral_constant<int, 16>(), one);
    else if (lanes == 32) f(std::integral_constant<int, 32>(), one);
    else f(std::integral_constant<int, 64>(), one);
}

int32_t check_select(uint64_t rows, uint32_t experts, uint32_t k, uint32_t score, uint32_t options, float scale) {
    // (a launch takes 2^32 threads, a row at most 64 of them)
    if (rows >= (uint64_t(1) << 26) || rows * k >= (uint64_t(1) << 31)) return step_fail(DCR_E_INVAL, "2^26 rows, 2^31 pairs or more");
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
    const uint32_t size = experts / groups;
    a.whole = experts <= 512 && size % 8 == 0 && !(size & (size - 1));
    with_type(type, [&](auto t) {
        // (at least a lane for each group)
        with_lanes(std::max(experts, top_groups < groups ? groups * 8 : 0), k, rows, [&](auto lanes, auto r) {
            constexpr int L = decltype(lanes)::value, ROWS = kET / L;
            a.group_log2 = 0;
            while (a.whole ? (8u << a.group_log2) < size : (2u << a.group_log2) * groups <= uint32_t(L)) ++a.group_log2;
            const uint32_t grid = uint32_t((rows + ROWS - 1) / ROWS);      // (rows: see check_select)
            hipLaunchKernelGGL((experts_select_kernel<decltype(t), L, decltype(r)::value>), dim3(grid), dim3(kET),
                               ROWS * select_lds(experts, k), st, a);
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
        with_lanes(experts, 0, rows, [&](auto lanes, auto r) {
            constexpr int L = decltype(lanes)::value, ROWS = kET / L;
            const uint32_t grid = uint32_t((rows + ROWS - 1) / ROWS);      // (rows: see check_select)
            const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(kET), 0, st, a); };
            a.renormalize ? go(experts_select_grad_kernel<decltype(t), L, decltype(r)::value, true>)
                          : go(experts_select_grad_kernel<decltype(t), L, decltype(r)::value, false>);
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
    // One workgroup for up to 2048 pairs (2048 pairs, 128 experts: 6.6 us, in two
    // runs and launches 8.1; 4096: 9.5 and 8.3), then runs of 1024 (16384: 9.1, of
    // 2048 9.9), of 2048 with many experts, whose counts a run has to add up
    // (32768 pairs, 512 experts: 15.7, of 1024 18.5).
    const uint64_t run = experts <= 256 ? 1024 : 2048;
    a.runs = n <= 2048 ? 1 : uint32_t(std::min<uint64_t>(kOrderRuns, (n + run - 1) / run));
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
