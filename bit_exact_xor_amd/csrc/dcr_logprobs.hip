// dcr_logprobs.hip -- log probabilities of given tokens, the entropy of their
// distribution and the most probable tokens; and the gradient.
//
// With z_j = scale x_j, m = max z, S = sum exp(z - m), T = sum exp(z - m) (z - m):
//   lse = m + log S,   log p_t = z_t - lse,   entropy = log S - T / S.
// (m, S, T) of two parts of a row join to those of both, so the logits are read
// once: every thread holds a running triple, in powers of two.  The entropy from
// log S and T, not from lse and a sum of z: where one token takes nearly all,
// log S and T / S are small themselves and nothing cancels.
//
// Bound by memory: one read of the logits.  A row is split over workgroups
// where there are few rows; a second launch joins the parts.
#include <algorithm>

#include "dcr_step.h"

namespace dcr {
namespace {

constexpr uint32_t kLT = 256;                // threads of a workgroup
constexpr uint32_t kLWaves = kLT / 64;
constexpr uint32_t kPiece = 16;              // logits of a thread in a step
constexpr uint32_t kMostParts = 4096;        // parts of all rows, where rows are split
static_assert(kMostParts * (16 + 8 * DCR_LOGPROBS_MAX_TOP) <= DCR_STEP_WORKSPACE_BYTES, "sums and keys of all parts");
constexpr uint32_t kMostKeys = 2048;         // keys of the parts of a row
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct LpArgs {
    const void* logits;
    const void* targets;
    float *logp, *lse, *entropy, *top_values;
    int32_t* top_ids;
    uint64_t stride;
    uint32_t rows, vocab, top, wide_ids, parts, part_len;   // part_len: a multiple of 8
    float scale;
    f32x4* sums;                             // [rows][parts]: m, S, T in base 2
    uint64_t* keys;                          // [rows][parts][top]
};

// m: the largest logit, not scaled; s and t: sums of 2^d and 2^d d over the
// differences to it, d = (x - m) unit.  The largest's own term is 1 exactly, so s
// is 1 at least, log p at most 0 and the entropy at least 0, and numbers of any
// size, as finite masks are, leave no rest in an exponent.  (One fused product
// x unit - mu with a rounded mu is no faster, 4096 x 151936 196 us where this takes
// 194, and the rest of that rounding stands in every exponent: log p of a
// certain token above 0, infinite sums where m unit passes 2^32.)
struct Sums {
    float m, s, t;
};

// the scale in base 2, a finite number (0 times infinity is none)
__device__ __forceinline__ float base2_of(float scale) { return fminf(scale * kLog2e, 0x1.fffffep127f); }

// the difference of a largest logit to a larger one; held to -160 (2^-160 is 0,
// and -infinity times that is not)
__device__ __forceinline__ float below(float a, float m, float unit) {
    return a == -INFINITY ? 0.0f : fmaxf((a - m) * unit, -160.0f);
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float unit) {
    const float m = fmaxf(a.m, b.m);
    const float da = below(a.m, m, unit), db = below(b.m, m, unit);
    const float fa = exp2f(da), fb = exp2f(db);
    return {m, __fmaf_rn(a.s, fa, b.s * fb), fa * __fmaf_rn(a.s, da, a.t) + fb * __fmaf_rn(b.s, db, b.t)};
}

// order of logits as that of unsigned integers, -0 as 0, NaN below all
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? 0u : b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // order_of(-infinity)
__device__ __forceinline__ float of_order(uint32_t u) {
    return u == 0 ? NAN : __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
// a logit and its index as one number, no two alike; 0 stands for none
__device__ __forceinline__ uint64_t key_of(float x, uint32_t at) { return (uint64_t(order_of(x)) << 32) | (0xFFFFFFFFu - at); }

// The best `top` keys that a workgroup has met, in order, in LDS.  Each round
// the threads bring some more, at most kMostPer each.  Only keys above the last
// one held come in question; where more than kDirect threads have such keys, a
// bound is taken first: the top-th largest of the best keys of 64 quads of
// threads (128 pairs, 256 threads where `top` is larger).  Only `top` of them
// reach it, so what is gathered is bounded whatever the order of the logits, and
// with logits in no order it is little more than `top`.  Ranks are counted (no
// two keys are alike), so nothing depends on the order in which threads arrive.
constexpr uint32_t kDirect = 32, kMostPer = 16, kQuads = 20, kPairs = 32;
constexpr uint32_t kGathered = kQuads * 4 * kMostPer;
static_assert(kGathered >= kPairs * 2 * kMostPer && kGathered >= DCR_LOGPROBS_MAX_TOP * kMostPer && kGathered >= kDirect * kMostPer,
              "room for what may pass the bound");
struct TopLds {
    uint64_t held[DCR_LOGPROBS_MAX_TOP];
    uint64_t best[kLT];
    uint64_t more[kGathered];
    uint64_t bound;
    uint32_t n;
};

// how many of the keys first, first + step, ... of n at `keys` (LDS) are larger
__device__ __forceinline__ uint32_t larger(const uint64_t* keys, uint32_t first, uint32_t n, uint32_t step, uint64_t key) {
    uint32_t r = 0, j = first;
    for (; j + 7 * step < n; j += 8 * step) {      // eight on their way together
        uint64_t k[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) k[u] = keys[j + u * step];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) r += k[u] > key ? 1u : 0u;
    }
    for (; j < n; j += step) r += keys[j] > key ? 1u : 0u;
    return r;
}

__device__ __forceinline__ void top_begin(TopLds& l) {
    if (threadIdx.x == 0) l.n = 0;
    __syncthreads();
}

// LANES threads share a key in the search for the bound
template <uint32_t LANES>
__device__ __forceinline__ void find_bound(TopLds& l, uint32_t top, uint64_t best) {
    const uint64_t mine = lanes_all<LANES>(best, [](uint64_t a, uint64_t b) { return max(a, b); });
    const uint32_t sub = threadIdx.x % LANES;
    if (sub == 0) l.best[threadIdx.x / LANES] = mine;
    if (threadIdx.x == 0) l.bound = 0;
    __syncthreads();
    const uint32_t above = lanes_sum<LANES>(larger(l.best, sub, kLT / LANES, LANES, mine));
    if (sub == 0 && mine && above == top - 1) l.bound = mine - 1;
    __syncthreads();
}

// A round, of all threads: `passes` tells (it may be too often true) whether
// one of the thread's keys is above `least`, `best` gives its largest key, `each`
// calls a function with every key above its argument, or more.  Returns the last key held, 0 (nothing is)
// before the first round.
template <typename B, typename E>
__device__ __forceinline__ uint64_t top_round(TopLds& l, uint32_t top, uint64_t least, bool first, bool passes, B&& best, E&& each) {
    const uint32_t some = uint32_t(__syncthreads_count(passes));
    if (!some && !first) return least;
    uint64_t from = least;
    if (some > kDirect) {
        const uint64_t mine = best();
        if (top <= kQuads)
            find_bound<4>(l, top, mine);
        else if (top <= kPairs)
            find_bound<2>(l, top, mine);
        else
            find_bound<1>(l, top, mine);
        from = max(from, l.bound);
    }
    if (passes) {
        each(from, [&](uint64_t k) {
            if (k > from) l.more[atomicAdd(&l.n, 1u)] = k;
        });
    }
    __syncthreads();
    const uint32_t n = l.n, held = first ? 0 : top;
    constexpr uint32_t U = (kGathered + DCR_LOGPROBS_MAX_TOP + kLT - 1) / kLT;
    uint64_t mine[U];
    uint32_t at[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
        mine[u] = 0, at[u] = top;
        if (u * kLT >= n + held) continue;
        const uint32_t i = u * kLT + threadIdx.x;
        mine[u] = i < n ? l.more[i] : i - n < held ? l.held[i - n] : 0;
        if (mine[u]) at[u] = larger(l.more, 0, n, 1, mine[u]) + larger(l.held, 0, held, 1, mine[u]);
    }
    __syncthreads();
    if (threadIdx.x < top && threadIdx.x >= n + held) l.held[threadIdx.x] = 0;      // (fewer keys than `top` so far)
    if (threadIdx.x == 0) l.n = 0;
#pragma unroll
    for (uint32_t u = 0; u < U; ++u)
        if (at[u] < top) l.held[at[u]] = mine[u];
    __syncthreads();
    return l.held[top - 1];
}

// The sums of the lanes of a wave: the largest first, then each lane's by it.
__device__ __forceinline__ Sums join_wave(Sums a, float unit) {
    const float m = lanes_all<64>(a.m, [](float x, float y) { return fmaxf(x, y); });
    const float d = below(a.m, m, unit), f = exp2f(d);
    return {m, lanes_sum<64>(a.s * f), lanes_sum<64>(f * __fmaf_rn(a.s, d, a.t))};
}

__device__ __forceinline__ int64_t target_of(const LpArgs& a, uint32_t row) {
    return a.wide_ids ? static_cast<const int64_t*>(a.targets)[row] : int64_t(static_cast<const int32_t*>(a.targets)[row]);
}

// what turns a logit into its log probability
struct RowOf {
    float m, log_s;
    __device__ __forceinline__ float logp(float x, float scale) const {
        return m == -INFINITY && log_s == log_s ? -INFINITY : (x - m) * scale - log_s;
    }
};

__device__ __forceinline__ bool none_open(Sums s) { return s.m == -INFINITY && s.s == s.s; }     // an empty row
__device__ __forceinline__ RowOf row_of_sums(Sums s) { return {s.m, none_open(s) ? 0.0f : logf(s.s)}; }

// lse of a row that is not empty, a finite number also where it lies beyond those
// of 32 bits: -infinity stands for an empty row
__device__ __forceinline__ float lse_of(RowOf of, float scale) {
    const float l = __fmaf_rn(of.m, scale, of.log_s);
    return fabsf(l) == INFINITY ? copysignf(0x1.fffffep127f, l) : l;
}

// what a row's sums give; by one thread
template <typename T>
__device__ __forceinline__ RowOf finish_row(const LpArgs& a, uint32_t row, Sums s) {
    const bool none = none_open(s);
    const RowOf of = row_of_sums(s);
    if (a.lse) a.lse[row] = none ? -INFINITY : lse_of(of, a.scale);
    if (a.entropy) a.entropy[row] = none ? 0.0f : of.log_s - kLn2 * s.t / s.s;
    if (a.logp) {
        const int64_t t = target_of(a, row);
        float lp = t < 0 ? 0.0f : NAN;
        if (t >= 0 && t < int64_t(a.vocab))
            lp = of.logp(wide(static_cast<const T*>(a.logits)[uint64_t(row) * a.stride + uint64_t(t)]), a.scale);
        a.logp[row] = lp;
    }
    return of;
}

__device__ __forceinline__ void put_top(const LpArgs& a, uint32_t row, uint32_t r, uint64_t key, RowOf of) {
    const uint64_t to = uint64_t(row) * a.top + r;
    a.top_ids[to] = int32_t(0xFFFFFFFFu - uint32_t(key));
    a.top_values[to] = of.logp(of_order(uint32_t(key >> 32)), a.scale);
}

// a thread's logits of a step of THREADS: twice eight, 8 THREADS apart, so that a
// wave reads whole lines
template <uint32_t THREADS, typename T>
__device__ __forceinline__ void load_step(const T* x, uint32_t c0, uint32_t to, Raw8<T>* raw) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t at = c0 + (h * THREADS + threadIdx.x % THREADS) * 8;
        const int n = at < to ? int(min(8u, to - at)) : 0;
        if (n == 8)
            raw[h].load_once(x + at);
        else
            raw[h].load_some(x + at, n, kBf16MinusInf);
    }
}

// A step's logits into a thread's sums; returns the largest of them.  Masks make
// 0 times -infinity of a sum of t, which then is taken again with the difference
// held above that: an instruction of twelve that the others do without.  `cut`:
// the step ends behind the row, in masks.
template <int N = int(kPiece)>
__device__ __forceinline__ float add_step(const float* v, float unit, bool cut, Sums& sum) {
    float top = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
    const float m = fmaxf(sum.m, top);
    const float base = m == -INFINITY ? 0.0f : m;
    const float d = below(sum.m, m, unit), f = exp2f(d);
    float s = 0.0f, t = 0.0f;
    if (!cut) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float e = (v[i] - base) * unit, p = __builtin_amdgcn_exp2f(e);
            s += p;
            t = __fmaf_rn(p, e, t);
        }
    }
    if (cut || __any(t != t)) {
        s = t = 0.0f;
        float again = unit;                  // (so that nothing of the above is held in registers for this)
        asm("" : "+v"(again));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float e = (v[i] - base) * again, p = __builtin_amdgcn_exp2f(e);
            s += p;
            t = __fmaf_rn(p, fmaxf(e, -160.0f), t);
        }
    }
    sum.t = __fmaf_rn(f, __fmaf_rn(sum.s, d, sum.t), t);
    sum.s = __fmaf_rn(sum.s, f, s);
    sum.m = m;
    return top;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLT, !TOP ? 8 : sizeof(T) == 2 ? 6 : 5) logprobs_kernel(LpArgs a) {
    __shared__ Sums of_wave[kLWaves];
    __shared__ std::conditional_t<TOP, TopLds, uint32_t> lds;
    __shared__ RowOf row_of;
    const uint32_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    const uint32_t from = part * a.part_len, to = min(a.vocab, from + a.part_len);
    const T* x = static_cast<const T*>(a.logits) + uint64_t(row) * a.stride;
    const float unit = base2_of(a.scale);
    Sums sum = {-INFINITY, 0.0f, 0.0f};
    uint64_t least = 0;
    Raw8<T> raw[2];
    load_step<kLT>(x, from, to, raw);
    if constexpr (TOP) top_begin(lds);
    for (uint32_t c0 = from; c0 < to; c0 += kLT * kPiece) {
        float v[kPiece];
        raw[0].get(v);
        raw[1].get(v + 8);
        if (c0 + kLT * kPiece < to) load_step<kLT>(x, c0 + kLT * kPiece, to, raw);
        [[maybe_unused]] const float top = add_step(v, unit, c0 + kLT * kPiece > to, sum);
        if constexpr (TOP) {
            const auto key = [&](int i) {
                const uint32_t j = c0 + ((i / 8) * kLT + threadIdx.x) * 8 + i % 8;
                return j < to ? key_of(v[i], j) : 0;
            };
            // (without `top` keys every thread with logits comes in question, NaN too)
            const bool passes = least == 0 ? c0 + threadIdx.x * 8 < to : order_of(top) >= uint32_t(least >> 32);
            least = top_round(
                lds, a.top, least, c0 == from, passes,
                [&] {
                    uint64_t b = 0;
#pragma unroll
                    for (int i = 0; i < int(kPiece); ++i) b = max(b, key(i));
                    return b;
                },
                [&](uint64_t above, auto&& put) {
                    const float low = of_order(uint32_t(above >> 32));      // (NaN of 0: nothing is below)
#pragma unroll
                    for (int i = 0; i < int(kPiece); ++i)
                        if (!(v[i] < low)) put(key(i));
                });
        }
    }
    sum = join_wave(sum, unit);
    if (lane == 0) of_wave[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t w = 1; w < kLWaves; ++w) sum = join(sum, of_wave[w], unit);
        if (a.parts == 1)
            row_of = finish_row<T>(a, row, sum);
        else
            a.sums[blockIdx.x] = f32x4{sum.m, sum.s, sum.t, 0.0f};
    }
    if constexpr (TOP) {
        __syncthreads();
        if (threadIdx.x < a.top) {
            if (a.parts == 1)
                put_top(a, row, threadIdx.x, lds.held[threadIdx.x], row_of);
            else
                a.keys[uint64_t(blockIdx.x) * a.top + threadIdx.x] = lds.held[threadIdx.x];
        }
    }
}

// The best `top` keys that a wave has met, one a lane, the largest in lane 0.  What
// few lanes bring is put in one after the other: ranked by a ballot, the lanes
// behind move up.  Where many lanes pass a bound is taken first, the top-th
// largest logit of the bests of the 128 halves of the lanes' sixteens, found bit
// by bit with ballots; what reaches it goes to LDS with the keys held, and ranks
// are counted.  LDS of a wave: the keys held, then what was gathered, from `top`
// halves (some more where logits are equal); up to 32 keys whole sixteens serve.
// (By ranks of the sixteens' best keys the 64 best of 4096 x 16384 took 649 us,
// where all of them reach the bound, so 103; the 20 best 54 with either.)
constexpr uint32_t kFewLanes = 10;
// halves that may reach the bound, some equals among them
__host__ __device__ constexpr uint32_t most_halves(uint32_t top) { return (top <= 32 ? 2 * top : top) + 16; }
constexpr uint32_t wave_keys(uint32_t top) {   // an even number, at least 128 behind the keys held
    return 2 * DCR_LOGPROBS_MAX_TOP + 8 + most_halves(top) * (kPiece / 2);
}

__device__ __forceinline__ void wave_sync() {      // LDS of one wave is in order, the compiler has to keep it so
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    return uint64_t(uint32_t(__builtin_amdgcn_readlane(int(v >> 32), lane))) << 32 |
           uint32_t(__builtin_amdgcn_readlane(int(uint32_t(v)), lane));
}

struct TopWave {
    uint64_t* lds;
    uint64_t mine, least;                    // the lane's key; that of lane top - 1, or a larger one that `top` keys of the row reach
    uint32_t have;                           // keys held, 0 or `top`
    // The waves of a workgroup that have parts of one row tell one another the
    // logit of their share-th key: `top` logits reach the least of these.  Nobody
    // waits: what is read too early is smaller.
    volatile uint32_t* told;
    uint32_t wave, share;
    u32x4 not_ours;                          // ones for the waves of other rows

    __device__ __forceinline__ TopWave(uint64_t* at, uint32_t* told_, uint32_t wave_, uint32_t from, uint32_t to, uint32_t top)
        : lds(at), mine(0), least(0), have(0), told(told_), wave(wave_), share(to - from < 2 ? 0 : (top + to - from - 1) / (to - from)) {
#pragma unroll
        for (uint32_t w = 0; w < kLWaves; ++w) not_ours[w] = w >= from && w < to ? 0u : ~0u;
    }

    __device__ __forceinline__ void hear() {
        const u32x4 t = *reinterpret_cast<volatile u32x4*>(told) | not_ours;
        const uint32_t low = __builtin_amdgcn_readfirstlane(min(min(t[0], t[1]), min(t[2], t[3])));
        if (low) least = max(least, (uint64_t(low) << 32) - 1);
    }
    __device__ __forceinline__ void tell() {
        if (share) told[wave] = uint32_t(__builtin_amdgcn_readlane(int(mine >> 32), int(share) - 1));    // (all lanes the same)
    }

    __device__ __forceinline__ void insert(uint64_t key, uint32_t top) {
        const uint32_t lane = threadIdx.x & 63u, at = uint32_t(__popcll(__ballot(mine > key)));
        // (the lane in front's: a shift of the whole wave)
        const uint64_t front = uint64_t(uint32_t(__builtin_amdgcn_update_dpp(0, int(mine >> 32), 0x138, 0xF, 0xF, false))) << 32 |
                               uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(mine)), 0x138, 0xF, 0xF, false));
        mine = lane < at ? mine : lane == at ? key : front;
        least = max(least, lane_value(mine, int(top) - 1));
    }

    // LAST: the last bit of order_of that differs between values of the logits' type
    template <uint32_t LAST, typename K>
    __device__ __forceinline__ void round(uint32_t top, bool passes, float largest, const float* v, K&& key) {
        const uint32_t lane = threadIdx.x & 63u;
        if (share && __any(passes)) {
            hear();
            passes = passes && order_of(largest) >= uint32_t(least >> 32);
        }
        const uint32_t some = uint32_t(__popcll(__ballot(passes)));
        if (!some && have) return;
        if (some <= kFewLanes && have) {
            float low = of_order(uint32_t(least >> 32));       // (NaN of 0: nothing is below)
#pragma unroll
            for (int i = 0; i < int(kPiece); ++i) {
                uint64_t who = __ballot(passes && !(v[i] < low));
                if (!who) continue;
                const uint64_t k = key(v[i], i);
                for (; who; who &= who - 1) {
                    const uint64_t one = lane_value(k, __ffsll((unsigned long long)who) - 1);
                    if (one > least) insert(one, top);
                }
                low = of_order(uint32_t(least >> 32));
            }
            tell();
            return;
        }
        uint64_t *held = lds, *more = lds + DCR_LOGPROBS_MAX_TOP;
        uint64_t from = least;
        if (2 * some > top) {                                  // (else there is room for all)
            uint32_t bound = 0, reach = 0;
            const auto search = [&](auto&& reached) {          // by how many a logit's order is reached
#pragma unroll 1
                for (uint32_t bit = 1u << 31; bit >= LAST; bit >>= 1) {
                    const uint32_t n = reached(bound | bit);
                    if (n >= top) bound |= bit, reach = n;
                }
            };
            if (top <= 32) {
                const uint32_t order = order_of(largest);
                search([&](uint32_t b) { return uint32_t(__popcll(__ballot(order >= b))); });
                reach *= 2;
            } else {
                float best[2] = {v[0], v[8]};
#pragma unroll
                for (int i = 1; i < 8; ++i) best[0] = fmaxf(best[0], v[i]), best[1] = fmaxf(best[1], v[8 + i]);
                const uint32_t order[2] = {order_of(best[0]), order_of(best[1])};
                search([&](uint32_t b) {
                    return uint32_t(__popcll(__ballot(order[0] >= b)) + __popcll(__ballot(order[1] >= b)));
                });
            }
            // (-infinity also stands behind the end of a row)
            if (bound > kMinusInf && reach <= most_halves(top)) {
                from = max(from, (uint64_t(bound) << 32) - 1);
            } else {                                           // many equals, or fewer numbers: by whole keys
                uint64_t b[2] = {};
#pragma unroll
                for (int i = 0; i < int(kPiece); ++i) {
                    float x = v[i];
                    asm volatile("" : "+v"(x));                // (not kept for what follows: it would take 32 registers)
                    b[i / 8] = max(b[i / 8], key(x, i));
                }
                more[lane] = b[0], more[64 + lane] = b[1];
                wave_sync();
                uint32_t ahead[2] = {};
#pragma unroll 4
                for (int j = 0; j < 128; ++j) {
                    const uint64_t k = more[j];
                    ahead[0] += k > b[0] ? 1u : 0u, ahead[1] += k > b[1] ? 1u : 0u;
                }
                wave_sync();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t who = __ballot(b[h] && ahead[h] == top - 1);
                    if (who) from = max(from, lane_value(b[h], __ffsll((unsigned long long)who) - 1) - 1);
                }
            }
        }
        uint32_t n = 0;
        const float low = of_order(uint32_t(from >> 32));
#pragma unroll
        for (int i = 0; i < int(kPiece); ++i) {
            if (!__ballot(passes && !(v[i] < low))) continue;
            const uint64_t k = key(v[i], i);
            const bool in = passes && k > from;
            const uint64_t who = __ballot(in);
            if (in) more[n + uint32_t(__popcll(who & ((uint64_t(1) << lane) - 1)))] = k;
            n += uint32_t(__popcll(who));
        }
        if (lane < have) more[n + lane] = mine;
        n += have;
        if (lane < 8) more[n + lane] = 0;                      // (ranks are counted eight at a time)
        if (lane < top) held[lane] = 0;                        // (fewer keys than `top` so far)
        wave_sync();
        for (uint32_t i = lane; i < n; i += 64) {
            const uint64_t k = more[i];
            const uint32_t at = larger(more, 0, (n + 7) / 8 * 8, 1, k);
            if (k && at < top) held[at] = k;
        }
        wave_sync();
        mine = lane < top ? held[lane] : 0;
        wave_sync();
        have = top;
        least = max(least, lane_value(mine, int(top) - 1));
        tell();
    }
};

// A wave a part: no barriers.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kLT, TOP ? 6 : 8) logprobs_wave_kernel(LpArgs a) {
    extern __shared__ uint64_t wave_lds[];
    const uint32_t unit_of = __builtin_amdgcn_readfirstlane(blockIdx.x * kLWaves + (threadIdx.x >> 6)), lane = threadIdx.x & 63u;
    const uint32_t row = unit_of / a.parts, part = unit_of % a.parts;
    uint32_t* told = reinterpret_cast<uint32_t*>(wave_lds + kLWaves * wave_keys(a.top));
    if constexpr (TOP) {
        if (threadIdx.x < kLWaves) told[threadIdx.x] = 0;
        __syncthreads();
    }
    if (row >= a.rows) return;
    const uint32_t from = part * a.part_len, to = min(a.vocab, from + a.part_len);
    const T* x = static_cast<const T*>(a.logits) + uint64_t(row) * a.stride;
    const float unit = base2_of(a.scale);
    constexpr uint32_t STEP = 64 * kPiece;
    Sums sum = {-INFINITY, 0.0f, 0.0f};
    const uint32_t wave = unit_of % kLWaves;
    TopWave best(wave_lds + wave * wave_keys(a.top), told, wave, wave - min(wave, part), min(kLWaves, wave + a.parts - part), a.top);
    Raw8<T> raw[2];
    load_step<64>(x, from, to, raw);
    for (uint32_t c0 = from; c0 < to; c0 += STEP) {
        float v[kPiece];
        raw[0].get(v);
        raw[1].get(v + 8);
        if (c0 + STEP < to) load_step<64>(x, c0 + STEP, to, raw);
        [[maybe_unused]] const float top = add_step(v, unit, c0 + STEP > to, sum);
        if constexpr (TOP) {
            const bool passes = best.least == 0 ? c0 + lane * 8 < to : order_of(top) >= uint32_t(best.least >> 32);
            best.template round<sizeof(T) == 2 ? 1u << 16 : 1u>(a.top, passes, top, v, [&](float x, int i) {
                const uint32_t j = c0 + ((i / 8) * 64 + lane) * 8 + i % 8;
                return j < to ? key_of(x, j) : 0;
            });
        }
    }
    sum = join_wave(sum, unit);
    if (a.parts == 1) {
        if (lane == 0) finish_row<T>(a, row, sum);
        if constexpr (TOP) {
            if (lane < a.top) put_top(a, row, lane, best.mine, row_of_sums(sum));
        }
    } else {
        if (lane == 0) a.sums[unit_of] = f32x4{sum.m, sum.s, sum.t, 0.0f};
        if constexpr (TOP) {
            if (lane < a.top) a.keys[uint64_t(unit_of) * a.top + lane] = best.mine;
        }
    }
}

// the parts of a row; a workgroup a row
template <typename T, bool TOP>
__global__ void __launch_bounds__(kLT) logprobs_join_kernel(LpArgs a) {
    __shared__ std::conditional_t<TOP, TopLds, uint32_t> lds;
    __shared__ RowOf row_of;
    const uint32_t row = blockIdx.x;
    const float unit = base2_of(a.scale);
    const uint32_t n = a.parts * a.top;
    constexpr uint32_t MOST = kMostKeys / kLT;
    uint64_t keys[TOP ? MOST : 1];
    if constexpr (TOP) {
#pragma unroll
        for (uint32_t u = 0; u < MOST; ++u) {
            const uint32_t i = u * kLT + threadIdx.x;
            keys[u] = i < n ? a.keys[uint64_t(row) * n + i] : 0;
        }
        top_begin(lds);
    }
    if (threadIdx.x < 64) {
        Sums sum = {-INFINITY, 0.0f, 0.0f};
        for (uint32_t p = threadIdx.x; p < a.parts; p += 64) {
            const f32x4 q = a.sums[uint64_t(row) * a.parts + p];
            sum = join(sum, Sums{q[0], q[1], q[2]}, unit);
        }
        sum = join_wave(sum, unit);
        if (threadIdx.x == 0) row_of = finish_row<T>(a, row, sum);
    }
    if constexpr (TOP) {
        top_round(
            lds, a.top, 0, true, true,
            [&] {
                uint64_t b = 0;
#pragma unroll
                for (uint32_t u = 0; u < MOST; ++u) b = max(b, keys[u]);
                return b;
            },
            [&](uint64_t, auto&& put) {
#pragma unroll
                for (uint32_t u = 0; u < MOST; ++u) put(keys[u]);
            });
        if (threadIdx.x < a.top) put_top(a, row, threadIdx.x, lds.held[threadIdx.x], row_of);
    }
}

struct LpGradArgs {
    const void* logits;
    const void* targets;
    const float *lse, *dlogp, *entropy, *dentropy;
    void* dlogits;
    uint64_t stride, d_stride;
    uint32_t rows, vocab, wide_ids, pieces;      // pieces: workgroups, or threads, of a row
    float scale;
};

constexpr uint32_t kGU = 2;                      // eights of a thread in a row of its workgroup's

// Half a step of lse is in every p of its row: 2^-19 of it below 64, but 3e-5 at
// 1000 and all of it at the lowest finite number, a mask.  From 64 on a row's
// largest logit and log S are taken apart from one another again, from the logits
// (log p = scale (x - m) - log S, as the forward call has it), by one workgroup, or
// of short rows one wave or thread, which reads them twice (4096 x 151936 1085 us
// for 399, 10000 x 1264 33 for 13.9, 8 x 151936 88 for 7).  An lse that the logits do
// not give (of a vocabulary that is held in parts) is taken as it is.
constexpr float kFarLse = 64.0f, kOwnLse = 0x1p-22f;
__device__ __forceinline__ bool is_far(float lse) { return fabsf(lse) >= kFarLse && fabsf(lse) < INFINITY; }

// log p = scale (x - m) - log_s of a row with such an lse, m 0 and log_s the lse where
// it is another's; in all threads, from a wave's sums of the row
__device__ __forceinline__ RowOf row_of_far(Sums s, float lse, float scale) {
    const RowOf of = row_of_sums(s);
    return fabsf(lse_of(of, scale) - lse) <= kOwnLse * fabsf(lse) ? of : RowOf{0.0f, lse};
}

// sums of the row by THREADS threads, a thread's part
template <uint32_t THREADS, typename T>
__device__ __forceinline__ Sums part_of_row(const T* x, uint32_t vocab, float unit) {
    Sums sum = {-INFINITY, 0.0f, 0.0f};
    for (uint32_t c0 = 0; c0 < vocab; c0 += THREADS * kPiece) {
        Raw8<T> raw[2];
        float v[kPiece];
        load_step<THREADS>(x, c0, vocab, raw);
        raw[0].get(v);
        raw[1].get(v + 8);
        add_step(v, unit, c0 + THREADS * kPiece > vocab, sum);
    }
    return sum;
}

// dx_j = scale (dlogp (1[j = t] - p_j) - dentropy p_j (log p_j + entropy)), for
// the eight logits from `at` on.  Without FAR nothing is done and true returned
// where the lse is far (which the loads of the logits need not wait for: 10000 x
// 1264 13.9 us, else 15.0; 98 x 6368 2.98 in a graph, else 3.06).
template <typename T, int U, bool FAR = false>
__device__ __forceinline__ bool grad_of(const LpGradArgs& a, uint32_t row, const uint32_t* at, RowOf of = {}) {
    const T* x = static_cast<const T*>(a.logits) + uint64_t(row) * a.stride;
    T* y = static_cast<T*>(a.dlogits) + uint64_t(row) * a.d_stride;
    const int64_t target = a.wide_ids ? static_cast<const int64_t*>(a.targets)[row]
                                      : int64_t(static_cast<const int32_t*>(a.targets)[row]);
    const float lse = a.lse[row];
    float up = target < 0 ? 0.0f : a.dlogp[row];
    if (target >= int64_t(a.vocab)) up = NAN;
    const float b = a.dentropy ? a.dentropy[row] : 0.0f;
    const float c = a.dentropy ? __fmaf_rn(b, a.entropy[row], up) : up;
    const bool none = lse == -INFINITY;          // an empty row
    Raw8<T> raw[U];
    int n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        n[u] = at[u] < a.vocab ? int(min(8u, a.vocab - at[u])) : 0;
        n[u] == 8 ? raw[u].load_once(x + at[u]) : raw[u].load_some(x + at[u], n[u], kBf16MinusInf);
    }
    if (!FAR && is_far(lse)) return true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[8];
        raw[u].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float l = FAR ? __fmaf_rn(v[i] - of.m, a.scale, -of.log_s) : __fmaf_rn(v[i], a.scale, -lse);
            const float p = __builtin_amdgcn_exp2f(l * kLog2e);
            // p (up + b (log p + entropy)); p = 0 where log p is -infinity
            const float g = -p * __fmaf_rn(b, fmaxf(l, -110.0f), c);
            v[i] = none ? 0.0f : g * a.scale;
        }
        const int64_t hot = target - int64_t(at[u]);
        if (hot >= 0 && hot < 8 && !none) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i == int(hot)) v[i] = __fmaf_rn(up, a.scale, v[i]);
        }
        n[u] == 8 ? store8<true>(y + at[u], v) : store_some(y + at[u], v, n[u]);
    }
    return false;
}

// A workgroup has kGU eights a thread of one row; the first has all of a row with
// a far lse (the others would read logits that it may have written over).
template <typename T>
__global__ void __launch_bounds__(kLT) logprobs_grad_kernel(LpGradArgs a) {
    const uint32_t row = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces;
    uint32_t at[kGU];
    const auto place = [&](uint32_t first) {
#pragma unroll
        for (uint32_t u = 0; u < kGU; ++u) at[u] = first + (u * kLT + threadIdx.x) * 8;
    };
    place(piece * kGU * kLT * 8);
    if (!grad_of<T, kGU>(a, row, at) || piece) return;
    __shared__ Sums of_wave[kLWaves];
    const float unit = base2_of(a.scale);
    Sums sum = part_of_row<kLT>(static_cast<const T*>(a.logits) + uint64_t(row) * a.stride, a.vocab, unit);
    sum = join_wave(sum, unit);
    if ((threadIdx.x & 63u) == 0) of_wave[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = of_wave[0];
    for (uint32_t w = 1; w < kLWaves; ++w) sum = join(sum, of_wave[w], unit);
    const RowOf of = row_of_far(sum, a.lse[row], a.scale);
    for (uint32_t c0 = 0; c0 < a.vocab; c0 += kGU * kLT * 8) {
        place(c0);
        grad_of<T, kGU, true>(a, row, at, of);
    }
}

// Short rows: threads have an eight each, dealt over the rows one after the other.
// Rows with a far lse go to the threads that have their first eights, up to kAlone
// eights, else to the waves of these, one row after the other (16384 rows of 30
// logits 7.6 us, by waves 46; of 5 7.6 and 174; 10647 of 92 18.5 and 20).
constexpr uint32_t kAlone = 12;
template <typename T>
__global__ void __launch_bounds__(kLT, 8) logprobs_grad_short_kernel(LpGradArgs a) {
    const uint32_t i = blockIdx.x * kLT + threadIdx.x, row = i / a.pieces, at = (i - row * a.pieces) * 8;
    const bool far = row < a.rows && grad_of<T, 1>(a, row, &at);
    if (a.pieces <= kAlone) {
        if (!far || at) return;
        const T* x = static_cast<const T*>(a.logits) + uint64_t(row) * a.stride;
        Sums sum = {-INFINITY, 0.0f, 0.0f};
#pragma unroll 1
        for (uint32_t c = 0; c < a.vocab; c += 8) {
            Raw8<T> raw;
            float v[8];
            c + 8 <= a.vocab ? raw.load(x + c) : raw.load_some(x + c, int(a.vocab - c), kBf16MinusInf);
            raw.get(v);
            add_step<8>(v, base2_of(a.scale), true, sum);
        }
        const RowOf of = row_of_far(sum, a.lse[row], a.scale);
#pragma unroll 1
        for (uint32_t c = 0; c < a.vocab; c += 8) grad_of<T, 1, true>(a, row, &c, of);
        return;
    }
    for (uint64_t some = __ballot(far && at == 0); some; some &= some - 1) {
        const uint32_t r = uint32_t(__builtin_amdgcn_readlane(int(row), __ffsll((unsigned long long)some) - 1));
        const float unit = base2_of(a.scale);
        const Sums sum = part_of_row<64>(static_cast<const T*>(a.logits) + uint64_t(r) * a.stride, a.vocab, unit);
        const RowOf of = row_of_far(join_wave(sum, unit), a.lse[r], a.scale);
        for (uint32_t c = (threadIdx.x & 63u) * 8; c < a.vocab; c += 64 * 8) grad_of<T, 1, true>(a, r, &c, of);
    }
}

int32_t check_logits(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint64_t vocab, const void* targets,
                     uint32_t targets_bytes, float scale) {
    int32_t rc;
    if (rows >= (uint64_t(1) << 31)) return step_fail(DCR_E_INVAL, "2^31 rows or more");
    if (!vocab || vocab >= (uint64_t(1) << 31) - kLT * kPiece) return step_fail(DCR_E_INVAL, "vocabulary of 0 or about 2^31 tokens or more");
    if (!(scale > 0.0f && scale < INFINITY)) return step_fail(DCR_E_INVAL, "scale is not positive and finite");
    if ((rc = check_matrix(logits, type, rows, vocab, stride, "logits"))) return rc;
    if (targets_bytes != 4 && targets_bytes != 8) return step_fail(DCR_E_INVAL, "targets are neither int32 nor int64");
    return targets ? check_array(targets, "targets", targets_bytes) : DCR_OK;
}

int32_t logprobs(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint64_t vocab, const void* targets,
                 uint32_t targets_bytes, float scale, float* logp, float* lse, float* entropy, uint32_t top, int32_t* top_ids,
                 float* top_values, void* ws, uint64_t ws_bytes, hipStream_t st) {
    int32_t rc;
    if ((rc = check_logits(logits, type, stride, rows, vocab, targets, targets_bytes, scale))) return rc;
    if (top > DCR_LOGPROBS_MAX_TOP || top > vocab) return step_fail(DCR_E_INVAL, "top is more than 64 or than the vocabulary");
    if (!rows) return DCR_OK;
    if (logp && !targets) return step_fail(DCR_E_INVAL, "targets: NULL");
    if ((logp && (rc = check_array(logp, "logp"))) || (lse && (rc = check_array(lse, "lse"))) ||
        (entropy && (rc = check_array(entropy, "entropy"))) ||
        (top && ((rc = check_array(top_ids, "top_ids")) || (rc = check_array(top_values, "top_values")))) ||
        (rc = check_step_workspace(ws, ws_bytes)))
        return rc;
    LpArgs a{};
    a.logits = logits, a.targets = targets, a.logp = logp, a.lse = lse, a.entropy = entropy;
    a.top_values = top_values, a.top_ids = top_ids, a.stride = rows > 1 ? stride : 0;
    a.rows = uint32_t(rows), a.vocab = uint32_t(vocab), a.top = top, a.wide_ids = targets_bytes == 8, a.scale = scale;
    // Who takes a row (us; `top` 0 and 20).  A wave, where a row is one step of
    // it (16384 x 1000: 12 and 29, a workgroup 33 and 95) or rows fill the GPU
    // (4096 x 16384: 26 and 54, a workgroup 29 and 67; of longest rows only with
    // `top`: 4096 x 151936 214 and 273, a workgroup 197 and 373); several, up to 4096
    // in all, where fewer rows are long (1024 x 151936: 60 and 91, workgroups 61 and
    // 131; but 1024 x 32000 18, workgroups 16; above 2048 rows that is one a row:
    // 2048 x 151936 110 and 152, 2049 121 and 187) and, with `top`, of 256 rows
    // or more (256 x 151936: 42, workgroups 48; 512 x 32000: 28.6 and 29.5; but 2500
    // x 20000, a wave each, 55 and 51).  Else at least 1024 workgroups, each with a
    // step or more (8 x 151936: 6.5 and 14 in 38 parts, 8.2 and 27 in 10; 256 rows
    // without `top` 21, in 512 workgroups 24).
    const bool is_long = vocab >= 65536;
    bool by_wave = vocab <= 64 * kPiece;
    uint64_t parts = 1;
    if (!by_wave) {
        by_wave = rows >= 4096 ? top || !is_long : (rows >= 1024 && is_long) || (top && rows >= 256 && rows <= 1024);
        const uint64_t step = (by_wave && top ? 64 : kLT) * kPiece;
        parts = std::min<uint64_t>(by_wave ? 4096 / rows : (1024 + rows - 1) / rows, (vocab + step - 1) / step);
        if (top) parts = std::min<uint64_t>(parts, kMostKeys / top);
        parts = std::max<uint64_t>(1, std::min<uint64_t>(parts, kMostParts / rows));
    }
    const uint64_t len = ((vocab + parts - 1) / parts + 7) / 8 * 8;
    parts = (vocab + len - 1) / len;
    a.parts = uint32_t(parts), a.part_len = uint32_t(len);
    a.sums = static_cast<f32x4*>(ws);
    a.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + kMostParts * sizeof(f32x4));
    const uint64_t grid = by_wave ? (rows * parts + kLWaves - 1) / kLWaves : rows * parts;
    if (grid * kLT >= (uint64_t(1) << 32)) return step_fail(DCR_E_INVAL, "too many rows for one launch");
    with_type(type, [&](auto t) {
        auto go = [&](auto some) {
            constexpr bool TOP = decltype(some)::value;
            if (by_wave)
                hipLaunchKernelGGL((logprobs_wave_kernel<decltype(t), TOP>), dim3(uint32_t(grid)), dim3(kLT),
                                   TOP ? kLWaves * wave_keys(top) * 8 + sizeof(u32x4) : 0, st, a);
            else
                hipLaunchKernelGGL((logprobs_kernel<decltype(t), TOP>), dim3(uint32_t(grid)), dim3(kLT), 0, st, a);
            if (parts > 1) hipLaunchKernelGGL((logprobs_join_kernel<decltype(t), TOP>), dim3(a.rows), dim3(kLT), 0, st, a);
        };
        top ? go(std::true_type()) : go(std::false_type());
    });
    return step_launched();
}

int32_t logprobs_grad(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint64_t vocab, const void* targets,
                      uint32_t targets_bytes, float scale, const float* lse, const float* dlogp, const float* entropy,
                      const float* dentropy, void* dlogits, uint64_t d_stride, hipStream_t st) {
    int32_t rc;
    if ((rc = check_logits(logits, type, stride, rows, vocab, targets, targets_bytes, scale)) ||
        (rc = check_matrix(dlogits, type, rows, vocab, d_stride, "dlogits")))
        return rc;
    if (!rows) return DCR_OK;
    if (!targets) return step_fail(DCR_E_INVAL, "targets: NULL");
    if ((rc = check_array(lse, "lse")) || (rc = check_array(dlogp, "dlogp")) ||
        (dentropy && ((rc = check_array(dentropy, "dentropy")) || (rc = check_array(entropy, "entropy")))))
        return rc;
    LpGradArgs a{};
    a.logits = logits, a.targets = targets, a.lse = lse, a.dlogp = dlogp, a.entropy = entropy, a.dentropy = dentropy;
    a.dlogits = dlogits, a.stride = stride, a.d_stride = d_stride, a.rows = uint32_t(rows), a.vocab = uint32_t(vocab);
    a.wide_ids = targets_bytes == 8, a.scale = scale;
    // 10000 x 512 bf16 19.8 us by row, short 11.2; x 1264 21.1 and 14.7, x 2048 (8000)
    // 18.5 and 18.0, x 4096 (8000) 25.8 and 31.4
    const bool by_row = vocab >= 2048;
    const uint64_t unit = by_row ? kLT * 8 * kGU : 8;
    a.pieces = uint32_t((vocab + unit - 1) / unit);
    const uint64_t grid = by_row ? rows * a.pieces : (rows * a.pieces + kLT - 1) / kLT;
    if (grid * kLT >= (uint64_t(1) << 32)) return step_fail(DCR_E_INVAL, "too many logits for one launch");
    with_type(type, [&](auto t) {
        typedef decltype(t) T;
        const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(uint32_t(grid)), dim3(kLT), 0, st, a); };
        by_row ? go(logprobs_grad_kernel<T>) : go(logprobs_grad_short_kernel<T>);
    });
    return step_launched();
}

}  // namespace
}  // namespace dcr

extern "C" {

int32_t dcr_logprobs(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint64_t vocab, const void* targets,
                     uint32_t targets_bytes, float scale, float* logp, float* lse, float* entropy, uint32_t top,
                     int32_t* top_ids, float* top_values, void* workspace_dev, uint64_t ws_bytes, void* stream) try {
    dcr::set_error("");
    return dcr::logprobs(logits, type, stride, rows, vocab, targets, targets_bytes, scale, logp, lse, entropy, top, top_ids,
                         top_values, workspace_dev, ws_bytes, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_logprobs_grad(const void* logits, uint32_t type, uint64_t stride, uint64_t rows, uint64_t vocab,
                          const void* targets, uint32_t targets_bytes, float scale, const float* lse, const float* dlogp,
                          const float* entropy, const float* dentropy, void* dlogits, uint64_t dlogits_stride,
                          void* stream) try {
    dcr::set_error("");
    return dcr::logprobs_grad(logits, type, stride, rows, vocab, targets, targets_bytes, scale, lse, dlogp, entropy, dentropy,
                              dlogits, dlogits_stride, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

}  // extern "C"
