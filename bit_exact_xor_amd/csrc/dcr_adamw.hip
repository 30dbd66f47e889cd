// dcr_adamw.hip -- an AdamW step over many tensors in one launch (one for each
// combination of types that occurs).
//
//   g' = grad_scale g
//   m  = beta1 m + (1 - beta1) g'         v = beta2 v + (1 - beta2) g'^2
//   p  = p - (lr decay p + lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps))
//
// (the decay as a part of p that is taken off: a factor 1 - lr decay comes in steps
// of 6e-8, and at lr = 1e-6 and decay = 0.1 the decay itself is 1e-7)
//
// Bound by memory: everything is read once and written once, 28 bytes an
// element with fp32 states, bf16 gradients and a bf16 copy, 16.1 with states in
// 8 bits.  A workgroup takes 512 consecutive elements of a tensor and ends, so
// small tensors cost a workgroup each and no launch, and what runs at once covers
// a short stretch of every buffer (176 M elements with fp32 states 796 to 810 us;
// 1024 elements 820, in two steps 857; 4096 in four 922).  With states in 8 bits the
// arithmetic comes near: about 80 instructions an element, where 151 M take 393 us
// (with the compiler's division and root and every code's two ways 100, and 413).
//
// States in 8 bits: blocks of 32 elements under one power of two (an e8m0
// byte), e4m3 codes; of the second moment the square root is held, whose range
// is half as wide in powers of two.  A power of two as the scale makes both
// conversions exact but for the one rounding of a code.  With only three bits
// behind the leading one a moment that is rounded to nearest would stop
// following: v moves by a twentieth of itself or less, half a step is a
// sixteenth.  So a code is rounded up with the probability of the remainder
// (the dither); the random numbers are a function of the seed, the step and
// the element's index, so equal calls give equal bits, whatever the shards.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "dcr_step.h"

namespace dcr {
namespace {

constexpr uint32_t kAT = 128;                 // threads of a workgroup
constexpr uint32_t kAChunk = 4 * kAT;         // elements of a workgroup
constexpr uint32_t kAShare = 8;               // workgroups of an entry of the table
constexpr uint64_t kAMostGroups = (uint64_t(1) << 32) / kAT / kAShare * kAShare - kAShare;      // of a launch
constexpr uint32_t kStateBlock = DCR_ADAMW_BLOCK;
// Tensors of more bytes than this (the last cache holds 256 MiB) go past the
// caches (1 to 3 %).
constexpr uint64_t kFarBytes = uint64_t(256) << 20;

// what the steps of a call share
struct AdamArgs {
    float grad_scale, beta1, new1, beta2, new2;   // new: 1 - beta
    float rate, root, eps, decay;                 // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t), eps, lr decay
    uint32_t key, dither;
};

// Square root of a number well inside the range, rounded once: the hardware's
// estimate of its inverse, a step of Newton's iteration for both and the rest put
// right.
__device__ __forceinline__ float root_of(float x) {
    const float y = __builtin_amdgcn_rsqf(x);
    float s = x * y, h = 0.5f * y;
    const float e = __fmaf_rn(-h, s, 0.5f);
    s = __fmaf_rn(s, e, s), h = __fmaf_rn(h, e, h);
    return __fmaf_rn(__fmaf_rn(-s, s, x), h, s);
}

// What a workgroup does: everything of its elements in one entry, so that a small
// tensor's time is two loads behind one another, not three.  Eight consecutive
// workgroups share an entry, of 4096 elements; what is left of a tensor has entries
// of up to 512, behind those (176 M elements 3.4 MB of table, with an entry a
// workgroup 27.5, in the same time).
struct DevAdam {
    uint8_t *param, *m, *v, *m_scales, *v_scales;
    const uint8_t* grad;
    uint16_t* copy;
    uint64_t first;
    uint32_t numel, no_decay, pad[2];
};
static_assert(sizeof(DevAdam) == 80, "DevAdam");

// Odd numbers of the fractions of square roots of 2, 3, 5 and of the golden
// ratio, which spreads consecutive numbers evenly.
constexpr uint32_t kGolden = 0x9E3779B1u, kRoot2 = 0x6A09E667u, kRoot3 = 0xBB67AE85u, kRoot5 = 0x3C6EF373u;

// two 16-bit random numbers of an element i: low half for m, high half for v.  x:
// i's low half times kGolden, its high half times kRoot3 and the key, added up.
__device__ __forceinline__ uint32_t dither_of(uint32_t x) {
    x = (x ^ (x >> 16)) * kRoot2;
    x = (x ^ (x >> 15)) * kRoot5;
    return x ^ (x >> 16);
}

// Four elements at fp32 or bf16; FAR: of buffers that fill the caches many times
// over, which are then read and written past them.
template <bool FAR, typename Q, typename P>
__device__ __forceinline__ Q fetch(const P* p) {
    if constexpr (FAR)
        return __builtin_nontemporal_load(reinterpret_cast<const Q*>(p));
    else
        return *reinterpret_cast<const Q*>(p);
}
template <bool FAR, typename Q, typename P>
__device__ __forceinline__ void put(Q q, P* p) {
    if constexpr (FAR)
        __builtin_nontemporal_store(q, reinterpret_cast<Q*>(p));
    else
        *reinterpret_cast<Q*>(p) = q;
}
template <bool FAR>
__device__ __forceinline__ void load4(const float* p, float* v) {
    const u32x4 q = fetch<FAR, u32x4>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
}
template <bool FAR>
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
    const u32x2 q = fetch<FAR, u32x2>(p);
    unpack2(q[0], v);
    unpack2(q[1], v + 2);
}
template <bool FAR>
__device__ __forceinline__ void save4(float* p, const float* v) {
    put<FAR>(f32x4{v[0], v[1], v[2], v[3]}, p);
}
template <bool FAR>
__device__ __forceinline__ void save4(uint16_t* p, const float* v) {
    put<FAR>(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])}, p);
}
template <typename T>
__device__ __forceinline__ void load4_some(const T* p, float* v, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? wide(p[i]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void save4_some(T* p, const float* v, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) narrow(v[i], p + i);
}

__device__ __forceinline__ void codes4(uint32_t q, uint32_t byte, float* v) {
    const float unit = byte == 255 ? NAN : ldexpf(1.0f, int(byte) - 127);
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(q), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(q), true);
    v[0] = a[0] * unit, v[1] = a[1] * unit, v[2] = b[0] * unit, v[3] = b[1] * unit;
}

// the scale byte of a block whose largest magnitude has these bits: the least
// power of two that brings it to 448 or below
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7F800000u) return 255;
    const int e = int(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return uint32_t(max(e, 0));
}

// e4m3 code of magnitude y (at most 448): down to the code below where the rest
// is less than 1 - r / 65536 of the code's step.  Above 2^-6 the codes are the
// leading bits of the number itself, below they are multiples of 2^-9.  `some`:
// a lane of the wave has one below (else its steps are left out).
constexpr float kLeastNormal = 0x1p-6f;
__device__ __forceinline__ uint32_t code_of(float y, uint32_t r, bool some) {
    const uint32_t normal = ((__float_as_uint(y) + (r << 4)) >> 20) - (120u << 3);
    if (!some) return normal;
    asm volatile("");                                // (a branch, not both and a choice)
    return y >= kLeastNormal ? normal : uint32_t(floorf(__fmaf_rn(y, 512.0f, float(r) * 0x1p-16f)));
}

// largest of the eight lanes of a block
__device__ __forceinline__ uint32_t block_top(const float* v) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return lanes_all<8>(t, [](uint32_t a, uint32_t b) { return max(a, b); });
}

template <typename TP, typename TG, uint32_t BITS, bool FAR>
__global__ void __launch_bounds__(kAT) adamw_kernel(const DevAdam* entries, uint32_t shared, AdamArgs args, const AdamArgs* live) {
    // the first `shared` workgroups share entries
    const bool shares = blockIdx.x < shared;
    const uint32_t from = shares ? blockIdx.x % kAShare * kAChunk : 0;      // the workgroup's first element of the entry's
    const DevAdam t = entries[shares ? blockIdx.x / kAShare : blockIdx.x - shared + shared / kAShare];
    const AdamArgs a = live ? *live : args;
    const float decay = t.no_decay ? 0.0f : a.decay;
    const uint32_t i = from + threadIdx.x * 4;
    const int n = i < t.numel ? int(min(4u, t.numel - i)) : 0;
    TP* pp = reinterpret_cast<TP*>(t.param) + i;
    const TG* gp = reinterpret_cast<const TG*>(t.grad) + i;
    float p[4], g[4], m[4], v[4], w[4];
    if (n == 4) {
        load4<FAR>(pp, p);
        load4<FAR>(gp, g);
    } else {
        load4_some(pp, p, n);
        load4_some(gp, g, n);
    }
    if (BITS == 32) {
        float *mp = reinterpret_cast<float*>(t.m) + i, *vp = reinterpret_cast<float*>(t.v) + i;
        if (n == 4) {
            load4<FAR>(mp, m);
            load4<FAR>(vp, v);
        } else {
            load4_some(mp, m, n);
            load4_some(vp, v, n);
        }
    } else {
        uint32_t mq = 0, vq = 0, mb = 0, vb = 0;
        if (n) {
            if (n == 4) {
                mq = fetch<FAR, uint32_t>(t.m + i);
                vq = fetch<FAR, uint32_t>(t.v + i);
            } else {
                for (int j = 0; j < n; ++j) {
                    mq |= uint32_t(t.m[i + j]) << (8 * j);
                    vq |= uint32_t(t.v[i + j]) << (8 * j);
                }
            }
            mb = t.m_scales[i / kStateBlock];
            vb = t.v_scales[i / kStateBlock];
        }
        codes4(mq, mb, m);
        codes4(vq, vb, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= v[j];
    }
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float s = g[j] * a.grad_scale;
        m[j] = __fmaf_rn(m[j], a.beta1, s * a.new1);
        v[j] = __fmaf_rn(v[j], a.beta2, s * s * a.new2);
        odd |= !(v[j] >= 0x1p-90f && v[j] <= 0x1p90f);
    }
    const bool plain = BITS == 8 && !__any(odd);     // (fp32 states: memory alone bounds the step)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (plain) {
            asm volatile("");                        // (a branch, not both and a choice)
            w[j] = root_of(v[j]);
        } else {
            asm volatile("");
            w[j] = sqrtf(v[j]);
        }
        // (8 bits: the hardware's reciprocal, one step off, where instructions are as
        // near a bound as the memory; with fp32 states the division costs no time)
        const float den = __fmaf_rn(w[j], a.root, a.eps);
        const float u = BITS == 8 ? a.rate * m[j] * __builtin_amdgcn_rcpf(den) : a.rate * m[j] / den;
        // (an infinite parameter stays what it is, as one that a mask is held in)
        p[j] -= __fmaf_rn(__builtin_amdgcn_fmed3f(p[j], -0x1.fffffep127f, 0x1.fffffep127f), decay, u);
    }
    if (n == 4)
        save4<FAR>(pp, p);
    else
        save4_some(pp, p, n);
    if (t.copy) n == 4 ? save4<FAR>(t.copy + i, p) : save4_some(t.copy + i, p, n);
    if (BITS == 32) {
        float *mp = reinterpret_cast<float*>(t.m) + i, *vp = reinterpret_cast<float*>(t.v) + i;
        if (n == 4) {
            save4<FAR>(mp, m);
            save4<FAR>(vp, v);
        } else {
            save4_some(mp, m, n);
            save4_some(vp, v, n);
        }
    } else {
        // (behind the end moments and gradients are 0, as a block of zeros has them)
        const uint32_t mb = scale_byte(block_top(m)), wb = scale_byte(block_top(w));
        float ym[4], yw[4];
        float least = INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ym[j] = fabsf(ldexpf(m[j], 127 - int(mb))), yw[j] = ldexpf(w[j], 127 - int(wb));
            least = fminf(least, fminf(ym[j], yw[j]));
        }
        const bool some = __any(least < kLeastNormal);
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = uint32_t(t.first), hi = uint32_t(t.first >> 32) * kRoot3 + a.key;
            x[j] = (lo * kGolden + hi) + i * kGolden + j * kGolden;
            x[j] += i + j > ~lo ? kRoot3 : 0;    // (i + j carry into the high half)
        }
        uint32_t mq = 0, wq = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t rm = 0x8000u, rw = 0x8000u;
            if (a.dither) {
                const uint32_t r = dither_of(x[j]);
                rm = r & 0xFFFFu, rw = r >> 16;
            }
            const uint32_t cm = code_of(ym[j], rm, some);
            uint32_t cw = code_of(yw[j], rw, some);
            cw = max(cw, w[j] > 0.0f ? 1u : 0u); // (0 would make the next update one of eps)
            mq |= (cm | (__float_as_uint(m[j]) >> 31) << 7) << (8 * j);
            wq |= cw << (8 * j);
        }
        if (mb == 255) mq = 0;
        if (wb == 255) wq = 0;
        if (n == 4) {
            put<FAR>(mq, t.m + i);
            put<FAR>(wq, t.v + i);
        } else {
            for (int j = 0; j < n; ++j) {
                t.m[i + j] = uint8_t(mq >> (8 * j));
                t.v[i + j] = uint8_t(wq >> (8 * j));
            }
        }
        if (n && i % kStateBlock == 0) {
            t.m_scales[i / kStateBlock] = uint8_t(mb);
            t.v_scales[i / kStateBlock] = uint8_t(wb);
        }
    }
}

// x^n by squaring, alike on the host and the GPU
__host__ __device__ inline double power(double x, uint64_t n) {
    double r = 1.0;
    for (; n; n >>= 1, x *= x)
        if (n & 1) r *= x;
    return r;
}

__host__ __device__ inline AdamArgs adam_args(const dcr_adamw_args& h, double step, double lr, double grad_scale) {
    AdamArgs a{};
    const uint64_t t = uint64_t(step);
    a.grad_scale = float(grad_scale);
    a.beta1 = float(h.beta1), a.new1 = float(1.0 - h.beta1), a.beta2 = float(h.beta2), a.new2 = float(1.0 - h.beta2);
    a.rate = float(lr / (1.0 - power(h.beta1, t)));
    a.root = float(1.0 / sqrt(1.0 - power(h.beta2, t)));
    a.eps = float(h.eps), a.decay = float(lr * h.weight_decay);
    a.key = uint32_t(h.dither_seed) * kGolden + uint32_t(t) * kRoot2, a.dither = h.dither_seed ? 1 : 0;
    return a;
}

// the step's arguments from device memory: step, lr, grad_scale
__global__ void adamw_live_kernel(dcr_adamw_args h, AdamArgs* out) {
    *out = adam_args(h, h.live[0], h.live[1], h.live[2]);
}

constexpr uint32_t kVariants = 8;             // param type | gradient type | bits

}  // namespace
}  // namespace dcr

struct dcr_adamw_plan {
    std::vector<uint8_t> blob;                // AdamArgs of a live step | entries, by variant: shared ones, then others
    uint64_t off_entries = 0;
    uint64_t first[dcr::kVariants + 1] = {}, shared[dcr::kVariants] = {};      // entries
    uint8_t* dev = nullptr;
    bool far = false;                         // more than the caches hold
};

namespace dcr {
namespace {

int32_t check_adam(const dcr_adamw_tensor& t, uint64_t at) {
    const std::string w = "tensor " + std::to_string(at);
    if (t.param_type > DCR_BF16 || t.grad_type > DCR_BF16) return step_fail(DCR_E_INVAL, w + ": type is neither fp32 nor bf16");
    if (t.state_bits != 8 && t.state_bits != 32) return step_fail(DCR_E_INVAL, w + ": state_bits is neither 8 nor 32");
    if (t.flags & ~uint32_t(DCR_ADAMW_NO_DECAY)) return step_fail(DCR_E_INVAL, w + ": unknown flag");
    if (t.numel > (uint64_t(1) << 40)) return step_fail(DCR_E_INVAL, w + ": more than 2^40 elements");
    if (!t.numel) return DCR_OK;
    if (!t.param || !t.grad || !t.m || !t.v) return step_fail(DCR_E_INVAL, w + ": NULL");
    if (!al16(t.param) || !al16(t.grad) || !al16(t.m) || !al16(t.v) || !al16(t.copy))
        return step_fail(DCR_E_INVAL, w + ": a buffer is not 16-byte aligned");
    if (t.state_bits == 8 && (!t.m_scales || !t.v_scales)) return step_fail(DCR_E_INVAL, w + ": NULL scales");
    if (t.copy && t.param_type != DCR_F32) return step_fail(DCR_E_INVAL, w + ": a bf16 copy is of fp32 parameters");
    return DCR_OK;
}

// whether memory that the step writes is written or read through another tensor too
bool overlaps(const dcr_adamw_tensor* tensors, uint64_t n) {
    struct Range {
        uintptr_t from, to;
        bool written;
    };
    std::vector<Range> r;
    const auto add = [&](const void* at, uint64_t bytes, bool written) {
        if (at && bytes) r.push_back({reinterpret_cast<uintptr_t>(at), reinterpret_cast<uintptr_t>(at) + bytes, written});
    };
    for (uint64_t i = 0; i < n; ++i) {
        const dcr_adamw_tensor& t = tensors[i];
        const uint64_t state = t.numel * (t.state_bits / 8), scales = t.state_bits == 8 ? (t.numel + kStateBlock - 1) / kStateBlock : 0;
        add(t.param, t.numel * type_bytes(t.param_type), true);
        add(t.grad, t.numel * type_bytes(t.grad_type), false);
        add(t.m, state, true), add(t.v, state, true);
        add(t.m_scales, scales, true), add(t.v_scales, scales, true);
        add(t.copy, t.numel * 2, true);
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
    uintptr_t any = 0, written = 0;
    for (const Range& x : r) {
        if (x.from < (x.written ? any : written)) return true;
        any = std::max(any, x.to);
        if (x.written) written = std::max(written, x.to);
    }
    return false;
}

int32_t adamw_build(const dcr_adamw_tensor* tensors, uint64_t n, dcr_adamw_plan& p) {
    constexpr uint64_t kEntry = uint64_t(kAChunk) * kAShare;
    uint64_t chunks = 0, bytes = 0, others[kVariants] = {};
    const auto variant = [](const dcr_adamw_tensor& t) { return t.param_type | t.grad_type << 1 | (t.state_bits == 8 ? 4u : 0u); };
    for (uint64_t i = 0; i < n; ++i) {
        const dcr_adamw_tensor& t = tensors[i];
        if (int32_t rc = check_adam(t, i)) return rc;
        chunks += (t.numel + kAChunk - 1) / kAChunk;
        if (chunks >= (uint64_t(1) << 28)) return step_fail(DCR_E_INVAL, "2^37 elements or more");
        p.shared[variant(t)] += t.numel / kEntry;
        others[variant(t)] += (t.numel % kEntry + kAChunk - 1) / kAChunk;
    }
    if (overlaps(tensors, n)) return step_fail(DCR_E_INVAL, "buffers of the tensors overlap");
    p.off_entries = (sizeof(AdamArgs) + 15) / 16 * 16;
    uint64_t to[kVariants][2];                // where the next entry goes
    for (uint32_t k = 0; k < kVariants; ++k) {
        to[k][0] = p.first[k], to[k][1] = p.first[k] + p.shared[k];
        p.first[k + 1] = to[k][1] + others[k];
    }
    p.blob.resize(p.off_entries + p.first[kVariants] * sizeof(DevAdam));
    for (uint64_t i = 0; i < n; ++i) {
        const dcr_adamw_tensor& t = tensors[i];
        const uint32_t p_bytes = type_bytes(t.param_type), g_bytes = type_bytes(t.grad_type), s_bytes = t.state_bits / 8;
        bytes += t.numel * (p_bytes + g_bytes + 2 * s_bytes + (t.copy ? 2 : 0));
        for (uint64_t at = 0, size; at < t.numel; at += size) {
            const bool shares = t.numel - at >= kEntry;
            size = shares ? kEntry : std::min<uint64_t>(kAChunk, t.numel - at);
            DevAdam d{};
            d.param = static_cast<uint8_t*>(t.param) + at * p_bytes, d.grad = static_cast<const uint8_t*>(t.grad) + at * g_bytes;
            d.m = static_cast<uint8_t*>(t.m) + at * s_bytes, d.v = static_cast<uint8_t*>(t.v) + at * s_bytes;
            if (t.state_bits == 8) {
                d.m_scales = static_cast<uint8_t*>(t.m_scales) + at / kStateBlock;
                d.v_scales = static_cast<uint8_t*>(t.v_scales) + at / kStateBlock;
            }
            if (t.copy) d.copy = static_cast<uint16_t*>(t.copy) + at;
            d.first = t.first + at, d.numel = uint32_t(size);
            d.no_decay = t.flags & DCR_ADAMW_NO_DECAY;
            memcpy(p.blob.data() + p.off_entries + to[variant(t)][!shares]++ * sizeof(DevAdam), &d, sizeof(d));
        }
    }
    p.far = bytes > kFarBytes;
    return DCR_OK;
}

bool fraction(double x) { return x >= 0.0 && x < 1.0; }

int32_t adamw_step(const dcr_adamw_plan* p, const dcr_adamw_args* h, hipStream_t st) {
    if (!p || !h) return step_fail(DCR_E_INVAL, "NULL argument");
    if (!p->dev) return step_fail(DCR_E_INVAL, "plan not uploaded");
    if (h->reserved) return step_fail(DCR_E_INVAL, "reserved field not 0");
    if (!fraction(h->beta1) || !fraction(h->beta2)) return step_fail(DCR_E_INVAL, "beta1 or beta2 is not in [0, 1)");
    if (!(h->eps >= 0x1p-100 && h->eps < INFINITY)) return step_fail(DCR_E_INVAL, "eps is below 2^-100 or not finite");
    if (!std::isfinite(h->weight_decay)) return step_fail(DCR_E_INVAL, "weight_decay is not finite");
    if (!h->live && (!h->step || h->step > (uint64_t(1) << 53))) return step_fail(DCR_E_INVAL, "step is not 1 .. 2^53");
    if (!h->live && (!std::isfinite(h->lr) || !std::isfinite(h->grad_scale)))
        return step_fail(DCR_E_INVAL, "lr or grad_scale is not finite");
    if (reinterpret_cast<uintptr_t>(h->live) & 7u) return step_fail(DCR_E_INVAL, "live is not 8-byte aligned");
    AdamArgs a{};
    AdamArgs* live = nullptr;
    if (h->live) {
        live = reinterpret_cast<AdamArgs*>(p->dev);
        hipLaunchKernelGGL(adamw_live_kernel, dim3(1), dim3(1), 0, st, *h, live);
    } else {
        a = adam_args(*h, double(h->step), h->lr, h->grad_scale);
    }
    const DevAdam* entries = reinterpret_cast<const DevAdam*>(p->dev + p->off_entries);
    for (uint32_t k = 0; k < kVariants; ++k) {
        with_type(k & 1, [&](auto tp) {
            with_type(k >> 1 & 1, [&](auto tg) {
                typedef decltype(tp) TP;
                typedef decltype(tg) TG;
                const auto go = [&](auto kernel) {
                    // entries that are shared, then the others, as many as a launch takes
                    for (uint64_t e = p->first[k], left = p->shared[k]; e < p->first[k + 1];) {
                        const uint64_t both = std::min(left, kAMostGroups / kAShare);
                        const uint64_t one = both < left ? 0 : std::min(p->first[k + 1] - e - both, kAMostGroups - both * kAShare);
                        hipLaunchKernelGGL(kernel, dim3(uint32_t(both * kAShare + one)), dim3(kAT), 0, st, entries + e,
                                           uint32_t(both * kAShare), a, live);
                        e += both + one, left -= both;
                    }
                };
                if (k & 4)
                    go(p->far ? adamw_kernel<TP, TG, 8, true> : adamw_kernel<TP, TG, 8, false>);
                else
                    go(p->far ? adamw_kernel<TP, TG, 32, true> : adamw_kernel<TP, TG, 32, false>);
            });
        });
    }
    return step_launched();
}

}  // namespace
}  // namespace dcr

extern "C" {

int32_t dcr_adamw_plan_build(const dcr_adamw_tensor* tensors, uint64_t n, dcr_adamw_plan** out) try {
    using namespace dcr;
    set_error("");
    if (!out) return step_fail(DCR_E_INVAL, "out is NULL");
    *out = nullptr;
    if (n && !tensors) return step_fail(DCR_E_INVAL, "tensors: NULL");
    if (n >= (uint64_t(1) << 31)) return step_fail(DCR_E_INVAL, "2^31 tensors or more");
    dcr_adamw_plan* p = new (std::nothrow) dcr_adamw_plan();
    if (!p) return step_fail(DCR_E_NOMEM, "out of host memory");
    int32_t rc;
    try {
        rc = adamw_build(tensors, n, *p);
    } catch (...) {
        rc = step_fail(DCR_E_NOMEM, "out of host memory");
    }
    if (rc) {
        delete p;
        return rc;
    }
    *out = p;
    return DCR_OK;
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_adamw_plan_bytes(const dcr_adamw_plan* plan, uint64_t* bytes) try {
    using namespace dcr;
    set_error("");
    if (!plan || !bytes) return step_fail(DCR_E_INVAL, "NULL argument");
    *bytes = plan->blob.size();
    return DCR_OK;
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_adamw_plan_upload(dcr_adamw_plan* plan, void* table_dev, uint64_t bytes, void* stream) try {
    using namespace dcr;
    set_error("");
    if (!plan || !table_dev) return step_fail(DCR_E_INVAL, "NULL argument");
    if (!al16(table_dev)) return step_fail(DCR_E_INVAL, "table not 16-byte aligned");
    if (bytes < plan->blob.size()) return step_fail(DCR_E_CAPACITY, "table too small");
    const hipError_t e = hipMemcpyAsync(table_dev, plan->blob.data(), plan->blob.size(), hipMemcpyHostToDevice,
                                        static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return step_fail(DCR_E_HIP, std::string("plan upload: ") + hipGetErrorString(e));
    plan->dev = static_cast<uint8_t*>(table_dev);
    return DCR_OK;
} catch (...) {
    return DCR_E_NOMEM;
}

void dcr_adamw_plan_destroy(dcr_adamw_plan* plan) { delete plan; }

int32_t dcr_adamw_step(const dcr_adamw_plan* plan, const dcr_adamw_args* args, void* stream) try {
    dcr::set_error("");
    return dcr::adamw_step(plan, args, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

}  // extern "C"
