// dcr_fp4.hip -- 4-bit weights: quantisation and reading back (gfx950).
//
// A row is cut into blocks (32 elements in the MX format, 16 in the NV one);
// each block has one scale byte and each element a 4-bit e2m1 code
// (0 .5 1 1.5 2 3 4 6 and a sign), two codes a byte.
//   MX: scale 2^(byte - 127), byte = max(exponent bits of max|x| - 2, 0)
//   NV: scale e4m3(max|x| / (6 s)) times the tensor's fp32 scale s
// code = the nearest e2m1 value of x / scale, ties to the even code, beyond 6
// to 6.  Every decision is the one exact arithmetic gives, so a refit that
// quantises the same weights again gets the same bytes.
//
// Both directions are bound by memory: 2 (4) bytes of an element against 17/32
// or 9/16 of a byte, a few vector instructions an element.  A lane takes 16
// bytes of the wide side (8 bf16 or 4 fp32 elements), so that a wave's loads
// and stores are whole lines; the lanes of a block share its maximum by lane
// exchange, with no LDS and no second pass.  4096 x 4096 in bf16 takes 9.4 us
// to MX and 6.9 us back (42 MB each way, 4.5 and 6.1 TB/s: it fits the caches),
// 151936 x 2048 109 us back (788 MB, 7.2 TB/s); 12288 x 2048 in fp32 (101 MB)
// 17 us for the NV tensor scale, 21 us to NV and 19 us back.
#include "dcr_fp4.h"

namespace dcr {
namespace {

constexpr uint32_t kQT = 256;      // threads of a workgroup
constexpr uint32_t kQU = 4;        // 16-byte pieces a lane has in flight
constexpr uint32_t kParts = 1024;  // workgroups (and partial maxima) of a calibration

struct QArgs {
    const void* x;            // wide side (read by quantise, written by dequantise)
    uint8_t* codes;
    uint8_t* scales;
    float* tensor_scale;
    const uint32_t* parts;    // partial maxima of a calibration, or NULL
    uint64_t rows, x_stride, code_stride, scale_stride;
    uint64_t items;           // rows * per_row
    uint32_t cols, per_row;   // per_row: lane pieces of a row, whole blocks
};

// 16 bytes of the wide side at its elements' alignment, and the codes of as
// many elements at any: one access each on gfx950
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;
typedef uint16_t __attribute__((aligned(1))) u16_any;

// elements of a lane's piece: 16 bytes of the wide side; 32 where an NV scale
// is to be found for fp32 values, which costs a lane as much as eight codes
template <typename T, bool NV_SCALES = false>
constexpr uint32_t kPiece = sizeof(T) == 2 ? 8 : NV_SCALES ? 8 : 4;

// row and column of a lane's piece: the workgroup's first piece is divided
// once in 64 bits, the rest is a 32-bit step from there
struct Place {
    uint64_t row;
    uint32_t piece;
};
__device__ __forceinline__ Place place(uint64_t row0, uint32_t piece0, uint32_t step, uint32_t per_row) {
    const uint32_t p = piece0 + step;
    if (p < per_row) return {row0, p};
    const uint32_t q = p / per_row;
    return {row0 + q, p - q * per_row};
}

// maximum of |x|'s bits over the LANES lanes of a block
template <uint32_t LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
#pragma unroll
    for (uint32_t d = 1; d < LANES; d <<= 1) v = max(v, uint32_t(__shfl_xor(int(v), int(d), 64)));
    return v;
}

__device__ __forceinline__ uint32_t wg_max(uint32_t v, uint32_t* lds) {
#pragma unroll
    for (uint32_t d = 32; d; d >>= 1) v = max(v, uint32_t(__shfl_xor(int(v), int(d), 64)));
    if ((threadIdx.x & 63u) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t r = lds[0];
    for (uint32_t i = 1; i < blockDim.x / 64; ++i) r = max(r, lds[i]);
    return r;
}

// the scale a calibration gives for the largest finite |x|
__device__ __forceinline__ float calibrated(uint32_t amax_bits) {
    if (!amax_bits) return 1.0f;
    return fminf(fmaxf(__fdiv_rn(__uint_as_float(amax_bits), 2688.0f), kFp4MinScale), kFp4MaxScale);
}

// value and gap to the next of e4m3 index i (0 .. 126)
__device__ __forceinline__ float e4m3_gap(uint32_t i) { return __uint_as_float((max(i >> 3, 1u) + 117u) << 23); }
__device__ __forceinline__ float e4m3_val(uint32_t i) {
    return (i < 8 ? float(i) : float(8 + (i & 7u))) * e4m3_gap(i);
}

// Index of the e4m3 value nearest amax / (6 s), ties to even, at most 448.
// The conversion instruction rounds the quotient computed in fp32, off by less
// than 2^-21 of itself: moved that far down and up it gives the same index, or
// the borders decide.  6 * border has seven significant bits, so the sign of
// fma(-6 border, s, amax) is exact.
__device__ __forceinline__ uint32_t nv_scale(float amax, float s, float inv6s) {
    const float lo = fminf(amax * (inv6s * (1.0f - 0x1p-20f)), 448.0f), hi = fminf(amax * (inv6s * (1.0f + 0x1p-20f)), 448.0f);
    const uint32_t pk = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, 0, false));
    const uint32_t i = pk & 255u;
    if (i == ((pk >> 8) & 255u)) return i;
    const float d = __fmaf_rn(-6.0f * (e4m3_val(i) + 0.5f * e4m3_gap(i)), s, amax);
    return i + ((d > 0.0f || (d == 0.0f && (i & 1u))) ? 1u : 0u);
}

// code of x at block scale b, tensor scale s, by exact comparison with the
// seven borders (a border times b has seven significant bits)
__device__ __forceinline__ uint32_t nv_code_exact(float x, float b, float s) {
    const float a = fabsf(x);
    const float t[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const float d = __fmaf_rn(-t[i] * b, s, a);
        c += (d > 0.0f || (d == 0.0f && (i & 1))) ? 1u : 0u;
    }
    return c | ((__float_as_uint(x) >> 31) << 3);
}

// Eight codes (4 bits each) of v at scales b and s: found like the scale.
__device__ __forceinline__ uint32_t nv_codes(const float* v, float b, float s) {
    const float r = __builtin_amdgcn_rcpf(b * s), dn = r * (1.0f - 0x1p-20f), up = r * (1.0f + 0x1p-20f);
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[0] * dn, v[1] * dn, 1.0f, 0);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[0] * up, v[1] * up, 1.0f, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[2] * dn, v[3] * dn, 1.0f, 1);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[2] * up, v[3] * up, 1.0f, 1);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[4] * dn, v[5] * dn, 1.0f, 2);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[4] * up, v[5] * up, 1.0f, 2);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[6] * dn, v[7] * dn, 1.0f, 3);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[6] * up, v[7] * up, 1.0f, 3);
    if (lo != hi) {
        lo = 0;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) lo |= nv_code_exact(v[i], b, s) << (4 * i);
    }
    return lo;
}

// a lane's E elements as fp32 (zeros past the row's end) and max |bits|
// (LAST: not read again by this call)
template <typename T, uint32_t E, bool LAST>
__device__ __forceinline__ void load_piece(const T* row, uint32_t c0, uint32_t cols, float* v) {
    if (c0 + E <= cols) {
        const auto* from = reinterpret_cast<const u32x4_any*>(row + c0);
        const u32x4 q = LAST ? u32x4(__builtin_nontemporal_load(from)) : u32x4(*from);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(q[i] << 16);
                v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q[i]);
            if constexpr (E == 8) {
                const u32x4 p = LAST ? u32x4(__builtin_nontemporal_load(from + 1)) : u32x4(from[1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 + i] = __uint_as_float(p[i]);
            }
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < E; ++i) {
            float f = 0.0f;
            if (c0 + i < cols) {
                if constexpr (sizeof(T) == 2)
                    f = __uint_as_float(uint32_t(row[c0 + i]) << 16);
                else
                    f = row[c0 + i];
            }
            v[i] = f;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kQT) fp4_amax_kernel(QArgs a, uint32_t* parts) {
    constexpr uint32_t E = kPiece<T, true>;
    __shared__ uint32_t lds[kQT / 64];
    uint32_t m = 0;
    const uint64_t step = uint64_t(gridDim.x) * kQT * kQU;
    for (uint64_t base = uint64_t(blockIdx.x) * kQT * kQU; base < a.items; base += step) {
        const uint64_t row0 = base / a.per_row;
        const uint32_t piece0 = uint32_t(base - row0 * a.per_row);
#pragma unroll
        for (uint32_t u = 0; u < kQU; ++u) {
            const uint32_t off = u * kQT + threadIdx.x;
            if (base + off >= a.items) continue;
            const Place p = place(row0, piece0, off, a.per_row);
            float v[E];
            load_piece<T, E, false>(static_cast<const T*>(a.x) + p.row * a.x_stride, p.piece * E, a.cols, v);
#pragma unroll
            for (uint32_t i = 0; i < E; ++i) {
                const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
                m = max(m, b < 0x7F800000u ? b : 0u);
            }
        }
    }
    m = wg_max(m, lds);
    if (threadIdx.x == 0) parts[blockIdx.x] = m;
}

template <typename T, uint32_t FMT>
__global__ void __launch_bounds__(kQT) fp4_quantize_kernel(QArgs a) {
    constexpr uint32_t E = kPiece<T, FMT == DCR_FP4_NV>, LANES = fp4_block(FMT) / E;
    float s = 1.0f;
    if constexpr (FMT == DCR_FP4_NV) {
        if (a.parts) {
            __shared__ uint32_t lds[kQT / 64];
            uint32_t m = 0;
            for (uint32_t i = threadIdx.x; i < kParts; i += kQT) m = max(m, a.parts[i]);
            s = calibrated(wg_max(m, lds));
            if (blockIdx.x == 0 && threadIdx.x == 0) *a.tensor_scale = s;
        } else {
            s = *a.tensor_scale;
        }
    }
    const float inv6s = FMT == DCR_FP4_NV ? __frcp_rn(6.0f * s) : 0.0f;
    const bool usable = FMT == DCR_FP4_MX || (s >= kFp4MinScale && s <= kFp4MaxScale);
    const uint64_t base = uint64_t(blockIdx.x) * kQT * kQU;
    const uint64_t row0 = base / a.per_row;
    const uint32_t piece0 = uint32_t(base - row0 * a.per_row);
    float v[kQU][E];
    Place p[kQU];
#pragma unroll
    for (uint32_t u = 0; u < kQU; ++u) {
        const uint32_t off = u * kQT + threadIdx.x;
        p[u] = place(row0, piece0, off, a.per_row);
        if (base + off < a.items) {
            load_piece<T, E, true>(static_cast<const T*>(a.x) + p[u].row * a.x_stride, p[u].piece * E, a.cols, v[u]);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < E; ++i) v[u][i] = 0.0f;
        }
    }
#pragma unroll
    for (uint32_t u = 0; u < kQU; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (uint32_t i = 0; i < E; ++i) m = max(m, __float_as_uint(v[u][i]) & 0x7FFFFFFFu);
        m = block_max<LANES>(m);
        const bool finite = usable && m < 0x7F800000u;
        uint32_t sbyte, c = 0;
        if constexpr (FMT == DCR_FP4_MX) {
            sbyte = finite ? max(m >> 23, 2u) - 2u : 255u;
            const float unit = e8m0_f32(sbyte);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][0], v[u][1], unit, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][2], v[u][3], unit, 1);
            if constexpr (E == 8) {
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][4], v[u][5], unit, 2);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[u][6], v[u][7], unit, 3);
            }
        } else {
            sbyte = finite ? nv_scale(__uint_as_float(m), s, inv6s) : 127u;
            if (finite && sbyte) {
                c = nv_codes(v[u], e4m3_f32(sbyte), s);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < E; ++i) c |= (__float_as_uint(v[u][i]) >> 31) << (4 * i + 3);
            }
        }
        if (!finite) c = 0;
        if (base + u * kQT + threadIdx.x >= a.items) continue;
        const uint32_t c0 = p[u].piece * E;
        if (c0 >= a.cols) continue;     // a lane behind the row's end, in its last block
        uint8_t* out = a.codes + p[u].row * a.code_stride + c0 / 2;
        if (c0 + E <= a.cols) {
            if constexpr (E == 8)
                *reinterpret_cast<u32_any*>(out) = c;
            else
                *reinterpret_cast<u16_any*>(out) = uint16_t(c);
        } else {
            const uint32_t n = min(E, a.cols - c0);
            if (n < 8) c &= (1u << (4 * n)) - 1u;
            for (uint32_t i = 0; i < (n + 1) / 2; ++i) out[i] = uint8_t(c >> (8 * i));
        }
        if (p[u].piece % LANES == 0) a.scales[p[u].row * a.scale_stride + p[u].piece / LANES] = uint8_t(sbyte);
    }
}

template <typename T, uint32_t FMT>
__global__ void __launch_bounds__(kQT) fp4_dequantize_kernel(QArgs a) {
    constexpr uint32_t E = kPiece<T>, LANES = fp4_block(FMT) / E;
    const float s = FMT == DCR_FP4_NV ? *a.tensor_scale : 1.0f;
    const uint64_t base = uint64_t(blockIdx.x) * kQT * kQU;
    const uint64_t row0 = base / a.per_row;
    const uint32_t piece0 = uint32_t(base - row0 * a.per_row);
    uint32_t c[kQU], sb[kQU];
    Place p[kQU];
    bool live[kQU];
#pragma unroll
    for (uint32_t u = 0; u < kQU; ++u) {
        const uint32_t off = u * kQT + threadIdx.x;
        p[u] = place(row0, piece0, off, a.per_row);
        const uint32_t c0 = p[u].piece * E;
        live[u] = base + off < a.items && c0 < a.cols;
        c[u] = sb[u] = 0;
        if (!live[u]) continue;
        const uint8_t* in = a.codes + p[u].row * a.code_stride + c0 / 2;
        if (c0 + E <= a.cols) {
            if constexpr (E == 8)
                c[u] = *reinterpret_cast<const u32_any*>(in);
            else
                c[u] = *reinterpret_cast<const u16_any*>(in);
        } else {
            const uint32_t n = min(E, a.cols - c0);
            for (uint32_t i = 0; i < (n + 1) / 2; ++i) c[u] |= uint32_t(in[i]) << (8 * i);
        }
        sb[u] = a.scales[p[u].row * a.scale_stride + p[u].piece / LANES];
    }
#pragma unroll
    for (uint32_t u = 0; u < kQU; ++u) {
        if (!live[u]) continue;
        const uint32_t c0 = p[u].piece * E;
        float v[8];
        fp4_unpack8<FMT>(c[u], sb[u], v);
        if (FMT == DCR_FP4_NV) {
#pragma unroll
            for (uint32_t i = 0; i < E; ++i) v[i] *= s;   // one rounding: code times scale is exact
        }
        T* out = static_cast<T*>(const_cast<void*>(a.x)) + p[u].row * a.x_stride + c0;
        if constexpr (sizeof(T) == 2) {
            uint16_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
            if (c0 + E <= a.cols) {
                u32x4 q;
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = h[2 * i] | (uint32_t(h[2 * i + 1]) << 16);
                __builtin_nontemporal_store(q, reinterpret_cast<u32x4_any*>(out));
            } else {
                for (uint32_t i = 0; i < min(E, a.cols - c0); ++i) out[i] = h[i];
            }
        } else {
            if (c0 + E <= a.cols) {
                const f32x4 q = {v[0], v[1], v[2], v[3]};
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, q), reinterpret_cast<u32x4_any*>(out));
            } else {
                for (uint32_t i = 0; i < min(E, a.cols - c0); ++i) out[i] = v[i];
            }
        }
    }
}

// the kernels' arguments for a tensor and its wide side, E elements a piece; false if there is
// nothing to do
bool plan_pieces(const dcr_fp4_tensor& t, const void* x, uint32_t E, uint64_t x_stride, QArgs* a) {
    if (!t.rows || !t.cols) return false;
    const uint32_t B = fp4_block(t.format);
    QArgs r{};
    r.x = x;
    r.codes = static_cast<uint8_t*>(t.codes);
    r.scales = static_cast<uint8_t*>(t.scales);
    r.tensor_scale = t.tensor_scale;
    r.rows = t.rows;
    r.x_stride = t.rows > 1 ? x_stride : t.cols;
    r.code_stride = t.code_stride;
    r.scale_stride = t.scale_stride;
    uint64_t cols = t.cols;
    // rows that follow one another without a gap, in whole blocks, are one
    // long row: no piece then needs a division
    if (t.rows > 1 && cols % B == 0 && x_stride == cols && t.code_stride == cols / 2 && t.scale_stride == cols / B &&
        t.rows * cols < (uint64_t(1) << 32) - B) {
        cols *= t.rows;
        r.rows = 1;
    }
    r.cols = uint32_t(cols);
    r.per_row = uint32_t((cols + B - 1) / B) * (B / E);
    r.items = r.rows * r.per_row;
    *a = r;
    return true;
}

int32_t check_wide(const void* x, uint32_t type, uint64_t stride, const dcr_fp4_tensor& t, const char* what) {
    const std::string w = what;
    if (type != DCR_F32 && type != DCR_BF16) return fp4_fail(DCR_E_INVAL, w + ": type is neither fp32 nor bf16");
    if (!t.rows || !t.cols) return DCR_OK;
    if (!x) return fp4_fail(DCR_E_INVAL, w + ": NULL");
    if (reinterpret_cast<uintptr_t>(x) & (type == DCR_F32 ? 3u : 1u))
        return fp4_fail(DCR_E_INVAL, w + ": not aligned to its elements");
    if (t.rows > 1 && stride < t.cols) return fp4_fail(DCR_E_INVAL, w + ": row stride smaller than a row");
    if (t.rows > 1 && stride >= (uint64_t(1) << 40)) return fp4_fail(DCR_E_INVAL, w + ": row stride of 2^40 elements or more");
    return DCR_OK;
}

// f(element type, format) with the types and formats as compile-time values
template <typename F>
void dispatch(uint32_t type, uint32_t fmt, F&& f) {
    const std::integral_constant<uint32_t, DCR_FP4_MX> mx;
    const std::integral_constant<uint32_t, DCR_FP4_NV> nv;
    if (type == DCR_BF16)
        fmt == DCR_FP4_MX ? f(uint16_t(), mx) : f(uint16_t(), nv);
    else
        fmt == DCR_FP4_MX ? f(float(), mx) : f(float(), nv);
}

int32_t quantize(const void* x, uint32_t x_type, uint64_t x_stride, const dcr_fp4_tensor* q, uint32_t options,
                 void* ws, uint64_t ws_bytes, hipStream_t st) {
    int32_t rc = fp4_check(q, "quantised tensor");
    if (rc) return rc;
    if (options & ~uint32_t(DCR_FP4_CALIBRATE)) return fp4_fail(DCR_E_INVAL, "unknown option");
    const bool calibrate = options & DCR_FP4_CALIBRATE;
    if (calibrate && q->format != DCR_FP4_NV) return fp4_fail(DCR_E_INVAL, "only the NV format has a tensor scale to calibrate");
    if ((rc = check_wide(x, x_type, x_stride, *q, "source"))) return rc;
    QArgs a;
    if (!plan_pieces(*q, x, x_type == DCR_F32 && q->format == DCR_FP4_MX ? 4 : 8, x_stride, &a)) return DCR_OK;
    const uint64_t grid = (a.items + kQT * kQU - 1) / (kQT * kQU);
    if (grid >= (uint64_t(1) << 32) / kQT) return fp4_fail(DCR_E_INVAL, "tensor too large for one launch");
    if (calibrate) {
        if (!ws || !al16(ws)) return fp4_fail(DCR_E_INVAL, "workspace is NULL or not 16-byte aligned");
        if (ws_bytes < kParts * sizeof(uint32_t)) return fp4_fail(DCR_E_CAPACITY, "workspace too small");
        uint32_t* parts = static_cast<uint32_t*>(ws);
        if (x_type == DCR_BF16)
            hipLaunchKernelGGL((fp4_amax_kernel<uint16_t>), dim3(kParts), dim3(kQT), 0, st, a, parts);
        else
            hipLaunchKernelGGL((fp4_amax_kernel<float>), dim3(kParts), dim3(kQT), 0, st, a, parts);
        a.parts = parts;
    }
    dispatch(x_type, q->format, [&](auto elem, auto fmt) {
        hipLaunchKernelGGL((fp4_quantize_kernel<decltype(elem), decltype(fmt)::value>), dim3(uint32_t(grid)), dim3(kQT), 0, st, a);
    });
    return fp4_launched();
}

int32_t dequantize(const dcr_fp4_tensor* q, void* y, uint32_t y_type, uint64_t y_stride, hipStream_t st) {
    int32_t rc = fp4_check(q, "quantised tensor");
    if (rc) return rc;
    if ((rc = check_wide(y, y_type, y_stride, *q, "destination"))) return rc;
    QArgs a;
    if (!plan_pieces(*q, y, y_type == DCR_F32 ? 4 : 8, y_stride, &a)) return DCR_OK;
    const uint64_t grid = (a.items + kQT * kQU - 1) / (kQT * kQU);
    if (grid >= (uint64_t(1) << 32) / kQT) return fp4_fail(DCR_E_INVAL, "tensor too large for one launch");
    dispatch(y_type, q->format, [&](auto elem, auto fmt) {
        hipLaunchKernelGGL((fp4_dequantize_kernel<decltype(elem), decltype(fmt)::value>), dim3(uint32_t(grid)), dim3(kQT), 0, st, a);
    });
    return fp4_launched();
}

}  // namespace
}  // namespace dcr

extern "C" {

int32_t dcr_fp4_quantize(const void* x, uint32_t x_type, uint64_t x_stride, const dcr_fp4_tensor* q, uint32_t options,
                         void* workspace_dev, uint64_t ws_bytes, void* stream) try {
    dcr::set_error("");
    return dcr::quantize(x, x_type, x_stride, q, options, workspace_dev, ws_bytes, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_fp4_dequantize(const dcr_fp4_tensor* q, void* y, uint32_t y_type, uint64_t y_stride, void* stream) try {
    dcr::set_error("");
    return dcr::dequantize(q, y, y_type, y_stride, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

}  // extern "C"
