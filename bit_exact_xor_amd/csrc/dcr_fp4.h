// dcr_fp4.h -- what the 4-bit weight kernels share: the format, checks of a
// tensor's description, and the conversions of gfx950 they are built on.
#pragma once
#include <hip/hip_runtime.h>

#include <string>
#include <type_traits>

#include "dcr_internal.h"

namespace dcr {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kFp4BlockMx = 32, kFp4BlockNv = 16;
constexpr uint32_t fp4_block(uint32_t fmt) { return fmt == DCR_FP4_MX ? kFp4BlockMx : kFp4BlockNv; }
// tensor scales the NV format takes: below 2^117 (6 * 448 of them stay finite)
// and above 2^-100 (a threshold times the scale keeps all its bits)
constexpr float kFp4MinScale = 0x1p-100f, kFp4MaxScale = 0x1p117f;

// ---------------------------------------------------------------- host side

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int32_t fp4_fail(int32_t rc, const std::string& m) {
    set_error(m);
    return rc;
}

inline int32_t fp4_launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fp4_fail(DCR_E_HIP, std::string("launch: ") + hipGetErrorString(e));
    return DCR_OK;
}

// DCR_OK, or the refusal of a description's tensor scale
inline int32_t fp4_check_scale(const dcr_fp4_tensor* t, const std::string& w) {
    if (t->format != DCR_FP4_NV) return DCR_OK;
    if (!t->tensor_scale) return fp4_fail(DCR_E_INVAL, w + ": NULL tensor scale");
    if (reinterpret_cast<uintptr_t>(t->tensor_scale) & 3u)
        return fp4_fail(DCR_E_INVAL, w + ": tensor scale not 4-byte aligned");
    return DCR_OK;
}

// DCR_OK, or the refusal of a tensor description
inline int32_t fp4_check(const dcr_fp4_tensor* t, const char* what) {
    const std::string w = what;
    if (!t) return fp4_fail(DCR_E_INVAL, w + ": NULL description");
    if (t->format != DCR_FP4_MX && t->format != DCR_FP4_NV) return fp4_fail(DCR_E_INVAL, w + ": unknown format");
    if (t->reserved) return fp4_fail(DCR_E_INVAL, w + ": reserved field not 0");
    if (t->cols >= (uint64_t(1) << 31) || t->rows >= (uint64_t(1) << 40))
        return fp4_fail(DCR_E_INVAL, w + ": more than 2^31 - 1 columns or 2^40 - 1 rows");
    if (t->rows && t->cols) {
        if (!t->codes || !t->scales) return fp4_fail(DCR_E_INVAL, w + ": NULL codes or scales");
        if (!al16(t->codes) || !al16(t->scales)) return fp4_fail(DCR_E_INVAL, w + ": codes or scales not 16-byte aligned");
        if (t->rows > 1 && (t->code_stride < (t->cols + 1) / 2 ||
                            t->scale_stride < (t->cols + fp4_block(t->format) - 1) / fp4_block(t->format)))
            return fp4_fail(DCR_E_INVAL, w + ": a row stride is smaller than a row");
        if (t->rows > 1 && (t->code_stride >= (uint64_t(1) << 32) || t->scale_stride >= (uint64_t(1) << 32)))
            return fp4_fail(DCR_E_INVAL, w + ": row stride of 2^32 bytes or more");
        return fp4_check_scale(t, w);
    }
    return DCR_OK;
}

// -------------------------------------------------------------- device side

// Two codes of byte SEL of `c` times the power of two in `scale`'s exponent.
// The conversion is exact (two significant bits); exponent bits 0 stand for
// 2^-127 and 255 for NaN, which is how an e8m0 byte reads.
template <int SEL>
__device__ __forceinline__ bf16x2 fp4_bf16(uint32_t c, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, SEL);
}
template <int SEL>
__device__ __forceinline__ f32x2 fp4_f32(uint32_t c, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, SEL);
}
__device__ __forceinline__ float e8m0_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

// value of an e4m3 byte
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    return __builtin_amdgcn_cvt_f32_fp8(int(byte), 0);
}

// eight codes as fp32 times their block's scale: MX by its power of two, NV
// by its e4m3 value (six significant bits: exact)
template <uint32_t FMT>
__device__ __forceinline__ void fp4_unpack8(uint32_t c, uint32_t sbyte, float* v) {
    const float unit = FMT == DCR_FP4_MX ? e8m0_f32(sbyte) : 1.0f;
    f32x2 a = fp4_f32<0>(c, unit), b = fp4_f32<1>(c, unit), d = fp4_f32<2>(c, unit), e = fp4_f32<3>(c, unit);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = d[0]; v[5] = d[1]; v[6] = e[0]; v[7] = e[1];
    if (FMT == DCR_FP4_NV) {
        const float s = e4m3_f32(sbyte);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= s;
    }
}

// the same as bf16: both formats' values fit its eight significant bits
template <uint32_t FMT>
__device__ __forceinline__ bf16x8 fp4_unpack8_bf16(uint32_t c, uint32_t sbyte) {
    bf16x8 r;
    if (FMT == DCR_FP4_MX) {
        const float s = e8m0_f32(sbyte);
        const bf16x2 a = fp4_bf16<0>(c, s), b = fp4_bf16<1>(c, s), d = fp4_bf16<2>(c, s), e = fp4_bf16<3>(c, s);
        r = bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
    } else {
        float v[8];
        fp4_unpack8<FMT>(c, sbyte, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[i];
    }
    return r;
}

}  // namespace dcr
