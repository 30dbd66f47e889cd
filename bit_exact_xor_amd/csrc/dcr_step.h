// dcr_step.h -- what the calls of a training turn share (choice of experts,
// rows to experts, log probabilities, AdamW): checks of matrices, accesses of
// eight or four elements at any alignment, sums over lanes.
#pragma once
#include <hip/hip_runtime.h>

#include <string>
#include <type_traits>

#include "dcr_fp4.h"

namespace dcr {

// 16, 8 and 4 bytes at any alignment of whole elements (the hardware takes them)
typedef u32x4 u32x4_el __attribute__((aligned(2)));
typedef u32x2 u32x2_el __attribute__((aligned(2)));
typedef uint32_t u32_el __attribute__((aligned(2)));

// ---------------------------------------------------------------- host side

inline int32_t step_fail(int32_t rc, const std::string& m) { return fp4_fail(rc, m); }
inline int32_t step_launched() { return fp4_launched(); }

inline uint32_t type_bytes(uint32_t type) { return type == DCR_F32 ? 4 : 2; }

// DCR_OK, or the refusal of a matrix of fp32 or bf16
inline int32_t check_matrix(const void* x, uint32_t type, uint64_t rows, uint64_t cols, uint64_t stride, const char* what) {
    const std::string w = what;
    if (type != DCR_F32 && type != DCR_BF16) return step_fail(DCR_E_INVAL, w + ": type is neither fp32 nor bf16");
    if (!rows || !cols) return DCR_OK;
    if (!x) return step_fail(DCR_E_INVAL, w + ": NULL");
    if (reinterpret_cast<uintptr_t>(x) & (type_bytes(type) - 1)) return step_fail(DCR_E_INVAL, w + ": not aligned to its elements");
    if (rows > 1 && stride < cols) return step_fail(DCR_E_INVAL, w + ": row stride smaller than a row");
    if (rows > 1 && stride >= (uint64_t(1) << 32)) return step_fail(DCR_E_INVAL, w + ": row stride of 2^32 elements or more");
    return DCR_OK;
}

// DCR_OK, or the refusal of a contiguous array of 4-byte (or `bytes`-byte) elements
inline int32_t check_array(const void* x, const char* what, uint32_t bytes = 4) {
    if (!x) return step_fail(DCR_E_INVAL, std::string(what) + ": NULL");
    if (reinterpret_cast<uintptr_t>(x) & (bytes - 1)) return step_fail(DCR_E_INVAL, std::string(what) + ": not aligned to its elements");
    return DCR_OK;
}

inline int32_t check_step_workspace(const void* ws, uint64_t bytes) {
    if (!ws || !al16(ws)) return step_fail(DCR_E_INVAL, "workspace is NULL or not 16-byte aligned");
    if (bytes < DCR_STEP_WORKSPACE_BYTES) return step_fail(DCR_E_CAPACITY, "workspace too small");
    return DCR_OK;
}

// f(element) with the type's element (uint16_t: bf16)
template <typename F>
void with_type(uint32_t type, F&& f) {
    type == DCR_BF16 ? f(uint16_t()) : f(float());
}

// -------------------------------------------------------------- device side

__device__ __forceinline__ float wide(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
__device__ __forceinline__ float wide(float x) { return x; }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ void narrow(float x, uint16_t* p) { *p = __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ void narrow(float x, float* p) { *p = x; }

__device__ __forceinline__ void unpack2(uint32_t w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xFFFF0000u);
}

// 16 bytes that are read once, or not again before the caches have turned over:
// they leave the lines that are to the others (6 to 16 % on the large cases).
__device__ __forceinline__ u32x4 once(const u32x4_el* p) { return __builtin_nontemporal_load(p); }

// Eight elements as they lie in memory: held apart from their values so that
// loads can be on their way while others are used.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4 q;
    __device__ __forceinline__ void load(const uint16_t* p) { q = *reinterpret_cast<const u32x4_el*>(p); }
    __device__ __forceinline__ void load_once(const uint16_t* p) { q = once(reinterpret_cast<const u32x4_el*>(p)); }
    // n of them (0 .. 8), the others `rest`
    __device__ __forceinline__ void load_some(const uint16_t* p, int n, uint32_t rest) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = (2 * i < n ? uint32_t(p[2 * i]) : rest) | ((2 * i + 1 < n ? uint32_t(p[2 * i + 1]) : rest) << 16);
    }
    __device__ __forceinline__ void get(float* v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(q[i], v + 2 * i);
    }
};
template <>
struct Raw8<float> {
    u32x4 q[2];
    __device__ __forceinline__ void load(const float* p) {
        q[0] = *reinterpret_cast<const u32x4_el*>(p);
        q[1] = *reinterpret_cast<const u32x4_el*>(p + 4);
    }
    // (A line's halves go in two accesses: past the caches each would bring the whole
    // line, 20443 x 10 rows of 571 124 us instead of 107, 2048 x 100277 logits 157
    // instead of 149.)
    __device__ __forceinline__ void load_once(const float* p) { load(p); }
    __device__ __forceinline__ void load_some(const float* p, int n, uint32_t rest) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i >> 2][i & 3] = i < n ? __float_as_uint(p[i]) : rest << 16;
    }
    __device__ __forceinline__ void get(float* v) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(q[i >> 2][i & 3]);
    }
};
constexpr uint32_t kBf16MinusInf = 0xFF80u;   // `rest` of load_some: -infinity in either type

// FAR: results that fill the caches many times over before they are read go past
// them, except fp32 ones, whose lines are written in two accesses (8192 x 8 rows of
// 2048 133 us, past the caches 258)
template <bool FAR = false>
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack2(v[2 * i], v[2 * i + 1]);
    if constexpr (FAR)
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4_el*>(p));
    else
        *reinterpret_cast<u32x4_el*>(p) = q;
}
template <bool FAR = false>
__device__ __forceinline__ void store8(float* p, const float* v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x4 q = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        *reinterpret_cast<u32x4_el*>(p + 4 * h) = __builtin_bit_cast(u32x4, q);
    }
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, const float* v, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) narrow(v[i], p + i);
}

// What f makes of the values of LANES neighbouring lanes, in all of them; f
// commutes.  Registers only: permutations inside rows of 16 lanes, then swaps of
// rows and of halves (through LDS a step takes some 100 cycles, here about 8).
template <int STEP>
__device__ __forceinline__ void partners(uint32_t v, uint32_t* a, uint32_t* b) {
    if constexpr (STEP == 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        *a = p[0], *b = p[1];
    } else if constexpr (STEP == 32) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        *a = p[0], *b = p[1];
    } else {
        // neighbour; pair of a quad; the other quad of eight, the other eight (mirrored: within them all are alike by now)
        constexpr int CTRL = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
        *a = v, *b = uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xF, 0xF, true));
    }
}
template <int STEP, typename T>
__device__ __forceinline__ void partners_of(T v, T* a, T* b) {
    if constexpr (sizeof(T) == 4) {
        uint32_t x, y;
        partners<STEP>(__builtin_bit_cast(uint32_t, v), &x, &y);
        *a = __builtin_bit_cast(T, x), *b = __builtin_bit_cast(T, y);
    } else {
        const u32x2 q = __builtin_bit_cast(u32x2, v);
        u32x2 x, y;
        uint32_t lo[2], hi[2];
        partners<STEP>(q[0], &lo[0], &lo[1]);
        partners<STEP>(q[1], &hi[0], &hi[1]);
        x = u32x2{lo[0], hi[0]}, y = u32x2{lo[1], hi[1]};
        *a = __builtin_bit_cast(T, x), *b = __builtin_bit_cast(T, y);
    }
}
template <int LANES, int STEP = 1, typename T, typename F>
__device__ __forceinline__ T lanes_all(T v, F&& f) {
    if constexpr (STEP < LANES) {
        T a, b;
        partners_of<STEP>(v, &a, &b);
        return lanes_all<LANES, 2 * STEP>(f(a, b), f);
    } else {
        return v;
    }
}
template <int LANES, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
    return lanes_all<LANES>(v, [](T a, T b) { return a + b; });
}

}  // namespace dcr
