// dcr_fp4_mm.h -- what the kernels of the 4-bit products share: their
// arguments, the walk through grouped rows, and loads and stores at any
// alignment.
#pragma once
#include "dcr_fp4.h"

namespace dcr {

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

struct MArgs {
    const void* x;              // bf16 rows, or the codes of 4-bit ones
    const uint8_t* xs;          // scales of 4-bit rows
    const uint8_t* wc;          // codes of the weights
    const uint8_t* ws;          // their scales
    const float* tensor_scale;  // NV
    const int32_t* offsets;
    void* y;
    uint64_t m, x_stride, xs_stride, wc_stride, ws_stride, y_stride;
    uint32_t n, k, groups;      // of one group; k = w->cols
    uint32_t x_vec, w_vec;      // rows of x / codes of w start on 16-byte borders
    uint32_t y_vec;             // rows of y start on 16-byte borders
    uint32_t row_tiles, col_tiles;   // upper bounds of the grid
};

struct RowTile {
    uint32_t group;
    uint64_t begin, end;        // rows of the tile; begin = end: past the last
};

// Tile `t` of BM rows, counted through the groups in order (a tile never
// spans two groups).  Every wave looks through the offsets, 64 groups at a
// time: tiles of each by its lane, their running sum by lane exchange.
template <uint32_t BM>
__device__ __forceinline__ RowTile row_tile(const MArgs& a, uint64_t t) {
    if (!a.offsets) {
        const uint64_t b = t * BM;
        return {0, min(b, a.m), min(b + BM, a.m)};
    }
    const uint32_t lane = threadIdx.x & 63u;
    const int64_t top = int64_t(a.m);
    for (uint32_t g0 = 0; g0 < a.groups; g0 += 64) {
        const uint32_t g = g0 + lane;
        int64_t lo = 0, hi = 0;
        if (g < a.groups) {
            lo = min(max(int64_t(a.offsets[g]), int64_t(0)), top);
            hi = min(max(int64_t(a.offsets[g + 1]), lo), top);
        }
        const uint32_t tiles = uint32_t((uint64_t(hi - lo) + BM - 1) / BM);
        uint32_t sum = tiles;
#pragma unroll
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint32_t o = uint32_t(__shfl_up(int(sum), d, 64));
            if (lane >= d) sum += o;
        }
        const uint32_t all = uint32_t(__builtin_amdgcn_readlane(int(sum), 63));
        if (t < all) {
            const uint64_t hit = __ballot(t < sum);
            const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
            // the same in every lane: kept in scalar registers
            auto of_lane = [&](uint32_t v) { return uint32_t(__builtin_amdgcn_readlane(int(v), l)); };
            const uint32_t before = of_lane(sum - tiles);
            const uint64_t first = of_lane(uint32_t(lo)), last = of_lane(uint32_t(hi));
            const uint64_t b = first + (t - before) * BM;
            return {g0 + uint32_t(l), b, min(b + BM, last)};
        }
        t -= all;
    }
    return {0, 0, 0};
}

// 16 codes of a row from element c0 (a multiple of 16); zeros from `cols` on
__device__ __forceinline__ u32x2 codes16(const uint8_t* row, uint32_t c0, uint32_t cols, bool vec) {
    u32x2 r = {0u, 0u};
    if (c0 + 16 <= cols) {
        if (vec) return *reinterpret_cast<const u32x2*>(row + c0 / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i / 4] |= uint32_t(row[c0 / 2 + i]) << (8 * (i & 3));
        return r;
    }
    if (c0 >= cols) return r;
    const uint32_t n = cols - c0;       // 1 .. 15
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
        if (2 * i >= n) break;
        uint32_t b = row[c0 / 2 + i];
        if (2 * i + 1 == n) b &= 15u;
        r[i / 4] |= b << (8 * (i & 3));
    }
    return r;
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
    *reinterpret_cast<bf16x4*>(p) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
}

// Buffer descriptor: loads take a scalar base and step and a 32-bit lane
// offset, and give zeros at offsets of `bytes` or more.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
constexpr uint32_t kOutside = 0x80000000u;   // a lane offset past every descriptor's range

// 16 x 16 products of 128 codes each way, every lane's 32 codes with the power
// of two in byte WB / XB of its scale words.
typedef int i32x8 __attribute__((ext_vector_type(8)));
template <uint32_t WB, uint32_t XB>
__device__ __forceinline__ f32x4 mfma_fp4(u32x4 w, u32x4 x, f32x4 c, uint32_t ws, uint32_t xs) {
    const i32x8 p = {int(w[0]), int(w[1]), int(w[2]), int(w[3]), 0, 0, 0, 0};
    const i32x8 q = {int(x[0]), int(x[1]), int(x[2]), int(x[3]), 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, c, 4, 4, WB, int(ws), XB, int(xs));
}

// Rows of 128 bytes in LDS: piece c (16 bytes) of row r at place
// c ^ swizzle8(r).  A 128-bit read serves 16 lanes at a time: rows 0-3 and
// 12-15 of one quad with rows 4-11 of the quad beside, whose pieces differ in
// one of the low two bits; each half gets half of the places, and two rows
// fill the banks once (no conflicts counted).
__device__ __forceinline__ uint32_t swizzle8(uint32_t r) {
    return ((r >> 1) & 3u) | (((r >> 3) ^ (r >> 2)) & 1u) << 2;
}

// Waits until at most N of this wave's loads are in flight and its LDS reads
// are done, then for the other waves of the workgroup.
template <uint32_t N>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes a lane from memory straight to LDS: lane i's at lds + 16 i (`lds`
// the same in every lane).
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t lane_off, uint32_t off) {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, lane_off, off, 0, 0);
#endif
}

// Makes the compiler have `v` in its register here: products whose sums are
// held stay in front of the branches and barriers that follow.
__device__ __forceinline__ void held(f32x4& v) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" : "+v"(v));
#endif
}

// Row and column tile of a workgroup.  The eight compute dies take workgroups
// in turn: each gets a run of tiles, walked four row tiles at a time, so that
// its L2 serves a block of both operands.
struct TilePlace {
    uint32_t row, col, id;
};
__device__ __forceinline__ TilePlace tile_place(const MArgs& a, uint32_t id) {
    const uint32_t per = a.row_tiles * a.col_tiles / 8;
    if (id < per * 8) id = (id & 7u) * per + (id >> 3);
    constexpr uint32_t SM = 4;
    const uint32_t strip = id / (SM * a.col_tiles), in = id - strip * SM * a.col_tiles;
    const uint32_t sm = min(SM, a.row_tiles - strip * SM);
    return {strip * SM + in % sm, in / sm, id};
}

// loop over compile-time indices
template <uint32_t N, uint32_t I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<uint32_t, I>{});
        static_for<N, I + 1>(f);
    }
}

// The sums of a wave, times s, rounded once.  A lane holds four neighbouring
// results of one row in each 16 x 16 subtile: written as they are they make
// 32-byte pieces of lines, which costs as much time as the product itself.
// They go through LDS (`lds`: LB bytes of this wave alone) and leave as whole
// rows of the wave's tile, 128 or 256 bytes each.  16-byte pieces of a row sit
// at place p ^ row, which spreads both directions over the banks.
template <typename OUT, uint32_t MI, uint32_t NI, uint32_t LB>
__device__ __forceinline__ void store_tile(const MArgs& a, const f32x4 (&acc)[NI][MI], float s, const RowTile& rt,
                                           uint32_t rows, uint32_t row0, uint32_t col0, uint32_t outs, uint8_t* lds) {
    constexpr uint32_t E = 16 / sizeof(OUT), PR = NI * 16 / E, RB = PR * 16;     // elements of a piece, pieces, bytes of a row
    constexpr uint32_t MP = LB / RB / 16 < MI ? LB / RB / 16 : MI, RI = 64 / PR; // row subtiles of a pass, rows of a store
    static_assert(MP && MI % MP == 0 && 64 % PR == 0, "store_tile");
    const uint32_t lane = threadIdx.x & 63u, r16 = lane & 15u, quad = lane >> 4;
    const uint32_t piece = lane % PR, col = col0 + piece * E;
#pragma unroll
    for (uint32_t p = 0; p < MI / MP; ++p) {
#pragma unroll
        for (uint32_t m = 0; m < MP; ++m)
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) {
                const f32x4 v = acc[i][p * MP + m] * s;
                uint8_t* row = lds + (m * 16 + r16) * RB;
                if constexpr (sizeof(OUT) == 4)
                    store4(reinterpret_cast<float*>(row + ((i * 4 + quad) ^ (r16 & (PR - 1))) * 16), v);
                else
                    store4(reinterpret_cast<uint16_t*>(row + ((i * 2 + quad / 2) ^ (r16 & (PR - 1))) * 16 + (quad & 1u) * 8), v);
            }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (uint32_t i = 0; i < MP * 16 / RI; ++i) {
            const uint32_t lr = i * RI + lane / PR, r = row0 + p * MP * 16 + lr;
            const u32x4 v = *reinterpret_cast<const u32x4*>(lds + lr * RB + (piece ^ (lr & (PR - 1))) * 16);
            if (r >= rows) continue;
            OUT* out = static_cast<OUT*>(a.y) + (rt.begin + r) * a.y_stride + col;
            if (a.y_vec && col + E <= outs) {
                *reinterpret_cast<u32x4*>(out) = v;
            } else {
#pragma unroll
                for (uint32_t e = 0; e < E; ++e)
                    if (col + e < outs) {
                        if constexpr (sizeof(OUT) == 4)
                            out[e] = __uint_as_float(v[e]);
                        else
                            out[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
                    }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

// Tile size (256 or 128) and grid of a product with `outs` columns of
// results; 0 if there would be too many tiles.
inline uint32_t tile_grid(MArgs* a, uint32_t outs, uint32_t* grid) {
    uint32_t bm = 0;
    for (uint32_t b : {256u, 128u}) {
        const uint64_t rows = (a->m + b - 1) / b + (a->offsets ? a->groups : 0), cols = (uint64_t(outs) + b - 1) / b;
        if (rows * cols >= (1u << 22)) return 0;
        a->row_tiles = uint32_t(rows);
        a->col_tiles = uint32_t(cols);
        *grid = uint32_t(rows * cols);
        bm = b;
        if (!a->offsets && rows * cols >= 192) break;
    }
    return bm;
}

// kernels for parts of the range (false: not for these arguments)
bool fp4_mm_tile(MArgs a, uint32_t fmt, bool f32, hipStream_t st);
bool fp4_mm_rows(MArgs a, bool xq, uint32_t fmt, bool f32, hipStream_t st);
bool fp4_mm_tile4(MArgs a, bool f32, hipStream_t st);
bool fp4_mm_grad(MArgs a, uint32_t fmt, bool f32, hipStream_t st);

}  // namespace dcr
