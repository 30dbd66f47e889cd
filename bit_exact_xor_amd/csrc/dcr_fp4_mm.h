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
    uint32_t chunk, grid;            // neighbouring workgroups of one compute die; workgroups
    uint32_t splits, split_steps;    // parts of the sum, steps of a part (even)
    uint64_t split_elems;            // results of a part (y is then fp32 scratch)
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

// 32 codes of a row from element k; zeros from `cols` on
__device__ __forceinline__ u32x4 codes32(const uint8_t* row, uint32_t k, uint32_t cols, bool vec) {
    if (vec && k + 32 <= cols) return *reinterpret_cast<const u32x4*>(row + k / 2);
    const u32x2 a = codes16(row, k, cols, false), b = codes16(row, k + 16, cols, false);
    return u32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
    *reinterpret_cast<bf16x4*>(p) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
}

// The eight elements at `p`, any alignment, moved down by `past`: zeros move in.
__device__ __forceinline__ u32x4 last_elements(const uint8_t* p, uint32_t past) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    uint64_t lo = v[0] | uint64_t(v[1]) << 32, hi = v[2] | uint64_t(v[3]) << 32;
    const uint32_t bits = min(past, 8u) * 16, n = bits & 63u;
    lo = bits >= 64 ? hi : lo, hi = bits >= 64 ? 0 : hi;
    lo = n ? lo >> n | hi << (64 - n) : lo, hi >>= n;
    lo = bits >= 128 ? 0 : lo;
    return u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
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

// Waits until at most N of this wave's loads are in flight (they finish in
// order) and its LDS accesses are done, then for the other waves of the
// workgroup.  Loads to LDS are waited for here and nowhere else: a plain
// workgroup barrier does not cover them.
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

// Row and column tile of a workgroup, and its part of the sum.  The eight
// compute dies take workgroups in turn: each gets runs of `chunk` neighbouring
// tiles, walked four row tiles at a time, so that its L2 serves a block of
// both operands.
struct TilePlace {
    uint32_t row, col, split;
};
__device__ __forceinline__ TilePlace tile_place(const MArgs& a) {
    const uint32_t die = blockIdx.x & 7u, local = blockIdx.x >> 3, turn = local / a.chunk;
    const uint32_t id = (turn * 8 + die) * a.chunk + (local - turn * a.chunk);
    const uint32_t tile = id / a.splits, split = id - tile * a.splits;
    constexpr uint32_t SM = 4;
    const uint32_t strip = tile / (SM * a.col_tiles), in = tile - strip * SM * a.col_tiles;
    if (strip * SM >= a.row_tiles) return {a.row_tiles, 0, 0};     // (the grid is whole chunks)
    const uint32_t sm = min(SM, a.row_tiles - strip * SM);
    if (in >= sm * a.col_tiles) return {a.row_tiles, 0, 0};
    return {strip * SM + in % sm, in / sm, split};
}

// loop over compile-time indices
template <uint32_t N, uint32_t I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<uint32_t, I>{});
        static_for<N, I + 1>(f);
    }
}

// Row of a tile that is kept in row `l` of LDS: where WM waves share the rows
// they take every WM-th 16 of them, so that a tile that is less than half full
// is half of the work for each (tiles of 256 rows have no such form).
template <uint32_t BM, uint32_t WM>
__device__ __forceinline__ uint32_t tile_row(uint32_t l) {
    if constexpr (WM == 1 || BM == 256) return l;
    constexpr uint32_t R = BM / WM;
    return (l % R / 16 * WM + l / R) * 16 + (l & 15u);
}

// A workgroup's BM x BN sums, times s, rounded once.  A lane holds four
// neighbouring results of one row in each 16 x 16 subtile: stored as they are
// they make 32-byte pieces of lines, which cost as much time as the product
// itself (205 of 457 us at 8192 x 14336 x 4096 in 4 bits).  They go through
// LDS, half of a pass's rows in `lo` and half in `hi` (HB bytes each, unused
// by then), and leave as whole rows of the tile.  16-byte pieces of a row sit
// at place p ^ row, which spreads both directions over the banks.
// WM waves share the rows (see tile_row), `wm` this one's part; its columns
// start at `wcol`.
template <typename OUT, uint32_t BM, uint32_t BN, uint32_t W, uint32_t WM, uint32_t HB, uint32_t MI, uint32_t NI>
__device__ __forceinline__ void store_block(const MArgs& a, const f32x4 (&acc)[NI][MI], float s, const RowTile& rt,
                                            const TilePlace& at, uint32_t wm, uint32_t wcol, uint32_t outs, uint8_t* lo,
                                            uint8_t* hi) {
    constexpr uint32_t E = 16 / sizeof(OUT), RB = BN * sizeof(OUT), PR = RB / 16;   // elements of a piece; bytes, pieces of a row
    constexpr uint32_t HR = HB / RB < BM / 2 ? HB / RB : BM / 2, RP = 2 * HR;       // rows of a half, of a pass
    constexpr uint32_t RPW = RP / WM, RI = W * 64 / PR;                             // rows of a wave in a pass; of a store
    static_assert(HR % 16 == 0 && BM % RP == 0 && HR % RI == 0 && (WM == 1 || RPW == HR), "store_block");
    const uint32_t lane = threadIdx.x & 63u, r16 = lane & 15u, quad = lane >> 4;
    const uint32_t rows = uint32_t(rt.end - rt.begin), piece = threadIdx.x % PR, row_in = threadIdx.x / PR;
    const uint32_t col = at.col * BN + piece * E;
    OUT* y = static_cast<OUT*>(a.y) + at.split * a.split_elems;
#pragma unroll
    for (uint32_t p = 0; p < BM / RP; ++p) {
        __syncthreads();
#pragma unroll
        for (uint32_t m = 0; m < RPW / 16; ++m) {
            const bool up = WM == 1 ? m * 16 >= HR : wm != 0;
            uint8_t* row = (up ? hi : lo) + ((WM == 1 && up ? m * 16 - HR : m * 16) + r16) * RB;
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) {
                const f32x4 v = acc[i][p * (RPW / 16) + m] * s;
                const uint32_t c = wcol + i * 16 + quad * 4;
                if constexpr (sizeof(OUT) == 4)
                    store4(reinterpret_cast<float*>(row + ((c / 4) ^ r16) * 16), v);
                else
                    store4(reinterpret_cast<uint16_t*>(row + ((c / 8) ^ r16) * 16 + (quad & 1u) * 8), v);
            }
        }
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < RP / RI; ++i) {
            const bool up = i * RI >= HR;
            const uint32_t lr = (up ? i * RI - HR : i * RI) + row_in;      // in its half
            const u32x4 v = *reinterpret_cast<const u32x4*>((up ? hi : lo) + lr * RB + (piece ^ (lr & 15u)) * 16);
            const uint32_t r = tile_row<BM, WM>(WM == 1 ? p * RP + i * RI + row_in : (up ? BM / 2 : 0) + p * RPW + lr);
            if (r >= rows) continue;
            OUT* out = y + (rt.begin + r) * a.y_stride + col;
            if (col + E <= outs) {
                __builtin_memcpy(out, &v, 16);   // (at any alignment)
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
    }
}

// Most row tiles of b rows that offsets over m rows can make: a group that is
// not empty ends in one short tile at most.
inline uint64_t row_tile_bound(const MArgs& a, uint64_t b) {
    if (!a.offsets) return (a.m + b - 1) / b;
    const uint64_t g = a.m < a.groups ? a.m : a.groups;
    return g + (a.m - g) / b;
}

// Sums that the kernels below take are shorter: a single row has no stride to
// limit its length, and past 2^30 elements kOutside would lie inside it.
constexpr uint32_t kLongest = 1u << 26;

// kernels for parts of the range (false: not for these arguments)
bool fp4_mm_tile(MArgs a, uint32_t fmt, bool f32, void* ws, hipStream_t st);
bool fp4_mm_rows(MArgs a, bool xq, uint32_t fmt, bool f32, hipStream_t st);
bool fp4_mm_tile4(MArgs a, bool f32, void* ws, hipStream_t st);
bool fp4_mm_grad(MArgs a, uint32_t fmt, bool f32, void* ws, hipStream_t st);
// Chooses the tiling of a product with `outs` columns of results and `steps`
// steps of the sum, and fills in the grid; steps' costs in cycles of a compute
// unit by rows of a tile (256, 128, 64, 32; 0: there is none).  Returns the rows of a
// tile, 0 if no grid fits.
uint32_t fp4_mm_plan(MArgs* a, uint32_t outs, uint32_t steps, const uint32_t (&cost)[4]);
// With a->splits > 1: points a copy's y at the scratch, and joins the parts.
MArgs fp4_mm_parts(const MArgs& a, uint32_t outs, void* ws);
void fp4_mm_join(const MArgs& a, uint32_t outs, uint32_t fmt, bool f32, const void* ws, hipStream_t st);

}  // namespace dcr
