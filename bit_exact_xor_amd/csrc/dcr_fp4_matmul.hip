// dcr_fp4_matmul.hip -- products with 4-bit weights (gfx950).
//
//   y[i, j] = sum_k x[i, k] w[j, k]          dcr_fp4_matmul, dcr_fp4_matmul_q
//   dx[i, k] = sum_j dy[i, j] w[j, k]        dcr_fp4_matmul_grad
//
// A 4-bit value times its block's scale has at most six significant bits, so
// it is exact as bf16 and the matrix instructions take it as an operand with
// no loss; the tensor scale of the NV format multiplies the finished sum.
#include <algorithm>
#include <cmath>

#include "dcr_fp4_mm.h"

namespace dcr {
namespace {

// ------------------------------------------------------------ general tile
//
// 64 x 64 results a workgroup, sums over 64 at a time: both operands go to
// LDS as bf16 and four waves multiply 32 x 32 each.  Takes every size, stride
// and alignment, and is left with what the rows and tiles of the other files do
// not take: row strides from 2^21 elements on, sums below 8 and from 2^26 on,
// grids from 2^22 tiles on.
constexpr uint32_t kGT = 64, kGPad = 72;

template <bool GRAD, bool XQ, uint32_t WF, typename OUT>
__global__ void __launch_bounds__(256) fp4_mm_general_kernel(MArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t xt[kGT][kGPad], wt[kGT][kGPad];
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6;
    const uint32_t outs = GRAD ? a.k : a.n, red = GRAD ? a.n : a.k;
    const float s = WF == DCR_FP4_NV ? *a.tensor_scale : 1.0f;
    const uint64_t tiles = uint64_t(a.row_tiles) * a.col_tiles;
    for (uint64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const uint64_t mt = tile / a.col_tiles;
        const uint32_t o0 = uint32_t(tile - mt * a.col_tiles) * kGT;
        const RowTile rt = row_tile<kGT>(a, mt);
        if (rt.begin == rt.end) break;
        const uint64_t w0 = uint64_t(rt.group) * a.n;
        f32x4 acc[2][2] = {};
        for (uint32_t r0 = 0; r0 < red; r0 += kGT) {
            __syncthreads();
            {   // x: thread = 16 elements of a row
                const uint32_t row = t >> 2, c = r0 + (t & 3u) * 16;
                u32x4 v[2] = {};
                if (rt.begin + row < rt.end && c < red) {
                    if constexpr (XQ) {
                        const uint8_t* xr = static_cast<const uint8_t*>(a.x) + (rt.begin + row) * a.x_stride;
                        const u32x2 q = codes16(xr, c, red, a.x_vec);
                        const uint32_t sb = a.xs[(rt.begin + row) * a.xs_stride + c / 32];
                        v[0] = __builtin_bit_cast(u32x4, fp4_unpack8_bf16<DCR_FP4_MX>(q[0], sb));
                        v[1] = __builtin_bit_cast(u32x4, fp4_unpack8_bf16<DCR_FP4_MX>(q[1], sb));
                    } else {
                        const uint16_t* xr = static_cast<const uint16_t*>(a.x) + (rt.begin + row) * a.x_stride + c;
                        if (a.x_vec && c + 16 <= red) {
                            v[0] = reinterpret_cast<const u32x4*>(xr)[0];
                            v[1] = reinterpret_cast<const u32x4*>(xr)[1];
                        } else {
#pragma unroll
                            for (uint32_t i = 0; i < 16; ++i)
                                if (c + i < red) v[i / 8][(i / 2) & 3] |= uint32_t(xr[i]) << (16 * (i & 1));
                        }
                    }
                }
                *reinterpret_cast<u32x4*>(&xt[row][(t & 3u) * 16]) = v[0];
                *reinterpret_cast<u32x4*>(&xt[row][(t & 3u) * 16 + 8]) = v[1];
            }
            {   // w: thread = 16 elements of a row of w
                const uint32_t row = t >> 2, c16 = (t & 3u) * 16;
                const uint32_t j = (GRAD ? r0 : o0) + row, c = (GRAD ? o0 : r0) + c16;
                bf16x8 v[2] = {};
                if (j < a.n && c < a.k) {
                    const u32x2 q = codes16(a.wc + (w0 + j) * a.wc_stride, c, a.k, a.w_vec);
                    const uint32_t sb = a.ws[(w0 + j) * a.ws_stride + c / fp4_block(WF)];
                    v[0] = fp4_unpack8_bf16<WF>(q[0], sb);
                    v[1] = fp4_unpack8_bf16<WF>(q[1], sb);
                }
                if constexpr (GRAD) {
                    const u32x4 h[2] = {__builtin_bit_cast(u32x4, v[0]), __builtin_bit_cast(u32x4, v[1])};
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        wt[c16 + i][row] = uint16_t(h[i / 8][(i / 2) & 3] >> (16 * (i & 1)));
                } else {
                    *reinterpret_cast<bf16x8*>(&wt[row][c16]) = v[0];
                    *reinterpret_cast<bf16x8*>(&wt[row][c16 + 8]) = v[1];
                }
            }
            __syncthreads();
#pragma unroll
            for (uint32_t kk = 0; kk < kGT; kk += 32) {
                bf16x8 xa[2], wb[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t r = i * 16 + (lane & 15u), c = kk + (lane >> 4) * 8;
                    xa[i] = *reinterpret_cast<const bf16x8*>(&xt[(wave & 1u) * 32 + r][c]);
                    wb[i] = *reinterpret_cast<const bf16x8*>(&wt[(wave >> 1) * 32 + r][c]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], xa[i], acc[i][j], 0, 0, 0);
            }
        }
        // a lane holds four neighbouring results of one row
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t row = rt.begin + (wave & 1u) * 32 + i * 16 + (lane & 15u);
            if (row >= rt.end) continue;
            OUT* out = static_cast<OUT*>(a.y) + row * a.y_stride;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t c = o0 + (wave >> 1) * 32 + j * 16 + (lane >> 4) * 4;
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r)
                    if (c + r < outs) store_out(out + c + r, acc[i][j][r] * s);
            }
        }
    }
}

// ------------------------------------------------------------ joined parts
//
// Parts of a sum in fp32, [split][row][column]: added in order, four results a
// thread, times the tensor scale, rounded once.
template <uint32_t WF, typename OUT>
__global__ void __launch_bounds__(256) fp4_mm_join_kernel(MArgs a, const float* part, uint32_t outs, uint32_t stride) {
    const uint32_t quads = stride / 4, id = blockIdx.x * 256 + threadIdx.x;
    const uint32_t row = id / quads, c = (id - row * quads) * 4;
    if (row >= a.m) return;
    if (a.offsets && (int64_t(row) < int64_t(a.offsets[0]) || int64_t(row) >= int64_t(a.offsets[a.groups]))) return;
    const float* p = part + uint64_t(row) * stride + c;
    f32x4 v = *reinterpret_cast<const f32x4*>(p);
    for (uint32_t i = 1; i < a.splits; ++i) v += *reinterpret_cast<const f32x4*>(p + i * a.split_elems);
    if (WF == DCR_FP4_NV) v *= *a.tensor_scale;
    OUT* out = static_cast<OUT*>(a.y) + uint64_t(row) * a.y_stride + c;
    if (a.y_vec && c + 4 <= outs) {
        store4(out, v);
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (c + e < outs) store_out(out + e, v[e]);
    }
}

// ---------------------------------------------------------------- host side

constexpr uint32_t kMaxGrid = 1u << 20;   // workgroups of the general kernel; more tiles are walked

int32_t check_rows(const void* p, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t elem, const char* what) {
    const std::string w = what;
    if (!rows || !cols) return DCR_OK;
    if (!p) return fp4_fail(DCR_E_INVAL, w + ": NULL");
    if (reinterpret_cast<uintptr_t>(p) & (elem - 1)) return fp4_fail(DCR_E_INVAL, w + ": not aligned to its elements");
    if (rows > 1 && stride < cols) return fp4_fail(DCR_E_INVAL, w + ": row stride smaller than a row");
    if (rows > 1 && stride >= (uint64_t(1) << 40)) return fp4_fail(DCR_E_INVAL, w + ": row stride of 2^40 elements or more");
    return DCR_OK;
}

template <bool GRAD, bool XQ, uint32_t WF>
void launch_general(const MArgs& a, bool f32, uint32_t grid, hipStream_t st) {
    if (f32)
        hipLaunchKernelGGL((fp4_mm_general_kernel<GRAD, XQ, WF, float>), dim3(grid), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((fp4_mm_general_kernel<GRAD, XQ, WF, uint16_t>), dim3(grid), dim3(256), 0, st, a);
}

// Shared host path of the three products; xq: 4-bit x, else bf16 rows.
int32_t product(bool grad, const dcr_fp4_tensor* xq, const void* x, uint64_t m, uint64_t x_stride,
                const dcr_fp4_tensor* w, const int32_t* offsets, uint32_t n_groups, void* y, uint32_t y_type,
                uint64_t y_stride, void* ws, uint64_t ws_bytes, hipStream_t st) {
    int32_t rc = fp4_check(w, "weights");
    if (rc) return rc;
    if (xq) {
        if ((rc = fp4_check(xq, "x"))) return rc;
        if (xq->format != DCR_FP4_MX || w->format != DCR_FP4_MX)
            return fp4_fail(DCR_E_INVAL, "a product of two 4-bit operands takes the MX format");
        if (xq->cols != w->cols) return fp4_fail(DCR_E_INVAL, "x and the weights differ in columns");
        m = xq->rows;
    }
    if (!n_groups || w->rows % n_groups) return fp4_fail(DCR_E_INVAL, "n_groups does not divide the weights' rows");
    if (n_groups > 1 && !offsets) return fp4_fail(DCR_E_INVAL, "offsets is NULL");
    if (n_groups > 65536) return fp4_fail(DCR_E_INVAL, "more than 65536 groups");
    if (reinterpret_cast<uintptr_t>(offsets) & 3u) return fp4_fail(DCR_E_INVAL, "offsets not 4-byte aligned");
    if (y_type != DCR_F32 && y_type != DCR_BF16) return fp4_fail(DCR_E_INVAL, "result type is neither fp32 nor bf16");
    const uint64_t n = w->rows / n_groups, k = w->cols;
    if (m >= (uint64_t(1) << 31) || n >= (uint64_t(1) << 31))
        return fp4_fail(DCR_E_INVAL, "2^31 or more rows of x or of a group");
    const uint64_t outs = grad ? k : n, red = grad ? n : k;
    if (!xq && (rc = check_rows(x, m, red, x_stride, 2, grad ? "dy" : "x"))) return rc;
    if ((rc = check_rows(y, m, outs, y_stride, y_type == DCR_F32 ? 4 : 2, grad ? "dx" : "y"))) return rc;
    if (!ws || !al16(ws)) return fp4_fail(DCR_E_INVAL, "workspace is NULL or not 16-byte aligned");
    if (ws_bytes < DCR_FP4_WORKSPACE_BYTES) return fp4_fail(DCR_E_CAPACITY, "workspace too small");
    if (!m || !outs) return DCR_OK;
    // (sums of nothing are zeros that the kernels multiply with the scale too)
    if ((rc = fp4_check_scale(w, "weights"))) return rc;
    MArgs a{};
    a.x = xq ? xq->codes : x;
    a.m = m;
    a.x_stride = m > 1 ? (xq ? xq->code_stride : x_stride) : 0;
    if (xq) {
        a.xs = static_cast<const uint8_t*>(xq->scales);
        a.xs_stride = m > 1 ? xq->scale_stride : 0;
    }
    a.wc = static_cast<const uint8_t*>(w->codes);
    a.ws = static_cast<const uint8_t*>(w->scales);
    a.wc_stride = w->rows > 1 ? w->code_stride : 0;
    a.ws_stride = w->rows > 1 ? w->scale_stride : 0;
    a.tensor_scale = w->tensor_scale;
    a.offsets = offsets;
    a.y = y;
    a.y_stride = m > 1 ? y_stride : 0;
    a.n = uint32_t(n);
    a.k = uint32_t(k);
    a.groups = n_groups;
    a.x_vec = al16(a.x) && (a.x_stride * (xq ? 1 : 2)) % 16 == 0;
    a.w_vec = a.wc_stride % 16 == 0;
    const bool f32 = y_type == DCR_F32, mx = w->format == DCR_FP4_MX;
    a.y_vec = al16(y) && (a.y_stride * (f32 ? 4 : 2)) % 16 == 0;
    if (!grad && fp4_mm_rows(a, xq != nullptr, w->format, f32, st)) return fp4_launched();
    if (!xq && !grad && fp4_mm_tile(a, w->format, f32, ws, st)) return fp4_launched();
    if (xq && fp4_mm_tile4(a, f32, ws, st)) return fp4_launched();
    if (grad && fp4_mm_grad(a, w->format, f32, ws, st)) return fp4_launched();
    a.row_tiles = uint32_t(row_tile_bound(a, kGT));
    a.col_tiles = uint32_t((outs + kGT - 1) / kGT);
    const uint64_t tiles = uint64_t(a.row_tiles) * a.col_tiles;
    const uint32_t grid = uint32_t(tiles < kMaxGrid ? tiles : kMaxGrid);
    if (xq)
        launch_general<false, true, DCR_FP4_MX>(a, f32, grid, st);
    else if (grad)
        mx ? launch_general<true, false, DCR_FP4_MX>(a, f32, grid, st)
           : launch_general<true, false, DCR_FP4_NV>(a, f32, grid, st);
    else
        mx ? launch_general<false, false, DCR_FP4_MX>(a, f32, grid, st)
           : launch_general<false, false, DCR_FP4_NV>(a, f32, grid, st);
    return fp4_launched();
}

}  // namespace

uint32_t fp4_mm_plan(MArgs* a, uint32_t outs, uint32_t steps, const uint32_t (&cost)[4]) {
    // Time of a candidate: rounds of workgroups over 256 compute units, each
    // its steps and a fixed start and end; for parts of the sum the launch
    // that joins them and its traffic.  A step's cost (see each kernel's) is
    // what 4096 x 4096 results take more for a sum of 4096 than for one of
    // 1024, a round and step, with the tile forced, in units of 0.4 to 0.5 ns
    // (proportions decide).  Start and end are what is left, 10 us a round in
    // tiles of 256 rows, 3 of 128 and 1 of 64: kBlock, between them, is for all.
    // kJoin is the launch that joins, kJoinBytes what it moves a unit.  Over 100
    // products and gradients drawn at random (17 to 8192 rows) the choice takes
    // 1.7 % more than the best tile and number of parts, 52 % at worst (2551 x
    // 2432 x 384 in 4 bits: 13.1 us as chosen, 8.6 in tiles of 64 rows).
    // Groups make the start longer (offsets, weights that no neighbour has
    // read), which shows where a workgroup is alone on its compute unit: over
    // 100 of 8 to 256 experts the choice takes 2.7 % more than the best, without
    // that 4.5 % (16384 rows of 128 experts through 2048 x 768: 123 us in tiles
    // of 256 rows, 103 of 128).
    constexpr uint64_t kBlock = 6000, kGroupBlock = 12000, kJoin = 5000, kJoinBytes = 2500;
    const uint64_t stride = (uint64_t(outs) + 3) & ~uint64_t(3), pairs = (uint64_t(steps) + 1) / 2;
    uint64_t best = UINT64_MAX;
    uint32_t bm = 0;
    for (uint32_t i = 0; i < 4; ++i) {
        if (!cost[i]) continue;
        const uint32_t b = 256u >> i, bn = b == 256 ? 256 : 128;
        const uint64_t cols = (uint64_t(outs) + bn - 1) / bn, bound = row_tile_bound(*a, b);
        // Row tiles to expect of groups whose sizes the host does not know: as
        // of sizes spread exponentially.  (Half a tile a group more than the
        // rows fill, as once here, takes 256 rows a tile where most groups have
        // 64: 8192 rows of 128 experts through 2048 x 768 took 121 us, now 67.)
        const uint64_t rows = a->offsets ? std::min(bound, uint64_t(std::llround(a->groups / -std::expm1(-double(b) * a->groups / double(a->m)))))
                                         : bound;
        for (uint32_t s = 1; s <= 16; ++s) {
            if (s > 1 && (pairs / s < 2 || s * a->m * stride * 4 > DCR_FP4_WORKSPACE_BYTES)) break;
            if (bound * cols * s >= (1u << 22)) break;
            const uint64_t each = 2 * ((pairs + s - 1) / s);
            const uint64_t rounds = (rows * cols * s + 255) / 256;
            const uint64_t t = rounds * (each * cost[i] + (a->offsets && b == 256 ? kGroupBlock : kBlock)) + (s > 1 ? kJoin + s * a->m * stride * 8 / kJoinBytes : 0);
            if (t >= best) continue;
            best = t;
            bm = b;
            a->row_tiles = uint32_t(bound);
            a->col_tiles = uint32_t(cols);
            a->splits = s;
            a->split_steps = uint32_t(each);
        }
    }
    if (!bm) return 0;
    // Without groups an eighth of the tiles a die.  A grid for groups has spare
    // row tiles at its end: dies take strips of four row tiles in turn, which
    // spreads them.
    const uint32_t all = a->row_tiles * a->col_tiles * a->splits;
    a->chunk = a->offsets && a->row_tiles >= 64 ? 4 * a->col_tiles * a->splits : a->offsets ? a->splits : (all + 7) / 8;
    a->grid = (all + 8 * a->chunk - 1) / (8 * a->chunk) * 8 * a->chunk;
    a->split_elems = a->splits > 1 ? a->m * stride : 0;
    return bm;
}

MArgs fp4_mm_parts(const MArgs& a, uint32_t outs, void* ws) {
    MArgs p = a;
    if (a.splits > 1) {
        p.y = ws;
        p.y_stride = (uint64_t(outs) + 3) & ~uint64_t(3);
        p.y_vec = 1;
    }
    return p;
}

void fp4_mm_join(const MArgs& a, uint32_t outs, uint32_t fmt, bool f32, const void* ws, hipStream_t st) {
    if (a.splits <= 1) return;
    const uint32_t stride = (outs + 3) & ~3u, grid = uint32_t((a.m * (stride / 4) + 255) / 256);
    const float* part = static_cast<const float*>(ws);
    const bool mx = fmt == DCR_FP4_MX;
    if (f32 && mx)
        hipLaunchKernelGGL((fp4_mm_join_kernel<DCR_FP4_MX, float>), dim3(grid), dim3(256), 0, st, a, part, outs, stride);
    else if (f32)
        hipLaunchKernelGGL((fp4_mm_join_kernel<DCR_FP4_NV, float>), dim3(grid), dim3(256), 0, st, a, part, outs, stride);
    else if (mx)
        hipLaunchKernelGGL((fp4_mm_join_kernel<DCR_FP4_MX, uint16_t>), dim3(grid), dim3(256), 0, st, a, part, outs, stride);
    else
        hipLaunchKernelGGL((fp4_mm_join_kernel<DCR_FP4_NV, uint16_t>), dim3(grid), dim3(256), 0, st, a, part, outs, stride);
}

}  // namespace dcr

extern "C" {

int32_t dcr_fp4_matmul(const void* x, uint64_t m, uint64_t x_stride, const dcr_fp4_tensor* w, const int32_t* offsets,
                       uint32_t n_groups, void* y, uint32_t y_type, uint64_t y_stride, void* workspace_dev,
                       uint64_t ws_bytes, void* stream) try {
    dcr::set_error("");
    return dcr::product(false, nullptr, x, m, x_stride, w, offsets, n_groups, y, y_type, y_stride, workspace_dev,
                        ws_bytes, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_fp4_matmul_q(const dcr_fp4_tensor* x, const dcr_fp4_tensor* w, const int32_t* offsets, uint32_t n_groups,
                         void* y, uint32_t y_type, uint64_t y_stride, void* workspace_dev, uint64_t ws_bytes,
                         void* stream) try {
    dcr::set_error("");
    if (!x) return dcr::fp4_fail(DCR_E_INVAL, "x: NULL description");
    return dcr::product(false, x, nullptr, 0, 0, w, offsets, n_groups, y, y_type, y_stride, workspace_dev, ws_bytes,
                        static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_fp4_matmul_grad(const void* dy, uint64_t m, uint64_t dy_stride, const dcr_fp4_tensor* w,
                            const int32_t* offsets, uint32_t n_groups, void* dx, uint32_t dx_type,
                            uint64_t dx_stride, void* workspace_dev, uint64_t ws_bytes, void* stream) try {
    dcr::set_error("");
    return dcr::product(true, nullptr, dy, m, dy_stride, w, offsets, n_groups, dx, dx_type, dx_stride, workspace_dev,
                        ws_bytes, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

}  // extern "C"
