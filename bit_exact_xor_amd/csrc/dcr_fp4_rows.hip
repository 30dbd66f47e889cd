// dcr_fp4_rows.hip -- products of few rows with 4-bit weights (gfx950): single
// tokens, decode batches, experts with a handful of rows each.
//
// Bound by reading the weights once.  A workgroup takes 16 NT rows of w and up
// to 16 MT rows of x; its eight waves share the sum, each taking runs of 256
// elements (one 128-byte line of every row of w), so that even one token
// through a 4096 x 4096 weight has 2048 waves with all their loads in flight.
// Nothing is shared before the end: codes go from memory to registers and
// become matrix operands there; the waves' sums meet in LDS.
#include "dcr_fp4_mm.h"

namespace dcr {
namespace {

constexpr uint32_t kWaves = 8;

template <bool XQ, uint32_t WF, typename OUT, uint32_t MT, uint32_t NT>
__global__ void __launch_bounds__(kWaves * 64, 4) fp4_mm_rows_kernel(MArgs a) {
    constexpr uint32_t BM = 16 * MT, BN = 16 * NT;
    __shared__ __attribute__((aligned(16))) float sums[kWaves][MT * NT][64][4];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r16 = lane & 15u, quad = lane >> 4;
    const uint32_t ct = blockIdx.x / a.row_tiles, rt_i = blockIdx.x - ct * a.row_tiles;
    const RowTile rt = row_tile<BM>(a, rt_i);
    if (rt.begin == rt.end) return;
    const uint32_t rows = uint32_t(rt.end - rt.begin), n0 = ct * BN, cols = min(BN, a.n - n0);

    constexpr uint32_t XB = XQ ? 1 : 4;         // bytes of two elements of x
    const uint32_t xstep = uint32_t(a.x_stride) * (XQ ? 1 : 2), wstep = uint32_t(a.wc_stride), sstep = uint32_t(a.ws_stride);
    const auto xr = rsrc(static_cast<const uint8_t*>(a.x) + rt.begin * xstep, (rows - 1) * xstep + a.k / 2 * XB);
    const auto xsr = rsrc(XQ ? a.xs + rt.begin * a.xs_stride : nullptr, XQ ? (rows - 1) * uint32_t(a.xs_stride) + a.k / 32 : 0);
    const uint64_t wrow = uint64_t(rt.group) * a.n + n0;
    const auto wr = rsrc(a.wc + wrow * a.wc_stride, (cols - 1) * wstep + a.k / 2);
    const auto sr = rsrc(a.ws + wrow * a.ws_stride, (cols - 1) * sstep + a.k / fp4_block(WF));

    // lane offsets; rows past the end are zeros
    uint32_t xo[MT], xso[MT], wo[NT], so[NT];
#pragma unroll
    for (uint32_t m = 0; m < MT; ++m) {
        const uint32_t r = m * 16 + r16, out = r < rows ? 0u : kOutside;
        xo[m] = (__umul24(r, xstep) + quad * 16 * XB) | out;
        xso[m] = XQ ? (__umul24(r, uint32_t(a.xs_stride)) + quad) | out : 0;
    }
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i) {
        const uint32_t r = i * 16 + r16, out = r < cols ? 0u : kOutside;
        wo[i] = (__umul24(r, wstep) + quad * 16) | out;
        so[i] = (__umul24(r, sstep) + quad * (32 / fp4_block(WF))) | out;
    }

    f32x4 acc[NT][MT] = {};
    const uint32_t runs = (a.k + 255) / 256;
    for (uint32_t run = wave; run < runs; run += kWaves) {
        u32x4 wq[2][NT], xv[2][MT][XB];
        uint32_t sc[2][NT], xs[2][MT];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            // this lane's 32 elements of the half run; past the sum's end (a
            // multiple of 32) zeros
            const uint32_t k0 = run * 256 + h * 128, out = k0 + quad * 32 < a.k ? 0u : kOutside;
#pragma unroll
            for (uint32_t i = 0; i < NT; ++i) {
                wq[h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[i] | out, k0 / 2, 0));
                if (WF == DCR_FP4_MX)
                    sc[h][i] = __builtin_amdgcn_raw_buffer_load_b8(sr, so[i] | out, k0 / 32, 0);
                else
                    sc[h][i] = __builtin_amdgcn_raw_buffer_load_b16(sr, so[i] | out, k0 / 16, 0);
            }
#pragma unroll
            for (uint32_t m = 0; m < MT; ++m) {
#pragma unroll
                for (uint32_t j = 0; j < XB; ++j)
                    xv[h][m][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, (xo[m] + j * 16) | out, k0 / 2 * XB, 0));
                if (XQ) xs[h][m] = __builtin_amdgcn_raw_buffer_load_b8(xsr, xso[m] | out, k0 / 32, 0);
            }
        }
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            if constexpr (XQ) {
#pragma unroll
                for (uint32_t i = 0; i < NT; ++i)
#pragma unroll
                    for (uint32_t m = 0; m < MT; ++m)
                        acc[i][m] = mfma_fp4<0, 0>(wq[h][i], xv[h][m][0], acc[i][m], sc[h][i], xs[h][m]);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                    for (uint32_t i = 0; i < NT; ++i) {
                        const bf16x8 w = fp4_unpack8_bf16<WF>(wq[h][i][j], WF == DCR_FP4_MX ? sc[h][i] : (sc[h][i] >> (j / 2 * 8)) & 255u);
#pragma unroll
                        for (uint32_t m = 0; m < MT; ++m)
                            acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, xv[h][m][j]), acc[i][m], 0, 0, 0);
                    }
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i)
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m) *reinterpret_cast<f32x4*>(sums[wave][i * MT + m][lane]) = acc[i][m];
    __syncthreads();
    const float s = WF == DCR_FP4_NV ? *a.tensor_scale : 1.0f;
    // wave v joins subtiles v, v + 8, ...: waves' sums in order
    for (uint32_t t = wave; t < MT * NT; t += kWaves) {
        f32x4 v = {};
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(sums[w][t][lane]);
        v *= s;
        const uint32_t r = t % MT * 16 + r16, c = n0 + t / MT * 16 + quad * 4;
        if (r >= rows) continue;
        OUT* out = static_cast<OUT*>(a.y) + (rt.begin + r) * a.y_stride;
        if (a.y_vec && c + 4 <= a.n) {
            store4(out + c, v);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (c + e < a.n) store_out(out + c + e, v[e]);
        }
    }
}

template <bool XQ, uint32_t WF, typename OUT>
void launch(const MArgs& a, hipStream_t st, uint32_t grid) {
    const dim3 g(grid), t(kWaves * 64);
    hipLaunchKernelGGL((fp4_mm_rows_kernel<XQ, WF, OUT, 1, 1>), g, t, 0, st, a);
}

}  // namespace

bool fp4_mm_rows(MArgs a, bool xq, uint32_t fmt, bool f32, hipStream_t st) {
    if (!a.x_vec || !a.w_vec || a.k % 32 || a.x_stride >= (1u << 22) || a.wc_stride >= (1u << 22) ||
        a.xs_stride >= (1u << 22) || a.ws_stride >= (1u << 22))
        return false;
    // rows of a group, as far as the host can tell
    if ((a.m + a.groups - 1) / a.groups > 16) return false;
    const uint64_t rt = (a.m + 15) / 16 + (a.offsets ? a.groups : 0), ct = (uint64_t(a.n) + 15) / 16;
    if (rt * ct >= (1u << 22)) return false;
    a.row_tiles = uint32_t(rt);
    a.col_tiles = uint32_t(ct);
    const uint32_t grid = uint32_t(rt * ct);
    if (xq)
        f32 ? launch<true, DCR_FP4_MX, float>(a, st, grid) : launch<true, DCR_FP4_MX, uint16_t>(a, st, grid);
    else if (fmt == DCR_FP4_MX)
        f32 ? launch<false, DCR_FP4_MX, float>(a, st, grid) : launch<false, DCR_FP4_MX, uint16_t>(a, st, grid);
    else
        f32 ? launch<false, DCR_FP4_NV, float>(a, st, grid) : launch<false, DCR_FP4_NV, uint16_t>(a, st, grid);
    return true;
}

}  // namespace dcr
