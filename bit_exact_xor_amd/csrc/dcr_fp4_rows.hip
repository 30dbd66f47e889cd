// dcr_fp4_rows.hip -- products of up to 16 rows with 4-bit weights (gfx950):
// single tokens, small decode batches, experts with a handful of rows each.
//
// Bound by reading the weights once.  A workgroup takes 16 NT rows of w and up
// to 16 rows of x; its eight waves share the sum, each taking runs of 256
// elements (one 128-byte line of every row of w), so that even one token
// through a 4096 x 4096 weight has 2048 waves with all their loads in flight.
// Nothing is shared before the end: codes go from memory to registers and
// become matrix operands there; the waves' sums meet in LDS.
#include "dcr_fp4_mm.h"

namespace dcr {
namespace {

constexpr uint32_t kWaves = 8;

// Quads exchange 4 x 4 words: r[j] of quad q becomes r[q] of quad j.
__device__ __forceinline__ void transpose_quads(u32x4& r) {
    auto a = __builtin_amdgcn_permlane32_swap(r[0], r[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(r[1], r[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    r = u32x4{c[0], c[1], d[0], d[1]};
}

// SV: rows of scales start on borders of a half run's scales (4 or 8 bytes)
template <bool XQ, uint32_t WF, typename OUT, uint32_t NT, bool SV>
__global__ void __launch_bounds__(kWaves * 64, 4) fp4_mm_rows_kernel(MArgs a) {
    constexpr uint32_t BM = 16, BN = 16 * NT, SB = 128 / fp4_block(WF);   // scales of a half run
    __shared__ __attribute__((aligned(16))) float sums[kWaves][NT][64][4];
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

    // Lane offsets; rows past the end are zeros.  A lane of w reads 32 elements
    // of a half run's 128 and, for bf16 x, passes three quarters on to the
    // other quads: a matrix operand then holds 32 elements of the sum, eight
    // a quad, and x is read in 64-byte pieces of its rows (read 16 bytes here
    // and there to fit the codes instead, x costs three times the weights).
    const uint32_t xout = r16 < rows ? 0u : kOutside;
    const uint32_t xo = (__umul24(r16, xstep) + quad * 16) | xout;
    const uint32_t xso = XQ ? (__umul24(r16, uint32_t(a.xs_stride)) + quad) | xout : 0;
    uint32_t wo[NT], so[NT];
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i) {
        const uint32_t r = i * 16 + r16, out = r < cols ? 0u : kOutside;
        wo[i] = (__umul24(r, wstep) + quad * 16) | out;
        so[i] = (__umul24(r, sstep) + (XQ ? quad : 0)) | out;
    }

    f32x4 acc[NT] = {};
    const uint32_t runs = (a.k + 255) / 256;
    for (uint32_t run = wave; run < runs; run += kWaves) {
        u32x4 wq[2][NT], xv[2][XB];
        u32x2 sc[2][NT];
        uint32_t xs[2];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            // elements past the sum's end (a multiple of 32) are zeros
            const uint32_t k0 = run * 256 + h * 128, out = k0 + quad * 32 < a.k ? 0u : kOutside;
#pragma unroll
            for (uint32_t i = 0; i < NT; ++i) {
                wq[h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[i] | out, k0 / 2, 0));
                const uint32_t at = k0 / fp4_block(WF), all = k0 < a.k ? 0u : kOutside;
                if constexpr (XQ) {
                    sc[h][i][0] = __builtin_amdgcn_raw_buffer_load_b8(sr, so[i] | out, at, 0);
                } else if constexpr (SV && SB == 4) {
                    sc[h][i][0] = __builtin_amdgcn_raw_buffer_load_b32(sr, so[i] | all, at, 0);
                } else if constexpr (SV) {
                    sc[h][i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, so[i] | all, at, 0));
                } else {
                    sc[h][i] = u32x2{0, 0};
#pragma unroll
                    for (uint32_t b = 0; b < SB; ++b)
                        sc[h][i][b / 4] |= uint32_t(__builtin_amdgcn_raw_buffer_load_b8(
                                               sr, (so[i] + b) | ((at + b) * fp4_block(WF) < a.k ? 0u : kOutside), at, 0))
                                           << (8 * (b & 3));
                }
            }
            if constexpr (XQ) {
                xv[h][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, xo | out, k0 / 2, 0));
                xs[h] = __builtin_amdgcn_raw_buffer_load_b8(xsr, xso | out, k0 / 32, 0);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < XB; ++j)
                    xv[h][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                             xr, (xo + j * 64) | (k0 + j * 32 < a.k ? 0u : kOutside), k0 * 2, 0));
            }
        }
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
#pragma unroll
            for (uint32_t i = 0; i < NT; ++i) {
                if constexpr (XQ) {
                    acc[i] = mfma_fp4<0, 0>(wq[h][i], xv[h][0], acc[i], sc[h][i][0], xs[h]);
                } else {
                    transpose_quads(wq[h][i]);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint32_t byte = WF == DCR_FP4_MX ? sc[h][i][0] >> (8 * j)
                                                               : sc[h][i][j / 2] >> (16 * (j & 1) + 8 * (quad >> 1));
                        const bf16x8 w = fp4_unpack8_bf16<WF>(wq[h][i][j], byte & 255u);
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, xv[h][j]), acc[i], 0, 0, 0);
                    }
                }
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(sums[wave][i][lane]) = acc[i];
    __syncthreads();
    const float s = WF == DCR_FP4_NV ? *a.tensor_scale : 1.0f;
    // wave t joins subtile t: the waves' sums in order
    if (const uint32_t t = wave; t < NT) {
        f32x4 v = {};
#pragma unroll
        for (uint32_t w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(sums[w][t][lane]);
        v *= s;
        const uint32_t c = n0 + t * 16 + quad * 4;
        if (r16 >= rows) return;
        OUT* out = static_cast<OUT*>(a.y) + (rt.begin + r16) * a.y_stride;
        if (a.y_vec && c + 4 <= a.n) {
            store4(out + c, v);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (c + e < a.n) store_out(out + c + e, v[e]);
        }
    }
}

template <bool XQ, uint32_t WF, typename OUT, uint32_t NT>
void launch(const MArgs& a, hipStream_t st, bool sv) {
    const dim3 g(a.row_tiles * a.col_tiles), t(kWaves * 64);
    if constexpr (!XQ)
        if (sv) {
            hipLaunchKernelGGL((fp4_mm_rows_kernel<XQ, WF, OUT, NT, true>), g, t, 0, st, a);
            return;
        }
    hipLaunchKernelGGL((fp4_mm_rows_kernel<XQ, WF, OUT, NT, false>), g, t, 0, st, a);
}
template <bool XQ, uint32_t WF, typename OUT>
void launch(const MArgs& a, hipStream_t st, bool sv, uint32_t nt) {
    nt == 2 ? launch<XQ, WF, OUT, 2>(a, st, sv) : launch<XQ, WF, OUT, 1>(a, st, sv);
}

}  // namespace

bool fp4_mm_rows(MArgs a, bool xq, uint32_t fmt, bool f32, hipStream_t st) {
    if (!a.x_vec || !a.w_vec || a.k % 32 || a.x_stride >= (1u << 22) || a.wc_stride >= (1u << 22) ||
        a.xs_stride >= (1u << 22) || a.ws_stride >= (1u << 22))
        return false;
    // rows of a group, as far as the host can tell
    if ((a.m + a.groups - 1) / a.groups > 16) return false;
    // two subtiles of w a workgroup read x once for both, where that leaves
    // two workgroups a compute unit
    const uint64_t rt = (a.m + 15) / 16 + (a.offsets ? a.groups : 0);
    const uint32_t nt = rt * (a.n / 32) >= 512 ? 2 : 1;
    const uint64_t ct = (uint64_t(a.n) + 16 * nt - 1) / (16 * nt);
    if (rt * ct >= (1u << 22)) return false;
    a.row_tiles = uint32_t(rt);
    a.col_tiles = uint32_t(ct);
    const bool sv = a.k % 128 == 0 && a.ws_stride % (128 / fp4_block(fmt)) == 0;
    if (xq)
        f32 ? launch<true, DCR_FP4_MX, float>(a, st, sv, nt) : launch<true, DCR_FP4_MX, uint16_t>(a, st, sv, nt);
    else if (fmt == DCR_FP4_MX)
        f32 ? launch<false, DCR_FP4_MX, float>(a, st, sv, nt) : launch<false, DCR_FP4_MX, uint16_t>(a, st, sv, nt);
    else
        f32 ? launch<false, DCR_FP4_NV, float>(a, st, sv, nt) : launch<false, DCR_FP4_NV, uint16_t>(a, st, sv, nt);
    return true;
}

}  // namespace dcr
