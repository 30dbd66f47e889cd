// dcr_fp4_rows.hip -- products of up to 16 rows with 4-bit weights (gfx950):
// single tokens, small decode batches, experts with a handful of rows each.
//
// Bound by reading the weights once.  A workgroup takes 16 NT rows of w and up
// to 16 rows of x; its eight waves share the sum, each taking runs of 256
// elements (one 128-byte line of every row of w), so that even one token
// through a 4096 x 4096 weight has 2048 waves with all their loads in flight.
// Nothing is shared before the end: codes go from memory to registers, a run
// ahead of their use, and become matrix operands there; the waves' sums meet in
// LDS.  One row takes 4.7 us through 4096 x 4096 and 10.8 us through
// 14336 x 4096 (31 MB, 2.9 TB/s), 16 rows 7.3 and 12.8 us; without the run
// ahead, and with scales read for half a run, 5.0, 12.8, 7.8 and 14.0 us.
#include <algorithm>

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

// SV: a run's scales of a row lie in one aligned piece of 8 or 16 bytes, and
// the sum ends with a run.
template <bool XQ, uint32_t WF, typename OUT, uint32_t NT, bool SV>
__global__ void __launch_bounds__(kWaves * 64, NT == 4 ? 2 : 4) fp4_mm_rows_kernel(MArgs a) {
    constexpr uint32_t BM = 16, BN = 16 * NT, kB = fp4_block(WF);
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
    const auto sr = rsrc(a.ws + wrow * a.ws_stride, (cols - 1) * sstep + a.k / kB);

    // Lane offsets; rows past the end are zeros.  A lane of w reads 32 elements
    // of a half run's 128 and, for bf16 x, passes three quarters on to the
    // other quads: a matrix operand then holds 32 elements of the sum, eight
    // a quad, and x is read in 64-byte pieces of its rows (read 16 bytes here
    // and there to fit the codes instead, x costs three times the weights).
    // A load takes as long for one byte of each row as for 16, so a quad reads
    // one block of 32 elements' scales, or all read the run's.
    const uint32_t xout = r16 < rows ? 0u : kOutside;
    const uint32_t xo = (__umul24(r16, xstep) + quad * 16) | xout;
    const uint32_t xso = XQ ? (__umul24(r16, uint32_t(a.xs_stride)) + (SV ? 0 : quad)) | xout : 0;
    uint32_t wo[NT], so[NT];
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i) {
        const uint32_t r = i * 16 + r16, out = r < cols ? 0u : kOutside;
        wo[i] = (__umul24(r, wstep) + quad * 16) | out;
        so[i] = (__umul24(r, sstep) + (SV ? 0 : quad * (32 / kB))) | out;
    }

    // A run's weights: codes, and scales as they were read.
    struct Run {
        u32x4 codes[2][NT];
        u32x4 scales[NT];
    };
    auto load_w = [&](uint32_t run) {
        Run w;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            // elements past the sum's end (a multiple of 32) are zeros
            const uint32_t k0 = run * 256 + h * 128, out = k0 + quad * 32 < a.k ? 0u : kOutside;
#pragma unroll
            for (uint32_t i = 0; i < NT; ++i) {
                w.codes[h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[i] | out, k0 / 2, 0));
                if constexpr (!SV) {
                    w.scales[i][h] = __builtin_amdgcn_raw_buffer_load_b8(sr, so[i] | out, k0 / kB, 0);
                    if constexpr (kB == 16)
                        w.scales[i][2 + h] = __builtin_amdgcn_raw_buffer_load_b8(sr, (so[i] + 1) | out, k0 / kB, 0);
                }
            }
        }
        if constexpr (SV) {
            const uint32_t out = run * 256 < a.k ? 0u : kOutside;
#pragma unroll
            for (uint32_t i = 0; i < NT; ++i) {
                if constexpr (kB == 32) {
                    const auto v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, so[i] | out, run * 8, 0));
                    w.scales[i][0] = v[0];
                    w.scales[i][1] = v[1];
                } else {
                    w.scales[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(sr, so[i] | out, run * 16, 0));
                }
            }
        }
        return w;
    };

    f32x4 acc[NT] = {};
    const uint32_t runs = (a.k + 255) / 256;
    Run w = load_w(wave);
    for (uint32_t run = wave; run < runs; run += kWaves) {
        u32x4 x[2][XB];
        uint32_t xs[2];
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            const uint32_t k0 = run * 256 + h * 128;
            if constexpr (XQ) {
                const uint32_t out = k0 + quad * 32 < a.k ? 0u : kOutside;
                x[h][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, xo | out, k0 / 2, 0));
                if constexpr (!SV) xs[h] = __builtin_amdgcn_raw_buffer_load_b8(xsr, xso | out, k0 / 32, 0);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < XB; ++j)
                    x[h][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                            xr, (xo + j * 64) | (k0 + j * 32 < a.k ? 0u : kOutside), k0 * 2, 0));
            }
        }
        if constexpr (XQ && SV) {
            const auto v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(xsr, xso, run * 8, 0));
            xs[0] = v[0];
            xs[1] = v[1];
        }
        // the next run's weights are on their way before this one's are used
        const Run next = load_w(run + kWaves);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
#pragma unroll
            for (uint32_t i = 0; i < NT; ++i) {
                if constexpr (XQ) {
                    acc[i] = mfma_fp4<0, 0>(w.codes[h][i], x[h][0], acc[i], w.scales[i][h] >> (SV ? 8 * quad : 0),
                                           xs[h] >> (SV ? 8 * quad : 0));
                } else {
                    const uint32_t own = w.scales[i][h] | (SV || kB == 32 ? 0 : w.scales[i][2 + h] << 8);
                    u32x4 sc = {own, own, own, own};
                    if constexpr (!SV) transpose_quads(sc);     // quad j's in word j
                    transpose_quads(w.codes[h][i]);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint32_t byte = !SV ? sc[j] >> (kB == 32 ? 0 : 8 * (quad >> 1))
                                              : kB == 32 ? sc[j] >> (8 * j)
                                                         : w.scales[i][2 * h + j / 2] >> (16 * (j & 1) + 8 * (quad >> 1));
                        const bf16x8 v = fp4_unpack8_bf16<WF>(w.codes[h][i][j], byte & 255u);
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, x[h][j]), acc[i], 0, 0, 0);
                    }
                }
            }
        }
        w = next;
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
    if (sv)
        hipLaunchKernelGGL((fp4_mm_rows_kernel<XQ, WF, OUT, NT, true>), g, t, 0, st, a);
    else
        hipLaunchKernelGGL((fp4_mm_rows_kernel<XQ, WF, OUT, NT, false>), g, t, 0, st, a);
}
template <bool XQ, uint32_t WF, typename OUT>
void launch(const MArgs& a, hipStream_t st, bool sv, uint32_t nt) {
    nt == 4   ? launch<XQ, WF, OUT, 4>(a, st, sv)
    : nt == 2 ? launch<XQ, WF, OUT, 2>(a, st, sv)
              : launch<XQ, WF, OUT, 1>(a, st, sv);
}

}  // namespace

bool fp4_mm_rows(MArgs a, bool xq, uint32_t fmt, bool f32, hipStream_t st) {
    if (!a.x_vec || !a.w_vec || a.k % 32 || a.k >= kLongest || a.x_stride >= (1u << 22) || a.wc_stride >= (1u << 22) ||
        a.xs_stride >= (1u << 22) || a.ws_stride >= (1u << 22))
        return false;
    // rows of a group, as far as the host can tell
    if ((a.m + a.groups - 1) / a.groups > 16) return false;
    // Four or two subtiles of w a workgroup read x once for all, where that
    // leaves most compute units one: 16 rows through 14336 x 4096 take 22.6,
    // 16.6 and 12.8 us with one, two and four, through 4096 x 4096 7.3, 9.5 and
    // 12.1 us.
    const uint64_t rt = row_tile_bound(a, 16);
    const uint32_t nt = rt * (a.n / 64) >= 192 ? 4 : rt * (a.n / 32) >= 192 ? 2 : 1;
    const uint64_t ct = (uint64_t(a.n) + 16 * nt - 1) / (16 * nt);
    // The larger tiles stream better once there is more than one workgroup of
    // four subtiles a compute unit (16 rows through 28672 x 4096: 23.3 us here
    // and 19.0 there, through 14336 x 4096 12.8 and 14.2), and so they do when
    // workgroups read x more often than the weights (16 rows through
    // 4096 x 14336, 117 MB of x: 19.1 and 15.1; eight rows: 14.5 and 14.9).
    if (rt * ((a.n + 63) / 64) > 256) return false;
    if (rt * ct * std::min<uint64_t>(a.m, 16) * a.k * (xq ? 1 : 4) / 2 > (56u << 20)) return false;
    a.row_tiles = uint32_t(rt);
    a.col_tiles = uint32_t(ct);
    const uint32_t piece = 256 / fp4_block(fmt);
    const bool sv = a.k % 256 == 0 && a.ws_stride % piece == 0 && (!xq || (a.xs_stride % 8 == 0));
    if (xq)
        f32 ? launch<true, DCR_FP4_MX, float>(a, st, sv, nt) : launch<true, DCR_FP4_MX, uint16_t>(a, st, sv, nt);
    else if (fmt == DCR_FP4_MX)
        f32 ? launch<false, DCR_FP4_MX, float>(a, st, sv, nt) : launch<false, DCR_FP4_MX, uint16_t>(a, st, sv, nt);
    else
        f32 ? launch<false, DCR_FP4_NV, float>(a, st, sv, nt) : launch<false, DCR_FP4_NV, uint16_t>(a, st, sv, nt);
    return true;
}

}  // namespace dcr
