// dcr_fp4_tile.hip -- bf16 rows times 4-bit weights in large tiles (gfx950).
//
// Bound by the matrix unit, with the conversion of the codes next to it: an
// MX code pair is one instruction, an NV one four.  So a wave takes all the
// tile's rows of x and columns of its own: every code is converted once a
// tile, in the wave that multiplies with it, and never sees LDS.  x goes
// there by direct loads and is read by every wave (a quarter of what LDS
// gives).  Against 2 x 4 waves of 128 x 64, which convert twice, 8 waves of
// 256 x 32 take 8192 x 14336 x 4096 from 670 to 658 us (MX, 1460 TFLOP/s; the
// library's bf16 product of the same sizes takes 734 us) and from 778 to
// 712 us (NV).  The matrix unit is busy in 73 % of the cycles, at the 1.7 GHz
// that the card holds under this load.
#include "dcr_fp4_mm.h"

namespace dcr {
namespace {

constexpr uint32_t kBK = 128;          // elements of the sum a step takes
constexpr uint32_t kRowB = kBK * 2;    // bytes of a row of x in LDS

// x in LDS: a row is 16 pieces of 16 bytes, piece c of row r at place
// c ^ swizzle(r).  A 128-bit read serves 16 lanes at a time, half of them of
// the next quad (rows 0-3 and 12-15 with rows 4-11 of the quad beside), whose
// pieces differ in bit 2: those halves go to different halves of the row.
__device__ __forceinline__ uint32_t swizzle(uint32_t r) {
    return (r & 3u) | ((r >> 1) & 4u) | (((r >> 3) ^ (r >> 2)) & 1u) << 3;
}

// What is known of the rows: nothing; codes on 16-byte borders (what a row's
// last 16 bytes hold behind the sum's end is loaded too, and multiplied by
// zeros, see end_inside); x there too, and a sum of
// whole pieces of x; and scales of two steps at a time on borders of their
// own (then one load for 16 rows brings two steps' scales: a load costs as
// much for a byte of each row as for the 16 bytes of codes).
enum class Rows { kAny, kCodes, kAligned, kPaired };

template <uint32_t WF, typename OUT, uint32_t BM, uint32_t BN, uint32_t W, Rows ROWS>
__global__ void __launch_bounds__(W * 64, 2) fp4_mm_tile_kernel(MArgs a) {
    constexpr bool CODES = ROWS != Rows::kAny, ALIGNED = CODES && ROWS != Rows::kCodes, PAIRED = ROWS == Rows::kPaired;
    constexpr uint32_t MI = BM / 16, NI = BN / W / 16, DMA = BM / 4 / W;
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[BM * kRowB], buf1[BM * kRowB];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r16 = lane & 15u, quad = lane >> 4;

    const TilePlace at = tile_place(a);
    if (at.row >= a.row_tiles) return;
    const RowTile rt = row_tile<BM>(a, at.row);
    if (rt.begin == rt.end) return;
    const uint32_t rows = uint32_t(rt.end - rt.begin), n0 = at.col * BN;

    const uint8_t* xb = static_cast<const uint8_t*>(a.x) + rt.begin * a.x_stride * 2;
    const uint32_t xstep = uint32_t(a.x_stride) * 2;
    uint32_t xo[DMA];
#pragma unroll
    for (uint32_t i = 0; i < DMA; ++i) {
        const uint32_t r = (i * W + wave) * 4 + quad;
        xo[i] = min(r, rows - 1) * xstep + (r16 ^ swizzle(r)) * 16;
    }
    // w: lane (r16, quad) holds row r16 of a subtile, elements [32 quad, +32)
    // of a step: one MX block
    const uint8_t* wb = a.wc + (uint64_t(rt.group) * a.n + n0) * a.wc_stride;
    const uint8_t* sb = a.ws + (uint64_t(rt.group) * a.n + n0) * a.ws_stride;
    uint32_t wo[NI], so[NI];
#pragma unroll
    for (uint32_t i = 0; i < NI; ++i) {
        const uint32_t r = min(wave * (BN / W) + i * 16 + r16, a.n - 1 - n0);
        wo[i] = r * uint32_t(a.wc_stride) + quad * 16;
        so[i] = r * uint32_t(a.ws_stride) + (PAIRED ? 0 : quad * (WF == DCR_FP4_MX ? 1 : 2));
    }

    // buffer descriptors: scalar base and step, 32-bit lane offsets
    const auto xr = rsrc(xb, ((rows - 1) * uint32_t(a.x_stride) + a.k) * 2);
    const uint32_t wrows = min(BN, a.n - n0);
    const auto wr = rsrc(wb, (wrows - 1) * uint32_t(a.wc_stride) + (((a.k + 1) / 2 + 15) & ~15u));
    const auto sr = rsrc(sb, (wrows - 1) * uint32_t(a.ws_stride) + (a.k + fp4_block(WF) - 1) / fp4_block(WF));

    f32x4 acc[NI][MI] = {};
    u32x4 wq[2][NI];
    uint32_t wsc[2][NI];
    typename std::conditional<WF == DCR_FP4_MX, u32x2, u32x4>::type pair[NI];   // scales of two steps of a row
    bf16x8 w[2][NI];

    // this workgroup's steps: from `first` on, up to `steps`
    const uint32_t first = at.split * a.split_steps, steps = min(first + a.split_steps, (a.k + kBK - 1) / kBK);

    // Loads of a step of aligned rows.  From the step on in which the sum ends
    // (at a multiple of 8), lanes past the end read behind the descriptors'
    // range, which gives zeros; a lane once past it stays there, so its offset
    // is changed for good and the other steps spend nothing on it.
    auto x_past_end = [&](uint32_t step) {
        if ((step + 1) * kBK <= a.k) return;
        const uint32_t out = step * kBK + (r16 ^ swizzle(wave * 4 + quad)) * 8 < a.k ? 0u : kOutside;
#pragma unroll
        for (uint32_t i = 0; i < DMA; ++i) xo[i] |= out;
    };
    auto w_past_end = [&](uint32_t step) {
        if ((step + 1) * kBK <= a.k) return;
        const uint32_t out = step * kBK + quad * 32 < a.k ? 0u : kOutside;
#pragma unroll
        for (uint32_t i = 0; i < NI; ++i) wo[i] |= out, so[i] |= out;
    };
    auto load_w = [&](uint32_t step, auto odd) {
        constexpr uint32_t o = decltype(odd)::value;
#pragma unroll
        for (uint32_t i = 0; i < NI; ++i) {
            wq[o][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[i], step * (kBK / 2), 0));
            if constexpr (PAIRED)
                continue;
            else if constexpr (WF == DCR_FP4_MX)
                wsc[o][i] = __builtin_amdgcn_raw_buffer_load_b8(sr, so[i], step * (kBK / 32), 0);
            else
                wsc[o][i] = __builtin_amdgcn_raw_buffer_load_b16(sr, so[i], step * (kBK / 16), 0);
        }
    };
    auto load_pair = [&](uint32_t step) {
#pragma unroll
        for (uint32_t i = 0; i < NI; ++i) {
            if constexpr (!PAIRED)
                continue;
            else if constexpr (WF == DCR_FP4_MX)
                pair[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, so[i], step * (kBK / 32), 0));
            else
                pair[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(sr, so[i], step * (kBK / 16), 0));
        }
    };
    // this lane's scales of step `odd` of the pair
    auto from_pair = [&](auto odd) {
        constexpr uint32_t o = decltype(odd)::value;
#pragma unroll
        for (uint32_t i = 0; i < NI; ++i) {
            if constexpr (!PAIRED)
                continue;
            else if constexpr (WF == DCR_FP4_MX)
                wsc[o][i] = (pair[i][o] >> (8 * quad)) & 255u;
            else
                wsc[o][i] = (quad & 2u ? pair[i][2 * o + 1] : pair[i][2 * o]) >> (16 * (quad & 1u));
        }
    };
    auto load_x = [&](uint8_t* buf, uint32_t step, auto subtiles) {
#pragma unroll
        for (uint32_t i = 0; i < DMA * decltype(subtiles)::value / MI; ++i)
            load_lds16(xr, buf + (i * W + wave) * 1024, xo[i], step * kRowB);
        __builtin_amdgcn_sched_barrier(0);   // (the step's wait counts the loads after these)
    };
    // Any alignment: into registers while the step before multiplies, then to
    // LDS.  A piece of x that the sum's end cuts is read as the row's last eight
    // elements and moved down.
    u32x4 xn[DMA], wn[NI];
    uint32_t sn[NI];
    auto fetch_x = [&](uint32_t step) {
        if ((step + 1) * kBK <= a.k) {
#pragma unroll
            for (uint32_t i = 0; i < DMA; ++i) __builtin_memcpy(&xn[i], xb + step * kRowB + xo[i], 16);
            return;
        }
        const uint32_t c = step * kBK + (r16 ^ swizzle(wave * 4 + quad)) * 8, past = c - min(c, a.k - 8);
#pragma unroll
        for (uint32_t i = 0; i < DMA; ++i) {
            xn[i] = last_elements(xb + uint64_t(xo[i]) + step * kRowB - past * 2, past);
        }
    };
    auto put_x = [&](uint8_t* buf) {
#pragma unroll
        for (uint32_t i = 0; i < DMA; ++i) *reinterpret_cast<u32x4*>(buf + (i * W + wave) * 1024 + lane * 16) = xn[i];
    };
    auto fetch_w = [&](uint32_t step) {
        const uint32_t kw = step * kBK + quad * 32;
#pragma unroll
        for (uint32_t i = 0; i < NI; ++i) {
            wn[i] = u32x4{0, 0, 0, 0};
            sn[i] = 0;
            if (kw < a.k) {
                wn[i] = codes32(wb + wo[i] - quad * 16, kw, a.k, a.w_vec);
                const uint8_t* s = sb + step * (kBK / fp4_block(WF)) + so[i];
                sn[i] = s[0];
                if (WF == DCR_FP4_NV && kw + 16 < a.k) sn[i] |= uint32_t(s[1]) << 8;
            }
        }
    };
    auto put_w = [&] {
#pragma unroll
        for (uint32_t i = 0; i < NI; ++i) wq[0][i] = wn[i], wsc[0][i] = sn[i];
    };
    auto convert = [&](auto odd, uint32_t j, uint32_t i) {
        constexpr uint32_t o = decltype(odd)::value;
        w[j & 1][i] = fp4_unpack8_bf16<WF>(wq[o][i][j], WF == DCR_FP4_MX ? wsc[o][i] : (wsc[o][i] >> (j / 2 * 8)) & 255u);
    };
    // A sum that ends inside a block: codes behind a row's end become zeros.  (x
    // is zero there, but the largest MX scales take a code past bf16's range.)
    const uint32_t end_step = a.k % 32 ? a.k / kBK : ~0u;
    auto end_inside = [&](uint32_t step, auto odd) {
        constexpr uint32_t o = decltype(odd)::value;
        if (__builtin_expect(step != end_step, 1)) return;
        const uint32_t live = a.k - min(step * kBK + quad * 32, a.k);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t mask = live >= 8 * j + 8 ? ~0u : live <= 8 * j ? 0u : (1u << (4 * (live - 8 * j))) - 1u;
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) wq[o][i][j] &= mask;
        }
    };
    // A step's products, four row subtiles at a time.  While these multiply,
    // the next four are read from LDS and part of the next quarter's codes is
    // converted.  The codes' registers are free once the last quarter is
    // converted, and take those of the step after the next then: they may come
    // from HBM.
    auto compute = [&](const uint8_t* buf, uint32_t next, auto odd, auto subtiles) {
        constexpr uint32_t M = decltype(subtiles)::value, H = M < 4 ? M : 4, P = M / H, C = (NI + P - 1) / P;   // C subtiles of codes a phase
        const uint8_t* xl = buf + r16 * kRowB;
        bf16x8 x[2][H];
        auto read = [&](uint32_t ph) {
#pragma unroll
            for (uint32_t m = 0; m < H; ++m)
                x[ph & 1][m] = *reinterpret_cast<const bf16x8*>(xl + ((ph % P) * H + m) * 16 * kRowB +
                                                                (((quad * 4 + ph / P) ^ swizzle(r16)) * 16));
        };
        from_pair(odd);
        if (decltype(odd)::value) load_pair(next);
        read(0);
        if constexpr (CODES && !PAIRED && WF == DCR_FP4_MX) end_inside(next - 1, odd);
#pragma unroll
        for (uint32_t ph = 0; ph < 4 * P; ++ph) {
            const uint32_t j = ph / P;
            if (ph + 1 < 4 * P) read(ph + 1);
            if (ph == 0)
#pragma unroll
                for (uint32_t i = 0; i < NI; ++i) convert(odd, 0, i);
            if (CODES && ph == 3 * P) {
                load_w(next + 1, odd);
            }
            if (j < 3)
#pragma unroll
                for (uint32_t i = ph % P * C; i < (ph % P + 1) * C && i < NI; ++i) convert(odd, j + 1, i);
#pragma unroll
            for (uint32_t m = 0; m < H; ++m)
#pragma unroll
                for (uint32_t i = 0; i < NI; ++i)
                    acc[i][(ph % P) * H + m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        w[j & 1][i], x[ph & 1][m], acc[i][(ph % P) * H + m], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (uint32_t m = 0; m < MI; ++m)
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) held(acc[i][m]);
    };


    const std::integral_constant<uint32_t, 0> even;
    const std::integral_constant<uint32_t, 1> odd;
    const std::integral_constant<uint32_t, MI> full;
    // two steps a turn (one loop exit keeps the sums in their registers); a step
    // past the last is all zeros
    auto aligned = [&](auto subtiles) {
        if (first < steps) {
            x_past_end(first);
            load_x(buf0, first, subtiles);
            w_past_end(first);
            load_w(first, even);
            load_pair(first);
            w_past_end(first + 1);
            load_w(first + 1, odd);
        }
        for (uint32_t t = first; t < steps; t += 2) {
            step_barrier<2 * NI>();   // x is older than the last loads of codes and scales
            x_past_end(t + 1);
            load_x(buf1, t + 1, subtiles);
            w_past_end(t + 2);
            compute(buf0, t + 1, even, subtiles);
            step_barrier<PAIRED ? NI : 2 * NI>();
            x_past_end(t + 2);
            load_x(buf0, t + 2, subtiles);
            w_past_end(t + 3);
            compute(buf1, t + 2, odd, subtiles);
        }
    };
    if constexpr (ALIGNED) {
        // A group's last tile is often less than half full: 16384 rows of 128
        // experts through 768 x 2048 97.9 -> 92.1 us.  (Not in the largest tile,
        // which has no registers for a second loop: 651 -> 657 us at
        // 8192 x 14336 x 4096.)
        constexpr bool HALF = BM == 64 || BM == 128;
        if (HALF && rows <= BM / 2)
            aligned(std::integral_constant<uint32_t, HALF ? MI / 2 : MI>());
        else
            aligned(full);
    } else if constexpr (CODES) {
        if (first < steps) {
            w_past_end(first);
            load_w(first, even);
            w_past_end(first + 1);
            load_w(first + 1, odd);
            fetch_x(first);
            put_x(buf0);
        }
        for (uint32_t t = first; t < steps; t += 2) {
            __syncthreads();
            fetch_x(t + 1);
            w_past_end(t + 2);
            compute(buf0, t + 1, even, full);
            put_x(buf1);
            __syncthreads();
            fetch_x(t + 2);
            w_past_end(t + 3);
            compute(buf1, t + 2, odd, full);
            put_x(buf0);
        }
    } else {
        fetch_w(first);
        fetch_x(first);
#pragma unroll 1
        for (uint32_t t = first; t < steps; ++t) {
            __syncthreads();
            put_w();
            put_x(buf0);
            __syncthreads();
            fetch_w(t + 1);   // (past the last: zeros)
            fetch_x(t + 1);
            compute(buf0, 0, even, full);
        }
    }

    step_barrier<0>();
    store_block<OUT, BM, BN, W, 1, BM * kRowB>(a, acc, WF == DCR_FP4_NV && a.splits == 1 ? *a.tensor_scale : 1.0f, rt, at, 0,
                                               wave * (BN / W), a.n, buf0, buf1);
}

template <uint32_t WF, typename OUT, Rows ROWS>
void launch_tile(const MArgs& a, hipStream_t st, uint32_t bm) {
    const dim3 g(a.grid);
    constexpr bool ALIGNED = ROWS == Rows::kAligned || ROWS == Rows::kPaired;
    if (ALIGNED && bm == 256)
        hipLaunchKernelGGL((fp4_mm_tile_kernel<WF, OUT, 256, 256, 8, ALIGNED ? ROWS : Rows::kAligned>), g, dim3(512), 0, st, a);
    else if (bm == 128)
        hipLaunchKernelGGL((fp4_mm_tile_kernel<WF, OUT, 128, 128, 4, ROWS>), g, dim3(256), 0, st, a);
    else if (bm == 64)
        hipLaunchKernelGGL((fp4_mm_tile_kernel<WF, OUT, 64, 128, 4, ROWS>), g, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((fp4_mm_tile_kernel<WF, OUT, 32, 128, 4, ROWS>), g, dim3(256), 0, st, a);
}
template <uint32_t WF, typename OUT>
void launch(const MArgs& a, hipStream_t st, uint32_t bm, Rows rows) {
    if (rows == Rows::kAny)
        launch_tile<WF, OUT, Rows::kAny>(a, st, bm);
    else if (rows == Rows::kCodes)
        launch_tile<WF, OUT, Rows::kCodes>(a, st, bm);
    else if (rows == Rows::kPaired)
        launch_tile<WF, OUT, Rows::kPaired>(a, st, bm);
    else
        launch_tile<WF, OUT, Rows::kAligned>(a, st, bm);
}

}  // namespace

bool fp4_mm_tile(MArgs a, uint32_t fmt, bool f32, void* ws, hipStream_t st) {
    // offsets inside a tile are 30 bits
    if (a.k < 8 || a.k >= kLongest || a.x_stride >= (1u << 21) || a.wc_stride >= (1u << 22) || a.ws_stride >= (1u << 22)) return false;
    // A step measures 2762, 850, 551 and 431 ns (MX; NV 3070 to 417), with rows
    // of x anywhere 1124, 714 and 569, with codes anywhere 1782, 1390 and 1218
    // (the costs of these lean to small tiles more than that).
    constexpr uint32_t kCost[4] = {6100, 2000, 1200, 800}, kCostCodes[4] = {0, 2400, 1500, 900}, kCostAny[4] = {0, 2800, 1700, 1100};
    // (two NV scales are read at once, so both have to be there.  Sums that end
    // in the first half of a block of 32 read their codes byte by byte
    // therefore: 4096 x 4096 x 4072 takes 164 us and 4088 110, 24 rows through
    // 4096 x 4072 14.0 and through 4088 11.4)
    const bool codes = a.w_vec && (fmt == DCR_FP4_MX || (a.ws_stride % 2 == 0 && (a.k - 1) % 32 >= 16));
    const Rows rows = !codes                                            ? Rows::kAny
                      : !a.x_vec || a.k % 8                               ? Rows::kCodes
                      : a.k % 256 || a.ws_stride % (256 / fp4_block(fmt)) ? Rows::kAligned
                                                                          : Rows::kPaired;
    const uint32_t bm = fp4_mm_plan(&a, a.n, (a.k + kBK - 1) / kBK,
                                    rows == Rows::kAny ? kCostAny : rows == Rows::kCodes ? kCostCodes : kCost);
    if (!bm) return false;
    const MArgs p = fp4_mm_parts(a, a.n, ws);
    const bool wide = f32 || a.splits > 1;
    if (fmt == DCR_FP4_MX)
        wide ? launch<DCR_FP4_MX, float>(p, st, bm, rows) : launch<DCR_FP4_MX, uint16_t>(p, st, bm, rows);
    else
        wide ? launch<DCR_FP4_NV, float>(p, st, bm, rows) : launch<DCR_FP4_NV, uint16_t>(p, st, bm, rows);
    fp4_mm_join(a, a.n, fmt, f32, ws, st);
    return true;
}

}  // namespace dcr
