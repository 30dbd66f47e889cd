// dcr_fp4_grad.hip -- gradient of a 4-bit product with respect to x, in large
// tiles (gfx950): dx[i, k] = sum_j dy[i, j] w[j, k].
//
// The sum runs over the rows of w, along which neither the codes nor their
// scales are contiguous, while a matrix operand wants eight neighbours of the
// sum in a lane.  So a step's codes (64 rows of the tile's columns) are
// converted once for the workgroup, written to LDS as bf16 rows, and read
// back by the transposing LDS load, four rows of a column at a time.
//
// 4096 x 4096 x 14336 takes 372 us (1290 TFLOP/s; the library's bf16 product of
// the same sizes takes 470 us), the matrix unit busy in 63 % of the cycles; 64
// rows through 4096 x 4096 take 14 us.
#include "dcr_fp4_mm.h"

namespace dcr {
namespace {

constexpr uint32_t kBJ = 64;             // rows of w (elements of the sum) a step takes
constexpr uint32_t kRowB = kBJ * 2;      // bytes of a row of dy in LDS

// w in LDS: block b (16 columns, 32 bytes) of row j at place b ^ turn(j): the
// eight rows that half a wave reads at once, 0-3 and 8-11 of each 16, fall on
// different banks
__device__ __forceinline__ uint32_t turn(uint32_t j) { return (j & 3u) | ((j >> 1) & 4u); }

// What is known of the rows: nothing; codes on 16-byte borders; dy there too,
// and a sum of a multiple of 8.
enum class Rows { kAny, kCodes, kAligned };

template <uint32_t WF, typename OUT, uint32_t BM, uint32_t BO, uint32_t WM, uint32_t WN, Rows ROWS>
__global__ void __launch_bounds__(WM * WN * 64, 2) fp4_mm_grad_kernel(MArgs a) {
    constexpr bool CODES = ROWS != Rows::kAny, ALIGNED = ROWS == Rows::kAligned;
    constexpr uint32_t W = WM * WN, MI = BM / WM / 16, NI = BO / WN / 16;
    constexpr uint32_t XD = BM / 8 / W;          // 1 KiB loads of dy of a wave and step
    constexpr uint32_t NB = BO / 16, PP = NB / W;   // blocks of a row of w; of a thread and step
    constexpr uint32_t RP = W * 64 / NB;         // rows of w between a thread's blocks
    constexpr uint32_t kX = BM * kRowB, kW = kBJ * BO * 2;
    // (w apart from what loads to LDS write: the compiler takes a read of the
    // same array for one of what is still on its way, and waits)
    __shared__ __attribute__((aligned(1024))) uint8_t x0[kX], x1[kX], w0[kW], w1[kW];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r16 = lane & 15u, quad = lane >> 4;
    const uint32_t wm = wave % WM, wn = wave / WM;
    const TilePlace at = tile_place(a);
    if (at.row >= a.row_tiles) return;
    const RowTile rt = row_tile<BM>(a, at.row);
    if (rt.begin == rt.end) return;
    const uint32_t rows = uint32_t(rt.end - rt.begin), o0 = at.col * BO;

    const uint32_t xstep = uint32_t(a.x_stride) * 2, wstep = uint32_t(a.wc_stride), sstep = uint32_t(a.ws_stride);
    const uint8_t* xb = static_cast<const uint8_t*>(a.x) + rt.begin * a.x_stride * 2;
    const auto xr = rsrc(xb, (rows - 1) * xstep + a.n * 2);
    const uint8_t* wb = a.wc + uint64_t(rt.group) * a.n * a.wc_stride + o0 / 2;
    const uint8_t* sb = a.ws + uint64_t(rt.group) * a.n * a.ws_stride + o0 / fp4_block(WF);
    // (a row's last eight bytes are read whole: they start on an 8-byte border)
    const uint32_t wlast = ((a.k + 1) / 2 - o0 / 2 + 7) & ~7u, slast = (a.k + fp4_block(WF) - 1) / fp4_block(WF) - o0 / fp4_block(WF);

    const uint32_t blk = threadIdx.x % NB, row0 = threadIdx.x / NB;
    const uint32_t wdst = row0 * BO * 2;
    // Codes and scales are read AHEAD + 1 steps before they multiply: small
    // tiles are bound by reading them.
    constexpr uint32_t AHEAD = BM == 256 ? 1 : 2;
    u32x2 q[AHEAD][PP];
    uint32_t sc[AHEAD][PP];
    f32x4 acc[NI][MI] = {};
    // this workgroup's steps: from `first` on, up to `steps`
    const uint32_t first = at.split * a.split_steps, steps = min(first + a.split_steps, (a.n + kBJ - 1) / kBJ);

    // dy by loads straight to LDS.  From the step on in which the sum ends (at a
    // multiple of 8) lanes past the end read behind the descriptor's range,
    // which gives zeros; a lane once past it stays there, so its offset is
    // changed for good and the other steps spend nothing on it.
    const uint32_t lr = wave * 8 + (lane >> 3), lc = (lane & 7u) ^ swizzle8(lr);
    uint32_t xo[XD];
#pragma unroll
    for (uint32_t i = 0; i < XD; ++i) xo[i] = min(tile_row<BM, WM>(lr + i * W * 8), rows - 1) * xstep + lc * 16;
    auto load_x = [&](uint8_t* buf, uint32_t step, auto subtiles) {
        if ((step + 1) * kBJ > a.n) {
            const uint32_t out = step * kBJ + lc * 8 < a.n ? 0u : kOutside;
#pragma unroll
            for (uint32_t i = 0; i < XD; ++i) xo[i] |= out;
        }
#pragma unroll
        for (uint32_t i = 0; i < XD; ++i)
            if (i * W * 8 % (BM / WM) < decltype(subtiles)::value * 16)
                load_lds16(xr, buf + (i * W + wave) * 1024, xo[i], step * kRowB);
        __builtin_amdgcn_sched_barrier(0);   // (the step's wait counts the loads after these)
    };
    // 16 codes and their scale; rows past the sum's end and columns past the
    // row's are zeros.  The rows of a step get a descriptor of their own, so
    // that lane offsets stay small in a weight of any size.
    uint32_t wo[PP], so[PP];
#pragma unroll
    for (uint32_t i = 0; i < PP; ++i) {
        const uint32_t in_row = blk * 16 + o0 < a.k ? 0u : kOutside;
        wo[i] = ((row0 + i * RP) * wstep + blk * 8) | in_row;
        so[i] = ((row0 + i * RP) * sstep + blk * 16 / fp4_block(WF)) | in_row;
    }
    auto load_w = [&](uint32_t step, auto odd) {
        constexpr uint32_t o = decltype(odd)::value % AHEAD;
        const uint32_t j0 = min(step * kBJ, a.n - 1), nrow = min(kBJ, a.n - j0);
        const auto wr = rsrc(wb + uint64_t(j0) * wstep, (nrow - 1) * wstep + wlast);
        const auto sr = rsrc(sb + uint64_t(j0) * sstep, (nrow - 1) * sstep + slast);
        if ((step + 1) * kBJ > a.n) {
#pragma unroll
            for (uint32_t i = 0; i < PP; ++i) {
                const uint32_t out = step * kBJ + row0 + i * RP < a.n ? 0u : kOutside;
                wo[i] |= out, so[i] |= out;
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < PP; ++i) {
            q[o][i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(wr, wo[i], 0, 0));
            sc[o][i] = __builtin_amdgcn_raw_buffer_load_b8(sr, so[i], 0, 0);
        }
    };
    auto convert = [&](uint8_t* wl, auto odd) {
        constexpr uint32_t o = decltype(odd)::value % AHEAD;
#pragma unroll
        for (uint32_t i = 0; i < PP; ++i) {
            const uint32_t r = row0 + i * RP;
            uint8_t* dst = wl + wdst + i * RP * BO * 2 + (blk ^ turn(r)) * 32;
            *reinterpret_cast<bf16x8*>(dst) = fp4_unpack8_bf16<WF>(q[o][i][0], sc[o][i]);
            *reinterpret_cast<bf16x8*>(dst + 16) = fp4_unpack8_bf16<WF>(q[o][i][1], sc[o][i]);
        }
    };
    // `issue` starts the next loads.  The compiler takes a transposing read for
    // one of what loads to LDS are writing, and waits for them.  In the largest
    // tile, alone on its compute unit, all of a step's come before (390 -> 372
    // us at 4096 x 4096 x 14336); the others wait in the shade of their
    // neighbours and lose by the longer start (48 -> 53 us at 1024 x 4096 x 4096).
    auto compute = [&](const uint8_t* xbuf, const uint8_t* wbuf, auto subtiles, auto&& issue) {
        constexpr uint32_t M = decltype(subtiles)::value, H = M < 2 ? M : 2, P = M / H;
        const uint8_t* xl = xbuf + (wm * (BM / WM) + r16) * kRowB;
        // a lane names four columns of a row and gets four rows of a column
        const uint32_t jr = quad * 8 + (r16 >> 2);
        const uint8_t* wl = wbuf + jr * BO * 2 + (r16 & 3u) * 8;
        constexpr bool FIRST = BM == 256;
        bf16x8 x[2][H], w[FIRST ? 2 : 1][NI];
        auto read = [&](uint32_t ph) {
#pragma unroll
            for (uint32_t m = 0; m < H; ++m)
                x[ph & 1][m] = *reinterpret_cast<const bf16x8*>(xl + ((ph % P) * H + m) * 16 * kRowB +
                                                                (((ph / P * 4 + quad) ^ swizzle8(r16)) * 16));
        };
        auto read_w = [&](uint32_t h) {
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) {
                const uint8_t* p = wl + h * 32 * BO * 2 + ((wn * NI + i) ^ turn(jr)) * 32;
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * BO * 2));
                w[FIRST ? h : 0][i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        };
        if constexpr (FIRST) {
            read_w(0);
            read_w(1);
            read(0);
            __builtin_amdgcn_sched_barrier(0);
            issue();
        } else {
            issue();
            read(0);
        }
#pragma unroll
        for (uint32_t ph = 0; ph < 2 * P; ++ph) {
            if (!FIRST && ph % P == 0) read_w(ph / P);
            if (ph + 1 < 2 * P) read(ph + 1);
#pragma unroll
            for (uint32_t m = 0; m < H; ++m)
#pragma unroll
                for (uint32_t i = 0; i < NI; ++i)
                    acc[i][(ph % P) * H + m] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[FIRST ? ph / P : 0][i], x[ph & 1][m], acc[i][(ph % P) * H + m], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (uint32_t m = 0; m < MI; ++m)
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) held(acc[i][m]);
    };

    // Any alignment: into registers while the step before multiplies, then to
    // LDS.  A piece of dy that the sum's end cuts is read as the row's last
    // eight elements and moved down.
    u32x4 xn[XD];
    auto fetch_x = [&](uint32_t step) {
        if ((step + 1) * kBJ <= a.n) {
#pragma unroll
            for (uint32_t i = 0; i < XD; ++i) __builtin_memcpy(&xn[i], xb + step * kRowB + xo[i], 16);
            return;
        }
        const uint32_t j = step * kBJ + lc * 8, past = j - min(j, a.n - 8);
#pragma unroll
        for (uint32_t i = 0; i < XD; ++i)
            xn[i] = last_elements(xb + uint64_t(xo[i]) + step * kRowB - past * 2, past);
    };
    auto put_x = [&](uint8_t* buf) {
#pragma unroll
        for (uint32_t i = 0; i < XD; ++i) *reinterpret_cast<u32x4*>(buf + (i * W + wave) * 1024 + lane * 16) = xn[i];
    };
    auto fetch_w = [&](uint32_t step) {
#pragma unroll
        for (uint32_t i = 0; i < PP; ++i) {
            const uint32_t j = step * kBJ + row0 + i * RP, c = blk * 16;   // (columns from o0 on)
            q[0][i] = u32x2{0, 0};
            sc[0][i] = 0;
            if (j < a.n && o0 + c < a.k) {
                q[0][i] = codes16(wb + uint64_t(j) * wstep, c, a.k - o0, a.w_vec);
                sc[0][i] = sb[uint64_t(j) * sstep + c / fp4_block(WF)];
            }
        }
    };
    const std::integral_constant<uint32_t, 0> even;
    const std::integral_constant<uint32_t, 1> odd;
    const std::integral_constant<uint32_t, MI> full;
    if constexpr (!CODES) {
        fetch_x(first);
        fetch_w(first);
#pragma unroll 1
        for (uint32_t t = first; t < steps; ++t) {
            __syncthreads();
            put_x(x0);
            convert(w0, even);
            __syncthreads();
            compute(x0, w0, full, [&] {   // (past the last: zeros)
                fetch_x(t + 1);
                fetch_w(t + 1);
            });
        }
    }
    // two steps a turn (one loop exit keeps the sums in their registers); a
    // step past the last is all zeros
    // (the codes are converted before the next loads are issued: a wait for them
    // would be a wait for those too)
    auto steps_of = [&](auto subtiles) {
        if (first < steps) {
            if constexpr (ALIGNED)
                load_x(x0, first, subtiles);
            else
                fetch_x(first), put_x(x0);
            load_w(first, even);
            if (AHEAD == 2) load_w(first + 1, odd);
            convert(w0, even);
            load_w(first + AHEAD, even);
        }
        for (uint32_t t = first; t < steps; t += 2) {
            step_barrier<ALIGNED ? 2 * PP : 63>();   // dy is older than the last loads of codes and scales
            convert(w1, odd);
            compute(x0, w0, subtiles, [&] {
                ALIGNED ? load_x(x1, t + 1, subtiles) : fetch_x(t + 1);
                load_w(t + 1 + AHEAD, odd);
            });
            if constexpr (!ALIGNED) put_x(x1);
            step_barrier<ALIGNED ? 2 * PP : 63>();
            convert(w0, even);
            compute(x1, w1, subtiles, [&] {
                ALIGNED ? load_x(x0, t + 2, subtiles) : fetch_x(t + 2);
                load_w(t + 2 + AHEAD, even);
            });
            if constexpr (!ALIGNED) put_x(x0);
        }
    };
    if constexpr (CODES) {
        // a group's last tile is often less than half full: 4096 rows of 128
        // experts through 768 x 2048 59.7 -> 56.4 us
        constexpr bool HALF = ALIGNED && (BM == 64 || BM == 128);
        if (HALF && rows <= BM / 2)
            steps_of(std::integral_constant<uint32_t, HALF ? MI / 2 : MI>());
        else
            steps_of(full);
    }
    step_barrier<0>();
    store_block<OUT, BM, BO, W, WM, kW>(a, acc, WF == DCR_FP4_NV && a.splits == 1 ? *a.tensor_scale : 1.0f, rt, at, wm,
                                             wn * (BO / WN), a.k, w0, w1);
}

template <uint32_t WF, typename OUT, Rows ROWS>
void launch_tile(const MArgs& a, hipStream_t st, uint32_t bm) {
    const dim3 g(a.grid);
    if (ROWS == Rows::kAligned && bm == 256)
        hipLaunchKernelGGL((fp4_mm_grad_kernel<WF, OUT, 256, 256, 2, 4, Rows::kAligned>), g, dim3(512), 0, st, a);
    else if (bm == 128)
        hipLaunchKernelGGL((fp4_mm_grad_kernel<WF, OUT, 128, 128, 2, 2, ROWS>), g, dim3(256), 0, st, a);
    else if (ROWS != Rows::kAny && bm == 64)
        hipLaunchKernelGGL((fp4_mm_grad_kernel<WF, OUT, 64, 128, 1, 4, ROWS == Rows::kAny ? Rows::kCodes : ROWS>), g, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((fp4_mm_grad_kernel<WF, OUT, 32, 128, 1, 4, ROWS>), g, dim3(256), 0, st, a);
}
template <uint32_t WF, typename OUT>
void launch(const MArgs& a, hipStream_t st, uint32_t bm, Rows rows) {
    rows == Rows::kAligned ? launch_tile<WF, OUT, Rows::kAligned>(a, st, bm)
    : rows == Rows::kCodes ? launch_tile<WF, OUT, Rows::kCodes>(a, st, bm)
                           : launch_tile<WF, OUT, Rows::kAny>(a, st, bm);
}

}  // namespace

bool fp4_mm_grad(MArgs a, uint32_t fmt, bool f32, void* ws, hipStream_t st) {
    // offsets inside a tile, and inside the rows of w of a step, are 30 bits
    if (a.n < 8 || a.n >= kLongest || a.x_stride >= (1u << 21) || a.wc_stride >= (1u << 24) || a.ws_stride >= (1u << 24)) return false;
    // A step measures 1466, 471, 296 and 218 ns (MX; NV 1578 to 246), with rows
    // of dy anywhere 562, 335 and 227, with codes anywhere 561 and 260.
    constexpr uint32_t kCost[4] = {3800, 1300, 800, 600}, kCostCodes[4] = {0, 1500, 950, 700}, kCostAny[4] = {0, 2000, 0, 900};
    const Rows rows = !a.w_vec ? Rows::kAny : !a.x_vec || a.n % 8 ? Rows::kCodes : Rows::kAligned;
    const uint32_t bm = fp4_mm_plan(&a, a.k, (a.n + kBJ - 1) / kBJ,
                                    rows == Rows::kAny ? kCostAny : rows == Rows::kCodes ? kCostCodes : kCost);
    if (!bm) return false;
    const MArgs p = fp4_mm_parts(a, a.k, ws);
    const bool wide = f32 || a.splits > 1;
    if (fmt == DCR_FP4_MX)
        wide ? launch<DCR_FP4_MX, float>(p, st, bm, rows) : launch<DCR_FP4_MX, uint16_t>(p, st, bm, rows);
    else
        wide ? launch<DCR_FP4_NV, float>(p, st, bm, rows) : launch<DCR_FP4_NV, uint16_t>(p, st, bm, rows);
    fp4_mm_join(a, a.k, fmt, f32, ws, st);
    return true;
}

}  // namespace dcr
