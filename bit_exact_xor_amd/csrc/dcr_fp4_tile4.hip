// dcr_fp4_tile4.hip -- products of two 4-bit operands in large tiles (gfx950).
//
// The scaled matrix instruction multiplies 128 codes of a row with 128 of a
// column, each run of 32 with its own power of two: a lane's operand is one
// MX block and one scale byte, and nothing is converted.
//
// 8192 x 14336 x 4096 takes 271 us (3.55 PFLOP/s), the matrix unit busy in 46 %
// of the cycles: reads from LDS and products alone take 161 us; the codes' loads
// add some 65, the scales' way through LDS 35 and the results' 45.  Tried and
// not kept: four waves of 128 x 128 (a third less read from LDS, but the
// compiler moves full accumulation registers about: 415 us), scales eight
// bytes a row in LDS (285 us), columns' codes of a step's second half read
// ahead (even), raised priority for half of the waves (even).
#include "dcr_fp4_mm.h"

namespace dcr {
namespace {

constexpr uint32_t kBK = 256;                // elements of the sum a step takes
constexpr uint32_t kRowB = kBK / 2;          // bytes of a row of codes in LDS

// What is known of the rows: nothing; codes on 16-byte borders (a row's last
// codes and scales are then read with what shares their 16 or 4 bytes); and
// scales on 8-byte borders as well, with a sum of whole steps (sums that end
// anywhere cost 3 % at 8192 x 14336 x 4096).
enum class Rows { kAny, kAligned, kScales };

template <typename OUT, uint32_t BM, uint32_t BN, uint32_t WM, uint32_t WN, Rows ROWS>
__global__ void __launch_bounds__(WM * WN * 64, 2) fp4_mm_tile4_kernel(MArgs a) {
    constexpr bool SV = ROWS == Rows::kScales;
    constexpr uint32_t W = WM * WN, MI = BM / WM / 16, NI = BN / WN / 16;
    constexpr uint32_t XD = BM / 8 / W, WD = BN / 8 / W;   // 1 KiB loads of a wave and step
    static_assert(W * 64 >= BM + BN && BM % 64 == 0, "a thread stages the scales of one row, a wave those of one operand");
    static_assert(MI % 4 == 0 && (NI % 4 == 0 || NI == 2), "a subtile's scale byte is its index mod 4");
    constexpr uint32_t kCodes = (BM + BN) * kRowB, kScales = (BM + BN) * (kBK / 32);
    // (scales apart from what loads to LDS write: the compiler takes a read of
    // the same array for one of what is still on its way, and waits)
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[kCodes], buf1[kCodes];
    __shared__ __attribute__((aligned(16))) uint8_t sc0[kScales], sc1[kScales];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r16 = lane & 15u, quad = lane >> 4;
    const uint32_t wm = wave % WM, wn = wave / WM;
    const TilePlace at = tile_place(a);
    if (at.row >= a.row_tiles) return;
    const RowTile rt = row_tile<BM>(a, at.row);
    if (rt.begin == rt.end) return;
    const uint32_t rows = uint32_t(rt.end - rt.begin), n0 = at.col * BN, cols = min(BN, a.n - n0);

    const uint8_t* wb = a.wc + (uint64_t(rt.group) * a.n + n0) * a.wc_stride;
    const uint8_t* sb = a.ws + (uint64_t(rt.group) * a.n + n0) * a.ws_stride;
    const uint32_t xstep = uint32_t(a.x_stride), wstep = uint32_t(a.wc_stride);
    const uint32_t last_codes = ((a.k + 1) / 2 + 15) & ~15u;
    const auto xr = rsrc(static_cast<const uint8_t*>(a.x) + rt.begin * a.x_stride, (rows - 1) * xstep + last_codes);
    const auto wr = rsrc(wb, (cols - 1) * wstep + last_codes);

    // the row whose scales this thread stages (x's, then w's), and where they
    // go: [quarter of the step][quad][row of a subtile][subtile], so that a
    // lane reads the bytes of its subtiles at once
    const bool xside = wave < BM / 64;      // whole waves: the descriptor stays scalar
    const uint32_t srow = xside ? threadIdx.x : (threadIdx.x - BM) % BN;   // (spare threads do one over)
    const uint32_t last = (xside ? rows : cols) - 1;
    const uint32_t sstep = uint32_t(xside ? a.xs_stride : a.ws_stride), blocks = (a.k + 31) / 32;
    const uint8_t* srows = xside ? a.xs + rt.begin * a.xs_stride : sb;
    const uint32_t skew = SV ? 0 : uint32_t(reinterpret_cast<uintptr_t>(srows)) & 3u;
    const auto sr = rsrc(srows - skew, (skew + last * sstep + blocks + 3) & ~3u);
    const uint32_t soff = skew + min(xside ? tile_row<BM, WM>(srow) : srow, last) * sstep;
    const uint32_t subs = xside ? BM / 16 : BN / 16;
    const uint32_t sdst = (xside ? 0 : BM * (kBK / 32)) + (srow & 15u) * subs + (srow >> 4);

    f32x4 acc[NI][MI] = {};
    // this workgroup's steps: from `first` on, up to `steps`
    const uint32_t first = at.split * a.split_steps, steps = min(first + a.split_steps, (a.k + kBK - 1) / kBK);

    // Codes of a step by loads straight to LDS.  From the step on in which the
    // sum ends lanes whose block is past the end read behind the
    // descriptors' range, which gives zeros; a lane once past it stays there,
    // so its offset is changed for good and the other steps spend nothing on it.
    const uint32_t lr = wave * 8 + (lane >> 3), lc = (lane & 7u) ^ swizzle8(lr);
    uint32_t xo[XD], wo[WD];
#pragma unroll
    for (uint32_t i = 0; i < XD; ++i) xo[i] = min(tile_row<BM, WM>(lr + i * W * 8), rows - 1) * xstep + lc * 16;
#pragma unroll
    for (uint32_t i = 0; i < WD; ++i) wo[i] = min(lr + i * W * 8, cols - 1) * wstep + lc * 16;
    auto load = [&](uint8_t* buf, uint32_t step) {
        if ((step + 1) * kBK > a.k) {
            const uint32_t out = step * kBK + lc * 32 < a.k ? 0u : kOutside;
#pragma unroll
            for (uint32_t i = 0; i < XD; ++i) xo[i] |= out;
#pragma unroll
            for (uint32_t i = 0; i < WD; ++i) wo[i] |= out;
        }
#pragma unroll
        for (uint32_t i = 0; i < XD; ++i) load_lds16(xr, buf + (i * W + wave) * 1024, xo[i], step * kRowB);
#pragma unroll
        for (uint32_t i = 0; i < WD; ++i) load_lds16(wr, buf + BM * kRowB + (i * W + wave) * 1024, wo[i], step * kRowB);
    };
    // The eight scale bytes of a step of this thread's row, as whole words that
    // hold them (one load for eight bytes a row costs what one for a byte does).
    auto load_scales = [&](uint32_t step) -> u32x4 {
        const uint32_t b = step * (kBK / 32), out = b < blocks ? 0u : kOutside;
        if constexpr (SV) {
            const auto q = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, soff | out, b, 0));
            return u32x4{q[0], q[1], 0, 0};
        } else {
            u32x4 v = {};
#pragma unroll
            for (uint32_t i = 0; i < 3; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b32(sr, ((soff & ~3u) + b + 4 * i) | out, 0, 0);
            return v;
        }
    };
    // ... to LDS, zeros for blocks past the end
    auto store_scales = [&](uint8_t* sc, u32x4 v, uint32_t step) {
        const uint32_t n = blocks - min(blocks, step * (kBK / 32));
        if constexpr (!SV) {
            v[0] = __builtin_amdgcn_alignbyte(v[1], v[0], soff & 3u);
            v[1] = __builtin_amdgcn_alignbyte(v[2], v[1], soff & 3u);
        }
        if (!SV && n < 8) {
            v[0] &= n < 4 ? (1u << (8 * n)) - 1u : ~0u;
            v[1] &= n < 4 ? 0u : (1u << (8 * n - 32)) - 1u;
        }
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) sc[sdst + i * 16 * subs] = uint8_t(v[i / 4] >> (8 * (i & 3)));
    };
    // A sum that ends inside a block: x's codes past the end (w's are finite,
    // and the block's scales their own) become zeros in LDS.
    const uint32_t tail = a.k % 32;
    auto end_inside = [&](uint8_t* buf, uint32_t step) {
        if (SV || tail == 0 || step != a.k / kBK) return;
        if (threadIdx.x < BM) {
            u32x4* p = reinterpret_cast<u32x4*>(buf + threadIdx.x * kRowB + ((a.k % kBK / 32) ^ swizzle8(threadIdx.x)) * 16);
            u32x4 v = *p;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) v[i] &= tail >= 8 * i + 8 ? ~0u : tail <= 8 * i ? 0u : (1u << (4 * (tail - 8 * i))) - 1u;
            *p = v;
        }
        __syncthreads();
    };
    auto compute = [&](const uint8_t* buf, const uint8_t* sc) {
        constexpr uint32_t H = 2, P = MI / H;
        const uint8_t* xl = buf + (wm * (BM / WM) + r16) * kRowB;
        const uint8_t* wl = buf + BM * kRowB + (wn * (BN / WN) + r16) * kRowB;
        u32x4 x[2][H], w[NI];
        uint32_t xs[MI / 4], ws[(NI + 3) / 4];
        auto read = [&](uint32_t ph) {
#pragma unroll
            for (uint32_t m = 0; m < H; ++m)
                x[ph & 1][m] = *reinterpret_cast<const u32x4*>(xl + ((ph % P) * H + m) * 16 * kRowB +
                                                               (((ph / P * 4 + quad) ^ swizzle8(r16)) * 16));
        };
        read(0);
#pragma unroll
        for (uint32_t ph = 0; ph < 2 * P; ++ph) {
            const uint32_t j = ph / P;
            if (ph % P == 0) {
                const uint8_t* s = sc + (j * 4 + quad) * 16 * (BM / 16) + r16 * (BM / 16) + wm * MI;
                const uint8_t* t = sc + BM * (kBK / 32) + (j * 4 + quad) * 16 * (BN / 16) + r16 * (BN / 16) + wn * NI;
#pragma unroll
                for (uint32_t i = 0; i < MI / 4; ++i) xs[i] = *reinterpret_cast<const uint32_t*>(s + i * 4);
                if constexpr (NI % 4 == 0) {
#pragma unroll
                    for (uint32_t i = 0; i < NI / 4; ++i) ws[i] = *reinterpret_cast<const uint32_t*>(t + i * 4);
                } else {
                    ws[0] = *reinterpret_cast<const uint16_t*>(t);
                }
#pragma unroll
                for (uint32_t i = 0; i < NI; ++i)
                    w[i] = *reinterpret_cast<const u32x4*>(wl + i * 16 * kRowB + (((j * 4 + quad) ^ swizzle8(r16)) * 16));
            }
            if (ph + 1 < 2 * P) read(ph + 1);
            // byte of a subtile in its scale word: the subtile's index mod 4
            const auto mul = [&](auto mc, auto ic) {
                constexpr uint32_t m = decltype(mc)::value, i = decltype(ic)::value;
                const uint32_t mi = (ph % P) * H + m;
                acc[i][mi] = (mi & 3u) == m ? mfma_fp4<i & 3, m>(w[i], x[ph & 1][m], acc[i][mi], ws[i / 4], xs[mi / 4])
                                            : mfma_fp4<i & 3, m + H>(w[i], x[ph & 1][m], acc[i][mi], ws[i / 4], xs[mi / 4]);
            };
            static_for<H>([&](auto m) { static_for<NI>([&](auto i) { mul(m, i); }); });
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (uint32_t m = 0; m < MI; ++m)
#pragma unroll
            for (uint32_t i = 0; i < NI; ++i) held(acc[i][m]);
    };

    // Any step, any alignment: into registers while the step before multiplies
    // (zeros past the rows' ends), then to LDS.
    u32x4 xnext[XD], wnext[WD];
    u32x4 sn;
    auto fetch = [&](uint32_t step) {
        const uint32_t k = step * kBK + lc * 32;
        const uint8_t* x = static_cast<const uint8_t*>(a.x) + rt.begin * a.x_stride;
#pragma unroll
        for (uint32_t i = 0; i < XD; ++i) xnext[i] = codes32(x + uint64_t(min(tile_row<BM, WM>(lr + i * W * 8), rows - 1)) * xstep, k, a.k, a.x_vec);
#pragma unroll
        for (uint32_t i = 0; i < WD; ++i) wnext[i] = codes32(wb + uint64_t(min(lr + i * W * 8, cols - 1)) * wstep, k, a.k, a.w_vec);
        sn = load_scales(step);
    };
    if constexpr (ROWS == Rows::kAny) {
        fetch(first);
#pragma unroll 1
        for (uint32_t t = first; t < steps; ++t) {
            __syncthreads();
#pragma unroll
            for (uint32_t i = 0; i < XD; ++i) *reinterpret_cast<u32x4*>(buf0 + (i * W + wave) * 1024 + lane * 16) = xnext[i];
#pragma unroll
            for (uint32_t i = 0; i < WD; ++i)
                *reinterpret_cast<u32x4*>(buf0 + BM * kRowB + (i * W + wave) * 1024 + lane * 16) = wnext[i];
            store_scales(sc0, sn, t);
            __syncthreads();
            fetch(t + 1);   // (past the last: zeros)
            compute(buf0, sc0);
        }
    }
    if (ROWS != Rows::kAny && first < steps) {
        load(buf0, first);
        store_scales(sc0, load_scales(first), first);
    }
    // two steps a turn (one loop exit keeps the sums in their registers); a
    // step past the last is all zeros
    for (uint32_t t = first; ROWS != Rows::kAny && t < steps; t += 2) {
        step_barrier<0>();
        end_inside(buf0, t);
        const u32x4 s1 = load_scales(t + 1);
        load(buf1, t + 1);
        compute(buf0, sc0);
        store_scales(sc1, s1, t + 1);
        step_barrier<0>();
        end_inside(buf1, t + 1);
        const u32x4 s2 = load_scales(t + 2);
        load(buf0, t + 2);
        compute(buf1, sc1);
        store_scales(sc0, s2, t + 2);
    }
    step_barrier<0>();
    store_block<OUT, BM, BN, W, WM, kCodes>(a, acc, 1.0f, rt, at, wm, wn * (BN / WN), a.n, buf0, buf1);
}

template <typename OUT, Rows ROWS>
void launch(const MArgs& a, hipStream_t st, uint32_t bm) {
    const dim3 g(a.grid);
    if (ROWS != Rows::kAny && bm == 256)
        hipLaunchKernelGGL((fp4_mm_tile4_kernel<OUT, 256, 256, 2, 4, ROWS == Rows::kAny ? Rows::kAligned : ROWS>), g, dim3(512), 0, st, a);
    else if (bm == 128)
        hipLaunchKernelGGL((fp4_mm_tile4_kernel<OUT, 128, 128, 2, 2, ROWS>), g, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((fp4_mm_tile4_kernel<OUT, 64, 128, 1, 4, ROWS>), g, dim3(256), 0, st, a);
}
template <typename OUT>
void launch(const MArgs& a, hipStream_t st, uint32_t bm, Rows rows) {
    if (rows == Rows::kAny)
        launch<OUT, Rows::kAny>(a, st, bm);
    else if (rows == Rows::kAligned)
        launch<OUT, Rows::kAligned>(a, st, bm);
    else
        launch<OUT, Rows::kScales>(a, st, bm);
}

}  // namespace

bool fp4_mm_tile4(MArgs a, bool f32, void* ws, hipStream_t st) {
    // offsets inside a tile are 30 bits
    if (a.k >= kLongest || a.x_stride >= (1u << 22) || a.wc_stride >= (1u << 22) || a.xs_stride >= (1u << 22) || a.ws_stride >= (1u << 22))
        return false;
    const Rows rows = !a.x_vec || !a.w_vec                                             ? Rows::kAny
                      : a.k % kBK == 0 && a.xs_stride % 8 == 0 && a.ws_stride % 8 == 0 ? Rows::kScales
                                                                                       : Rows::kAligned;
    // A step measures 2055, 670 and 480 ns, with rows anywhere 1264 and 983.
    constexpr uint32_t kCost[4] = {4800, 1600, 1000, 0}, kCostAny[4] = {0, 3000, 1800, 0};
    const uint32_t bm = fp4_mm_plan(&a, a.n, (a.k + kBK - 1) / kBK, rows == Rows::kAny ? kCostAny : kCost);
    if (!bm) return false;
    const MArgs p = fp4_mm_parts(a, a.n, ws);
    f32 || a.splits > 1 ? launch<float>(p, st, bm, rows) : launch<uint16_t>(p, st, bm, rows);
    fp4_mm_join(a, a.n, DCR_FP4_MX, f32, ws, st);
    return true;
}

}  // namespace dcr
