// dcr_rows.hip -- rows of tokens to the slots of their experts and back.
//
//   dispatch      y[slot[t, j]] = x[t]
//   combine       y[t] = sum over j of w[t, j] x[slot[t, j]]   (w absent: 1)
//   combine_grad  dx[slot[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], x[slot[t, j]]>
//
// All are bound by memory: the rows of slots are read or written once, the
// tokens' rows once.  So the work goes by token, never by slot (which would
// read each token k times), and no row is moved in between.
#include "dcr_step.h"

namespace dcr {
namespace {

constexpr uint32_t kRT = 256;              // threads of a workgroup
constexpr uint32_t kRows = 4;              // rows that a thread has on their way

struct RowArgs {
    const void* a;         // dispatch, combine: x; gradient: dy
    const void* b;         // gradient: x
    void* y;               // dispatch, combine: y; gradient: dx
    const int32_t* slots;
    const float* weights;
    float* dweights;
    uint64_t a_stride, b_stride, y_stride;
    uint32_t tokens, width, k, n_slots;
    uint32_t pieces;       // of eight columns, of a row
};

// Eight columns from c on, of a row of at least eight: a piece that would end
// behind the row is moved back over the one in front, so all are whole (both then
// write the same; taken column by column the last piece holds up its whole wave:
// 32380 tokens' gradient, 10 rows of 198 columns each, 166 us, so 66).  Returns by
// how much.
__device__ __forceinline__ uint32_t moved_back(uint32_t width, uint32_t* c) {
    const uint32_t by = width >= 8 && *c + 8 > width ? *c + 8 - width : 0;
    *c -= by;
    return by;
}

// The thread's token and the first of its eight columns; false behind the end.
// Threads are dealt to pieces of eight columns one after the other, whatever the
// width, so none is without work in the middle of a row.
__device__ __forceinline__ bool piece_of(const RowArgs& a, uint32_t* at, uint32_t* c) {
    const uint32_t i = blockIdx.x * kRT + threadIdx.x;
    *at = i / a.pieces;
    *c = (i - *at * a.pieces) * 8;
    moved_back(a.width, c);
    return *at < a.tokens;
}

// One thread holds eight columns of a token and takes them to every slot.
template <typename TX, typename TY, bool FAR>
__global__ void __launch_bounds__(kRT) rows_dispatch_kernel(RowArgs a) {
    uint32_t at, c;
    if (!piece_of(a, &at, &c)) return;
    const int32_t* slots = a.slots + uint64_t(at) * a.k;
    const TX* x = static_cast<const TX*>(a.a) + uint64_t(at) * a.a_stride + c;
    const int n = int(min(8u, a.width - c));
    Raw8<TX> r;
    float v[8];
    n == 8 ? r.load_once(x) : r.load_some(x, n, 0);
    r.get(v);
    for (uint32_t j = 0; j < a.k; ++j) {
        const uint32_t s = uint32_t(slots[j]);
        if (s >= a.n_slots) continue;
        TY* y = static_cast<TY*>(a.y) + uint64_t(s) * a.y_stride + c;
        n == 8 ? store8<FAR>(y, v) : store_some(y, v, n);
    }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kRT) rows_combine_kernel(RowArgs a) {
    uint32_t at, c;
    if (!piece_of(a, &at, &c)) return;
    const int32_t* slots = a.slots + uint64_t(at) * a.k;
    const float* weights = a.weights + uint64_t(at) * a.k;
    const int n = int(min(8u, a.width - c));
    float sum[8] = {};
    // kRows rows on their way together
    for (uint32_t j0 = 0; j0 < a.k; j0 += kRows) {
        Raw8<TX> r[kRows];
        float w[kRows];
        bool has[kRows];
#pragma unroll
        for (uint32_t u = 0; u < kRows; ++u) {
            const uint32_t s = j0 + u < a.k ? uint32_t(slots[j0 + u]) : ~0u;
            has[u] = s < a.n_slots;
            if (!has[u]) continue;
            w[u] = a.weights ? weights[j0 + u] : 1.0f;
            const TX* x = static_cast<const TX*>(a.a) + uint64_t(s) * a.a_stride + c;
            n == 8 ? r[u].load_once(x) : r[u].load_some(x, n, 0);
        }
#pragma unroll
        for (uint32_t u = 0; u < kRows; ++u) {
            if (!has[u]) continue;
            float v[8];
            r[u].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = __fmaf_rn(w[u], v[i], sum[i]);
        }
    }
    TY* y = static_cast<TY*>(a.y) + uint64_t(at) * a.y_stride + c;
    n == 8 ? store8(y, sum) : store_some(y, sum, n);
}

// Part of a pair's row: WAVES waves of a workgroup have columns 8 (lane + 64
// wave), the next lie 512 WAVES further.  Returns the lane's share of dw.
template <typename TD, typename TX, typename TG, bool FAR, uint32_t WAVES>
__device__ __forceinline__ float pair_grad(const RowArgs& a, const TD* dy, const TX* x, TG* dx, float w, uint32_t first) {
    float dot = 0.0f;
#pragma unroll 2
    for (uint32_t c0 = first; c0 < a.width; c0 += 512 * WAVES) {
        uint32_t c = c0;
        const int twice = int(moved_back(a.width, &c)), n = int(min(8u, a.width - c));
        Raw8<TD> rd;
        Raw8<TX> rx;
        float d[8], v[8];
        if (n == 8) {
            rd.load(dy + c);
            rx.load_once(x + c);
        } else {
            rd.load_some(dy + c, n, 0);
            rx.load_some(x + c, n, 0);
        }
        rd.get(d);
        rx.get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dot = i < twice ? dot : __fmaf_rn(d[i], v[i], dot);
            d[i] *= w;
        }
        n == 8 ? store8<FAR>(dx + c, d) : store_some(dx + c, d, n);
    }
    return dot;
}

// A wave for each token, which reads dy once (from then on the cache has it).
template <typename TD, typename TX, typename TG, bool FAR>
__global__ void __launch_bounds__(kRT) rows_combine_grad_kernel(RowArgs a) {
    const uint32_t at = blockIdx.x * (kRT / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63u;
    if (at >= a.tokens) return;
    const TD* dy = static_cast<const TD*>(a.a) + uint64_t(at) * a.a_stride;
    for (uint32_t j = 0; j < a.k; ++j) {
        const uint64_t pair = uint64_t(at) * a.k + j;
        const uint32_t s = uint32_t(a.slots[pair]);
        float dot = 0.0f;
        if (s < a.n_slots)
            dot = pair_grad<TD, TX, TG, FAR, 1>(a, dy, static_cast<const TX*>(a.b) + uint64_t(s) * a.b_stride,
                                                static_cast<TG*>(a.y) + uint64_t(s) * a.y_stride, a.weights[pair], lane * 8);
        dot = lanes_sum<64>(dot);
        if (lane == 0) a.dweights[pair] = dot;
    }
}

// Narrow rows: LANES lanes hold a token's row of dy, several tokens share a wave,
// and kRows rows of x are on their way together.
template <typename TD, typename TX, typename TG, int LANES>
__global__ void __launch_bounds__(kRT) rows_combine_grad_narrow_kernel(RowArgs a) {
    const uint32_t at = blockIdx.x * (kRT / LANES) + threadIdx.x / LANES, first = threadIdx.x % LANES * 8;
    const bool live = at < a.tokens;
    const uint64_t safe = live ? at : 0;
    uint32_t c = first < a.width ? first : 0;
    const int twice = int(moved_back(a.width, &c)), n = first < a.width ? int(min(8u, a.width - c)) : 0;
    Raw8<TD> rd;
    float d[8];
    const TD* dy = static_cast<const TD*>(a.a) + safe * a.a_stride + c;
    n == 8 ? rd.load_once(dy) : rd.load_some(dy, n, 0);
    rd.get(d);
    for (uint32_t j0 = 0; j0 < a.k; j0 += kRows) {
        Raw8<TX> rx[kRows];
        uint32_t s[kRows];
#pragma unroll
        for (uint32_t u = 0; u < kRows; ++u) {
            s[u] = live && j0 + u < a.k ? uint32_t(a.slots[safe * a.k + j0 + u]) : ~0u;
            if (s[u] >= a.n_slots) continue;
            const TX* x = static_cast<const TX*>(a.b) + uint64_t(s[u]) * a.b_stride + c;
            n == 8 ? rx[u].load_once(x) : rx[u].load_some(x, n, 0);
        }
#pragma unroll
        for (uint32_t u = 0; u < kRows; ++u) {
            if (j0 + u >= a.k) break;
            const uint64_t pair = safe * a.k + j0 + u;
            float dot = 0.0f;
            if (s[u] < a.n_slots) {
                const float w = a.weights[pair];
                float v[8], g[8];
                rx[u].get(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot = i < twice ? dot : __fmaf_rn(d[i], v[i], dot);
                    g[i] = d[i] * w;
                }
                TG* dx = static_cast<TG*>(a.y) + uint64_t(s[u]) * a.y_stride + c;
                n == 8 ? store8(dx, g) : store_some(dx, g, n);
            }
            dot = lanes_sum<LANES>(dot);
            if (first == 0 && live) a.dweights[pair] = dot;
        }
    }
}

// A workgroup for each pair, where tokens alone do not fill the GPU.
template <typename TD, typename TX, typename TG>
__global__ void __launch_bounds__(kRT) rows_combine_grad_pair_kernel(RowArgs a) {
    __shared__ float of_wave[kRT / 64];
    const uint32_t pair = blockIdx.x;
    const uint32_t s = uint32_t(a.slots[pair]);
    float dot = 0.0f;
    if (s < a.n_slots)
        dot = pair_grad<TD, TX, TG, false, kRT / 64>(a, static_cast<const TD*>(a.a) + uint64_t(pair / a.k) * a.a_stride,
                                                   static_cast<const TX*>(a.b) + uint64_t(s) * a.b_stride,
                                                   static_cast<TG*>(a.y) + uint64_t(s) * a.y_stride, a.weights[pair], threadIdx.x * 8);
    dot = lanes_sum<64>(dot);
    if ((threadIdx.x & 63u) == 0) of_wave[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t w = 1; w < kRT / 64; ++w) dot += of_wave[w];
        a.dweights[pair] = dot;
    }
}

int32_t check_rows(uint64_t tokens, uint64_t width, uint32_t k, uint64_t n_slots, const int32_t* slots) {
    if (tokens >= (uint64_t(1) << 31) || n_slots >= (uint64_t(1) << 31) || width >= (uint64_t(1) << 31))
        return step_fail(DCR_E_INVAL, "2^31 rows, slots or columns or more");
    if (!k || k > DCR_EXPERTS_MAX_K) return step_fail(DCR_E_INVAL, "k is not 1 .. 64");
    if (tokens && width) return check_array(slots, "slots");
    return DCR_OK;
}

// f(whether so many bf16 results go past the caches: more than the last of them,
// 256 MiB, holds).  16384 tokens there and back with 8 rows of 2048 bf16
// 220 us, else 237; their gradient 234 and 246.  Below it they stay for the
// product that reads them next (4096 tokens' gradient 52 us, past the caches 63).
template <typename T, typename F>
void with_far(T, uint64_t elements, F&& f) {
    if constexpr (sizeof(T) == 2)
        if (elements * sizeof(T) > (uint64_t(256) << 20)) return f(std::true_type());
    f(std::false_type());
}

int32_t row_grid(uint64_t units, uint32_t per_group, uint32_t* grid) {
    const uint64_t g = (units + per_group - 1) / per_group;
    if (g * kRT >= (uint64_t(1) << 32)) return step_fail(DCR_E_INVAL, "too many rows for one launch");
    *grid = uint32_t(g);
    return DCR_OK;
}

int32_t dispatch_rows(const void* x, uint32_t x_type, uint64_t x_stride, uint64_t tokens, uint64_t width, const int32_t* slots,
                      uint32_t k, void* y, uint32_t y_type, uint64_t y_stride, uint64_t n_slots, hipStream_t st) {
    int32_t rc;
    if ((rc = check_rows(tokens, width, k, n_slots, slots)) || (rc = check_matrix(x, x_type, tokens, width, x_stride, "x")) ||
        (rc = check_matrix(y, y_type, n_slots, width, y_stride, "y")))
        return rc;
    if (!tokens || !width || !n_slots) return DCR_OK;
    RowArgs a{};
    a.a = x, a.y = y, a.slots = slots, a.a_stride = x_stride, a.y_stride = n_slots > 1 ? y_stride : 0;
    a.tokens = uint32_t(tokens), a.width = uint32_t(width), a.k = k, a.n_slots = uint32_t(n_slots);
    a.pieces = uint32_t((width + 7) / 8);
    uint32_t grid;
    if ((rc = row_grid(tokens * a.pieces, kRT, &grid))) return rc;
    with_type(x_type, [&](auto tx) {
        with_type(y_type, [&](auto ty) {
            with_far(ty, uint64_t(n_slots) * width, [&](auto far) {
                hipLaunchKernelGGL((rows_dispatch_kernel<decltype(tx), decltype(ty), decltype(far)::value>), dim3(grid), dim3(kRT),
                                   0, st, a);
            });
        });
    });
    return step_launched();
}

int32_t combine_rows(const void* x, uint32_t x_type, uint64_t x_stride, uint64_t n_slots, const int32_t* slots,
                     const float* weights, uint64_t tokens, uint64_t width, uint32_t k, void* y, uint32_t y_type,
                     uint64_t y_stride, hipStream_t st) {
    int32_t rc;
    if ((rc = check_rows(tokens, width, k, n_slots, slots)) || (rc = check_matrix(x, x_type, n_slots, width, x_stride, "x")) ||
        (rc = check_matrix(y, y_type, tokens, width, y_stride, "y")))
        return rc;
    if (!tokens || !width) return DCR_OK;
    if (weights && (rc = check_array(weights, "weights"))) return rc;
    RowArgs a{};
    a.a = x, a.y = y, a.slots = slots, a.weights = weights, a.a_stride = n_slots > 1 ? x_stride : 0, a.y_stride = y_stride;
    a.tokens = uint32_t(tokens), a.width = uint32_t(width), a.k = k, a.n_slots = uint32_t(n_slots);
    a.pieces = uint32_t((width + 7) / 8);
    uint32_t grid;
    if ((rc = row_grid(tokens * a.pieces, kRT, &grid))) return rc;
    with_type(x_type, [&](auto tx) {
        with_type(y_type, [&](auto ty) {
            hipLaunchKernelGGL((rows_combine_kernel<decltype(tx), decltype(ty)>), dim3(grid), dim3(kRT), 0, st, a);
        });
    });
    return step_launched();
}

int32_t combine_rows_grad(const void* dy, uint32_t dy_type, uint64_t dy_stride, uint64_t tokens, uint64_t width, const void* x,
                          uint32_t x_type, uint64_t x_stride, uint64_t n_slots, const int32_t* slots, const float* weights,
                          uint32_t k, void* dx, uint32_t dx_type, uint64_t dx_stride, float* dweights, hipStream_t st) {
    int32_t rc;
    if ((rc = check_rows(tokens, width, k, n_slots, slots)) || (rc = check_matrix(dy, dy_type, tokens, width, dy_stride, "dy")) ||
        (rc = check_matrix(x, x_type, n_slots, width, x_stride, "x")) ||
        (rc = check_matrix(dx, dx_type, n_slots, width, dx_stride, "dx")))
        return rc;
    if (!tokens) return DCR_OK;
    if ((rc = check_array(slots, "slots")) || (rc = check_array(weights, "weights")) || (rc = check_array(dweights, "dweights")))
        return rc;
    RowArgs a{};
    a.a = dy, a.b = x, a.y = dx, a.slots = slots, a.weights = weights, a.dweights = dweights;
    a.a_stride = dy_stride, a.b_stride = n_slots > 1 ? x_stride : 0, a.y_stride = n_slots > 1 ? dx_stride : 0;
    a.tokens = uint32_t(tokens), a.width = uint32_t(width), a.k = k, a.n_slots = uint32_t(n_slots);
    uint32_t grid;
    // Wide rows of few tokens by pair (256 tokens, 8 pairs of 2048 bf16: 5.6 us, a
    // wave a token 20; 2048 tokens, 8 pairs: even; 16384: 239 and 235).
    const bool narrow = width <= 512, by_pair = !narrow && tokens < 2048;
    uint32_t lanes = 8;
    while (narrow && lanes * 8 < width) lanes *= 2;
    if ((rc = by_pair ? row_grid(tokens * k, 1, &grid) : row_grid(tokens, narrow ? kRT / lanes : kRT / 64, &grid))) return rc;
    with_type(dy_type, [&](auto td) {
        with_type(x_type, [&](auto tx) {
            with_type(dx_type, [&](auto tg) {
                typedef decltype(td) TD;
                typedef decltype(tx) TX;
                typedef decltype(tg) TG;
                const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(kRT), 0, st, a); };
                if (narrow) {
                    lanes == 8    ? go(rows_combine_grad_narrow_kernel<TD, TX, TG, 8>)
                    : lanes == 16 ? go(rows_combine_grad_narrow_kernel<TD, TX, TG, 16>)
                    : lanes == 32 ? go(rows_combine_grad_narrow_kernel<TD, TX, TG, 32>)
                                  : go(rows_combine_grad_narrow_kernel<TD, TX, TG, 64>);
                } else if (by_pair) {
                    go(rows_combine_grad_pair_kernel<TD, TX, TG>);
                } else {
                    with_far(tg, uint64_t(n_slots) * width,
                             [&](auto far) { go(rows_combine_grad_kernel<TD, TX, TG, decltype(far)::value>); });
                }
            });
        });
    });
    return step_launched();
}

}  // namespace
}  // namespace dcr

extern "C" {

int32_t dcr_experts_dispatch(const void* x, uint32_t x_type, uint64_t x_stride, uint64_t tokens, uint64_t width,
                             const int32_t* slots, uint32_t k, void* y, uint32_t y_type, uint64_t y_stride, uint64_t n_slots,
                             void* stream) try {
    dcr::set_error("");
    return dcr::dispatch_rows(x, x_type, x_stride, tokens, width, slots, k, y, y_type, y_stride, n_slots,
                              static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_experts_combine(const void* x, uint32_t x_type, uint64_t x_stride, uint64_t n_slots, const int32_t* slots,
                            const float* weights, uint64_t tokens, uint64_t width, uint32_t k, void* y, uint32_t y_type,
                            uint64_t y_stride, void* stream) try {
    dcr::set_error("");
    return dcr::combine_rows(x, x_type, x_stride, n_slots, slots, weights, tokens, width, k, y, y_type, y_stride,
                             static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

int32_t dcr_experts_combine_grad(const void* dy, uint32_t dy_type, uint64_t dy_stride, uint64_t tokens, uint64_t width,
                                 const void* x, uint32_t x_type, uint64_t x_stride, uint64_t n_slots, const int32_t* slots,
                                 const float* weights, uint32_t k, void* dx, uint32_t dx_type, uint64_t dx_stride,
                                 float* dweights, void* stream) try {
    dcr::set_error("");
    return dcr::combine_rows_grad(dy, dy_type, dy_stride, tokens, width, x, x_type, x_stride, n_slots, slots, weights, k, dx,
                                  dx_type, dx_stride, dweights, static_cast<hipStream_t>(stream));
} catch (...) {
    return DCR_E_NOMEM;
}

}  // extern "C"
