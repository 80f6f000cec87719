// Gated feed-forward block and its gradients on the tensor cores:
//
//   a = x Wg^T, b = x Wu^T, h = act(a) * b                 x: M x K, W: N x K
//   dA = dh * b * act'(a), dB = dh * act(a)
//   dx = dA Wg + dB Wu, dWg = dA^T x, dWu = dB^T x
//
// Forward: one product kernel whose tile holds the same columns of a and of b
// side by side in tensor memory (the first half of B's rows come from Wg, the
// other half from Wu), so the epilogue has both in one thread and only h is
// written. Backward: the same product again, with an epilogue that reads dh
// and writes dA and dB (16 bits, as the tensor cores take them: the one extra
// rounding there is; a and b themselves are never rounded), then one product
// that sums dA Wg + dB Wu in one accumulator, and one launch for both weight
// gradients, computed as their transposes x^T dA and x^T dB from a transposed
// copy of x: a K-major A operand is worth more than the copy (both operands
// MN-major took 820 us for 4096 x 14336 x 4096, this 757 and 15 for the copy,
// before the waits were mended: 611 now). a and b are computed again instead of
// kept: kept in 16 bits they would bring two more roundings into dA and dB, and
// 4 M N bytes per block.
// A row or a few of x (a token at a time) go to the FP32 units (lwc_few.cuh).
#include <algorithm>

#include "lwc_few.cuh"
#include "lwc_tc.cuh"

namespace lwc {
namespace {

using tc::Product;

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + exp(-v)): exp overflows to infinity below -88, which gives 0.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// act(v) and, where asked, its derivative.
template <bool kSlope>
__device__ __forceinline__ float activation(uint32_t act, float v, float &slope) {
    switch (act) {
        case LWC_ACT_SILU: {
            const float p = sigmoid(v);
            if (kSlope) slope = p * (1.0f + v * (1.0f - p));
            return v * p;
        }
        case LWC_ACT_GELU: {
            // Phi(v) from erfc: no cancellation for negative v
            const float c = 0.5f * erfcf(-kSqrtHalf * v);
            if (kSlope) slope = c + v * kInvSqrt2Pi * __expf(-0.5f * v * v);
            return v * c;
        }
        case LWC_ACT_GELU_TANH: {
            // 0.5 (1 + tanh q) = sigmoid(2 q); beyond |v| = 10^4 p is 0 or 1 anyway, but v^2 may be infinite
            const float v2 = fminf(v * v, 1e8f), q2 = 2.0f * kGeluC * v * (1.0f + kGeluA * v2), p = sigmoid(q2);
            if (kSlope) slope = p + v * p * (1.0f - p) * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * v2);
            return v * p;
        }
        case LWC_ACT_RELU:
            if (kSlope) slope = v > 0.0f ? 1.0f : 0.0f;
            return v <= 0.0f ? 0.0f : v;   // NaN stays NaN
        default: {
            const float p = sigmoid(v);
            if (kSlope) slope = p * (1.0f - p);
            return p;
        }
    }
}

struct GatedForward {
    struct Args {
        uint16_t *h;
        uint64_t ld;
        uint32_t rows, cols, act, wide, fp16;
    };
    __device__ __forceinline__ GatedForward(const Args &, const tc::Tile &) {}
    __device__ __forceinline__ void finish(const Args &, const tc::Tile &) {}
    __device__ __forceinline__ void take(const Args &E, const tc::Tile &t, bool) {
        const uint32_t half = t.n_tile / 2, n0 = t.n * half, end = min(E.cols, n0 + half);
        uint16_t *row = E.h + (uint64_t)t.row * E.ld;
        for (uint32_t c = 16 * t.side; n0 + c < end; c += 32) {
            uint32_t a[16], b[16];
            umma::tmem_ld16_async(t.taddr + c, a);
            umma::tmem_ld16_async(t.taddr + half + c, b);
            umma::tmem_wait_ld();
            if (t.row >= E.rows) continue;
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; j++) {
                float unused;
                v[j] = activation<false>(E.act, __uint_as_float(a[j]), unused) * __uint_as_float(b[j]);
            }
            tc::store_row(row, n0 + c, end, E.wide, E.fp16, v);
        }
    }
};

struct GatedSlopes {
    struct Args {
        const uint16_t *dh;
        uint16_t *da, *db;   // in panels
        uint64_t ld_dh;
        uint32_t rows, cols, padded, act, wide, fp16;   // padded: cols filled up to whole panels, with zeros
    };
    __device__ __forceinline__ GatedSlopes(const Args &, const tc::Tile &) {}
    __device__ __forceinline__ void finish(const Args &, const tc::Tile &) {}
    __device__ __forceinline__ void take(const Args &E, const tc::Tile &t, bool) {
        const uint32_t half = t.n_tile / 2, n0 = t.n * half, end = min(E.padded, n0 + half);
        const uint64_t row = t.row;
        for (uint32_t c = 16 * t.side; n0 + c < end; c += 32) {
            uint32_t a[16], b[16];
            umma::tmem_ld16_async(t.taddr + c, a);
            umma::tmem_ld16_async(t.taddr + half + c, b);
            umma::tmem_wait_ld();
            if (t.row >= E.rows) continue;
            float dh[16], da[16], db[16];
            // past the last column dh is read as 0, and a and b are: dA = dB = 0
            tc::load_row16(E.dh + row * E.ld_dh, n0 + c, E.cols, E.wide, E.fp16, dh);
#pragma unroll
            for (int j = 0; j < 16; j++) {
                float slope;
                const float y = activation<true>(E.act, __uint_as_float(a[j]), slope);
                da[j] = dh[j] * __uint_as_float(b[j]) * slope;
                db[j] = dh[j] * y;
            }
            tc::store_panel(E.da, E.rows, t.row, n0 + c, end, E.fp16, da);
            tc::store_panel(E.db, E.rows, t.row, n0 + c, end, E.fp16, db);
        }
    }
};

// kRows rows of x on the FP32 units (see lwc_few.cuh): `share` warps of a
// block take a feature's two rows, so that few features still fill the device;
// their sums are added in order.
template <int kRows>
__global__ void __launch_bounds__(few::kWarps * 32)
    gated_few_kernel(const lwc_gated g, uint16_t *__restrict__ h, uint64_t ld_h, uint32_t share) {
    __shared__ float sums[few::kWarps][2][kRows];
    tc::wait_for_stream();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, per = few::kWarps / share;
    const uint32_t slot = warp / share, part = warp % share;
    const bool fp16 = g.elem == LWC_ELEM_FP16;
    const uint16_t *x = static_cast<const uint16_t *>(g.x);
    for (uint64_t f0 = blockIdx.x * (uint64_t)per; f0 < g.features; f0 += gridDim.x * (uint64_t)per) {
        const uint64_t f = f0 + slot;
        float acc[2][kRows] = {};
        if (f < g.features) {
            const uint16_t *const w[2] = {static_cast<const uint16_t *>(g.gate) + f * g.ld_gate,
                                          static_cast<const uint16_t *>(g.up) + f * g.ld_up};
            few::dot_rows<2, kRows>(acc, w, x, g.ld_x, (uint32_t)g.tokens, g.hidden, part, share, fp16);
        }
        if (share > 1) {
            __syncthreads();   // the sums of the turn before have been read
            if (lane == 0)
#pragma unroll
                for (int r = 0; r < kRows; r++) {
                    sums[warp][0][r] = acc[0][r];
                    sums[warp][1][r] = acc[1][r];
                }
            __syncthreads();
            if (part == 0)
                for (uint32_t o = 1; o < share; o++)
#pragma unroll
                    for (int r = 0; r < kRows; r++) {
                        acc[0][r] += sums[warp + o][0][r];
                        acc[1][r] += sums[warp + o][1][r];
                    }
        }
        if (part == 0 && f < g.features) {
            float a = 0.0f, b = 0.0f, unused;
#pragma unroll
            for (int r = 0; r < kRows; r++)
                if (lane == (uint32_t)r) {
                    a = acc[0][r];
                    b = acc[1][r];
                }
            if (lane < (uint32_t)kRows) h[lane * ld_h + f] = (uint16_t)tc::pack2(activation<false>(g.act, a, unused) * b, 0.0f, fp16);
        }
    }
}

// h = act(a) * b of FP32 products held in memory (two fused linear layers).
__global__ void gated_product_kernel(const float *__restrict__ a, const float *__restrict__ b, uint64_t n,
                                     uint32_t act, uint32_t fp16, uint16_t *__restrict__ h) {
    for (uint64_t i = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x; i < n; i += (uint64_t)gridDim.x * blockDim.x) {
        float unused;
        h[i] = (uint16_t)tc::pack2(activation<false>(act, a[i], unused) * b[i], 0.0f, fp16);
    }
}

bool rows16(const void *p, uint64_t ld) { return aligned16(p) && ld % 8 == 0; }

lwc_status check(const lwc_gated *g) {
    if (!g) return fail(LWC_ERR_INVALID_ARG, "NULL problem");
    if (g->elem != LWC_ELEM_BF16 && g->elem != LWC_ELEM_FP16)
        return fail(LWC_ERR_UNSUPPORTED, "element type %u (BF16 and FP16 are taken)", g->elem);
    if (g->act > LWC_ACT_SIGMOID) return fail(LWC_ERR_INVALID_ARG, "unknown activation %u", g->act);
    if (g->features == 0 || g->hidden == 0) return fail(LWC_ERR_INVALID_ARG, "features and hidden must be at least 1");
    if (g->tokens > 0x7FFFFFFFull || g->features > 0x3FFFFFFFull || g->hidden > 0x7FFFFFFFull)
        return fail(LWC_ERR_UNSUPPORTED, "sizes above 2^31 - 1 (features: 2^30 - 1)");
    if (g->ld_x < g->hidden || g->ld_gate < g->hidden || g->ld_up < g->hidden)
        return fail(LWC_ERR_INVALID_ARG, "a row stride is below hidden");
    if (!g->gate || !g->up || (g->tokens && !g->x)) return fail(LWC_ERR_INVALID_ARG, "NULL device pointer");
    if (!rows16(g->gate, g->ld_gate) || !rows16(g->up, g->ld_up) || (g->tokens && !rows16(g->x, g->ld_x)))
        return fail(LWC_ERR_MISALIGNED, "x, gate and up need 16-byte aligned rows (base and 2 x row stride)");
    return LWC_OK;
}

lwc_status check_status(const uint32_t *d_status) {
    if (reinterpret_cast<uintptr_t>(d_status) & 3u)
        return fail(LWC_ERR_MISALIGNED, "status word must be 4-byte aligned");
    return LWC_OK;
}

Product both(const lwc_gated *g, uint32_t *d_status) {
    Product p;
    p.a[0] = {g->x, g->tokens, g->hidden, g->ld_x};
    p.b[0] = {g->gate, g->features, g->hidden, g->ld_gate};
    p.b[1] = {g->up, g->features, g->hidden, g->ld_up};
    p.b_pick = tc::kHalves;
    p.m = g->tokens;
    p.n = g->features;
    p.k = g->hidden;
    p.fp16 = g->elem == LWC_ELEM_FP16;
    p.status = d_status;
    return p;
}

// Backward workspace: dA and dB, x transposed (all in panels), then the parts
// of split products.
struct BackwardPlan {
    uint64_t d_bytes, xt_bytes, part_bytes, total;
    Product dx, dw;
};

lwc_status plan_backward(const lwc_gated *g, const void *d_work, uint32_t *d_status, bool want_dx, uint32_t n_dw,
                         BackwardPlan &b) {
    b.d_bytes = round_up(tc::panel_bytes(g->tokens, g->features), 256);
    b.xt_bytes = n_dw ? round_up(tc::panel_bytes(g->hidden, g->tokens), 256) : 0;
    const uint8_t *da = static_cast<const uint8_t *>(d_work), *db = da + b.d_bytes, *xt = db + b.d_bytes;
    const bool fp16 = g->elem == LWC_ELEM_FP16;
    b.part_bytes = 0;
    if (want_dx) {
        Product &p = b.dx;
        p = Product();
        p.a[0] = {da, g->tokens, g->features, 0};
        p.a[1] = {db, g->tokens, g->features, 0};
        p.b[0] = {g->gate, g->features, g->hidden, g->ld_gate};
        p.b[1] = {g->up, g->features, g->hidden, g->ld_up};
        p.a_pick = p.b_pick = tc::kSegments;
        p.b_mn = true;
        p.m = g->tokens;
        p.n = g->hidden;
        p.k = p.k2 = g->features;
        p.fp16 = fp16;
        p.status = d_status;
        const lwc_status st = tc::plan_product(p, true);
        if (st) return st;
        b.part_bytes = p.part_bytes;
    }
    if (n_dw) {
        Product &p = b.dw;
        p = Product();
        p.a[0] = {xt, g->hidden, g->tokens, 0};
        p.b[0] = {da, g->tokens, g->features, 0};
        p.b[1] = {db, g->tokens, g->features, 0};
        p.b_pick = tc::kBatch;
        p.b_mn = true;
        p.m = g->hidden;
        p.n = g->features;
        p.k = g->tokens;
        p.batch = n_dw;
        p.fp16 = fp16;
        p.status = d_status;
        const lwc_status st = tc::plan_product(p, true);
        if (st) return st;
        b.part_bytes = std::max(b.part_bytes, p.part_bytes);
    }
    b.part_bytes = round_up(b.part_bytes, 256);
    b.total = 2 * b.d_bytes + b.xt_bytes + b.part_bytes;
    return LWC_OK;
}

// Whether the FP32 units take a forward call: one row always, two to four where
// the matrices are small (the FP32 units' time grows with rows x weights, the
// tensor cores' hardly does). us on the FP32 units / the tensor cores, N x K: 1365
// x 512: 4.0 / 6.6 (1 row), 6.1 / 6.6 (4); 1365 x 4096: 6.2 / 20.5 (1), 9.3 / 20.5
// (4); 4096 x 4096: 10.6 / 20.7 (1), 17.5 / 20.7 (4); 14336 x 4096: 38.4 / 45.4 (1),
// 44.6 / 45.6 (2), 49.0 / 45.8 (3); 28672 x 8192: 142 / 150 (1), 165 / 153 (2).
bool is_few(const lwc_gated *g) {
    const uint64_t m = g->tokens;
    return m == 1 || (m <= 4 && m * m <= 300000000ull / g->features / g->hidden);
}

lwc_status launch_few(const lwc_gated *g, uint16_t *h, uint64_t ld_h, cudaStream_t s) {
    int sms = 0;
    lwc_status st = tc::device_sms(sms);
    if (st) return st;
    // warps of a feature: as many as it takes to give every SM 32 warps
    uint32_t share = 1;
    while (share < few::kWarps && g->features * share < 32ull * sms) share *= 2;
    const uint64_t per = few::kWarps / share, blocks = std::min<uint64_t>((g->features + per - 1) / per, sms * 8ull);
    const dim3 grid((unsigned)blocks);
    const uint32_t threads = few::kWarps * 32;
    const cudaError_t err =
        g->tokens == 1   ? tc::launch_next(gated_few_kernel<1>, grid, threads, 0, 1, s, *g, h, ld_h, share)
        : g->tokens == 2 ? tc::launch_next(gated_few_kernel<2>, grid, threads, 0, 1, s, *g, h, ld_h, share)
        : g->tokens == 3 ? tc::launch_next(gated_few_kernel<3>, grid, threads, 0, 1, s, *g, h, ld_h, share)
                         : tc::launch_next(gated_few_kernel<4>, grid, threads, 0, 1, s, *g, h, ld_h, share);
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "gated launch: %s", cudaGetErrorString(err));
    return LWC_OK;
}

lwc_status zero(void *p, uint64_t bytes, cudaStream_t s) {
    const cudaError_t err = cudaMemsetAsync(p, 0, bytes, s);
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "output fill: %s", cudaGetErrorString(err));
    return LWC_OK;
}

}  // namespace
}  // namespace lwc

using namespace lwc;

extern "C" {

lwc_status lwc_gated_forward(const lwc_gated *g, void *d_h, uint64_t ld_h, uint32_t *d_status, lwc_stream_t stream) {
    lwc_status st = check(g);
    if (!st) st = check_status(d_status);
    if (st) return st;
    if (ld_h < g->features) return fail(LWC_ERR_INVALID_ARG, "the row stride of h is below features");
    if (g->tokens == 0) {
        clear_error();
        return LWC_OK;
    }
    if (!d_h || (reinterpret_cast<uintptr_t>(d_h) & 1u)) return fail(LWC_ERR_INVALID_ARG, "h: NULL or odd device pointer");
    if (is_few(g)) {
        st = launch_few(g, static_cast<uint16_t *>(d_h), ld_h, reinterpret_cast<cudaStream_t>(stream));
        if (!st) clear_error();
        return st;
    }
    Product p = both(g, d_status);
    st = tc::plan_product(p, false);
    if (st) return st;
    GatedForward::Args e;
    e.h = static_cast<uint16_t *>(d_h);
    e.ld = ld_h;
    e.rows = (uint32_t)g->tokens;
    e.cols = (uint32_t)g->features;
    e.act = g->act;
    e.wide = rows16(d_h, ld_h);
    e.fp16 = p.fp16;
    st = tc::launch_product<GatedForward, false>(p, e, reinterpret_cast<cudaStream_t>(stream));
    if (st) return st;
    clear_error();
    return LWC_OK;
}

uint64_t lwc_gated_backward_workspace_bytes(const lwc_gated *g, int want_dx, int want_dgate, int want_dup) {
    if (check(g)) return 0;
    if (g->tokens == 0) return 0;
    BackwardPlan b;
    if (plan_backward(g, nullptr, nullptr, want_dx != 0, (want_dgate ? 1u : 0u) + (want_dup ? 1u : 0u), b)) return 0;
    clear_error();
    return b.total;
}

lwc_status lwc_gated_backward(const lwc_gated *g, const void *d_dh, uint64_t ld_dh, void *d_dx, void *d_dgate,
                              void *d_dup, void *d_work, uint64_t work_bytes, uint32_t *d_status,
                              lwc_stream_t stream) {
    lwc_status st = check(g);
    if (!st) st = check_status(d_status);
    if (st) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (ld_dh < g->features) return fail(LWC_ERR_INVALID_ARG, "the row stride of dh is below features");
    for (const void *p : {(const void *)d_dx, (const void *)d_dgate, (const void *)d_dup, d_dh})
        if (reinterpret_cast<uintptr_t>(p) & 1u) return fail(LWC_ERR_MISALIGNED, "odd device pointer");
    const uint64_t w_bytes = 2 * g->features * g->hidden;
    if (g->tokens == 0) {
        if (d_dgate) st = zero(d_dgate, w_bytes, s);
        if (!st && d_dup) st = zero(d_dup, w_bytes, s);
        if (!st) clear_error();
        return st;
    }
    if (!d_dh) return fail(LWC_ERR_INVALID_ARG, "dh: NULL device pointer");
    if (!d_dx && !d_dgate && !d_dup) {
        clear_error();
        return LWC_OK;
    }
    if (!d_work || (reinterpret_cast<uintptr_t>(d_work) & 255u))
        return fail(LWC_ERR_MISALIGNED, "the workspace must be 256-byte aligned");
    const uint32_t n_dw = (d_dgate ? 1u : 0u) + (d_dup ? 1u : 0u);
    BackwardPlan b;
    st = plan_backward(g, d_work, d_status, d_dx != nullptr, n_dw, b);
    if (st) return st;
    if (work_bytes < b.total)
        return fail(LWC_ERR_INVALID_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)work_bytes,
                    (unsigned long long)b.total);
    uint8_t *work = static_cast<uint8_t *>(d_work);
    const bool fp16 = g->elem == LWC_ELEM_FP16;

    Product p = both(g, d_status);
    p.n = round_up(p.n, 64);   // whole panels
    st = tc::plan_product(p, false);
    if (st) return st;
    GatedSlopes::Args e;
    e.dh = static_cast<const uint16_t *>(d_dh);
    e.da = reinterpret_cast<uint16_t *>(work);
    e.db = reinterpret_cast<uint16_t *>(work + b.d_bytes);
    e.ld_dh = ld_dh;
    e.rows = (uint32_t)g->tokens;
    e.cols = (uint32_t)g->features;
    e.act = g->act;
    e.wide = rows16(d_dh, ld_dh);
    e.fp16 = fp16;
    e.padded = (uint32_t)p.n;
    st = tc::launch_product<GatedSlopes, false>(p, e, s);
    if (st) return st;

    uint8_t *xt = work + 2 * b.d_bytes;
    tc::OutEpi::Args o = {};
    o.part = reinterpret_cast<float *>(xt + b.xt_bytes);
    o.ld = g->hidden;
    o.fp16 = fp16;
    if (d_dx) {
        o.out[0] = static_cast<uint16_t *>(d_dx);
        o.rows = (uint32_t)g->tokens;
        o.cols = (uint32_t)g->hidden;
        o.wide = rows16(d_dx, g->hidden);
        o.tile_rows = b.dx.tile_rows();
        st = tc::launch_product<tc::OutEpi, true>(b.dx, o, s);
        if (st) return st;
    }
    if (n_dw) {
        st = tc::launch_transpose(g->x, g->ld_x, g->tokens, g->hidden, nullptr, xt, s);
        if (st) return st;
        // one of the two alone: its own dA (or dB) as the only batch
        if (!d_dgate) b.dw.b[0] = b.dw.b[1];
        o.out[0] = static_cast<uint16_t *>(d_dgate ? d_dgate : d_dup);
        o.out[1] = static_cast<uint16_t *>(d_dup);
        o.rows = (uint32_t)g->hidden;
        o.cols = (uint32_t)g->features;
        o.transposed = 1;
        o.wide = rows16(o.out[0], g->hidden) && (n_dw < 2 || rows16(o.out[1], g->hidden));
        o.tile_rows = b.dw.tile_rows();
        st = tc::launch_product<tc::OutEpi, true>(b.dw, o, s);
        if (st) return st;
    }
    clear_error();
    return LWC_OK;
}

lwc_status lwc_gated_product(uint32_t elem, uint32_t act, const float *d_a, const float *d_b, uint64_t n, void *d_h,
                             lwc_stream_t stream) {
    if (elem != LWC_ELEM_BF16 && elem != LWC_ELEM_FP16)
        return fail(LWC_ERR_UNSUPPORTED, "element type %u (BF16 and FP16 are taken)", elem);
    if (act > LWC_ACT_SIGMOID) return fail(LWC_ERR_INVALID_ARG, "unknown activation %u", act);
    if (n == 0) {
        clear_error();
        return LWC_OK;
    }
    if (!d_a || !d_b || !d_h) return fail(LWC_ERR_INVALID_ARG, "NULL device pointer");
    if ((reinterpret_cast<uintptr_t>(d_a) | reinterpret_cast<uintptr_t>(d_b)) & 3u ||
        reinterpret_cast<uintptr_t>(d_h) & 1u)
        return fail(LWC_ERR_MISALIGNED, "a and b must be 4-byte aligned, h 2-byte aligned");
    const uint64_t blocks = std::min<uint64_t>((n + 255) / 256, 148 * 8);
    gated_product_kernel<<<(unsigned)blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        d_a, d_b, n, act, elem == LWC_ELEM_FP16, static_cast<uint16_t *>(d_h));
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "gated product launch: %s", cudaGetErrorString(err));
    clear_error();
    return LWC_OK;
}

}  // extern "C"
