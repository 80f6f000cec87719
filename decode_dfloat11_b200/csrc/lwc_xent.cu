// Softmax cross entropy over a large vocabulary, straight from hidden states
// and the output matrix, without ever keeping the logits:
//
//   z = x W^T,  lse_i = log sum_v exp z_iv,  l_i = lse_i - z_i,t(i)
//   P_iv = c_i (exp(z_iv - lse_i) - [v = t(i)]),  dx = P W,  dW = P^T x
//
// (x: M x K, W: V x K; c_i: the gradient of l_i.) Forward: a product kernel
// whose epilogue keeps, per token and vocabulary tile, the largest logit and
// the sum of exponentials under it, both of the words that are not the target,
// and the target's logit; a second kernel joins the tiles. Backward: the
// vocabulary goes piece by piece; a piece's logits are computed again, by the
// same sums, turned into P (16 bits) by the epilogue, and used at once by two
// products, dW's rows of the piece and dx (summed over the pieces in 32 bits).
//
// A token that is sure of its target has a loss and a p - 1 far below the
// rounding of lse or of p, so neither is a difference of those: with R the
// other words' sum of exp(z_v - z_t), the loss is log(1 + R) by log1p, and the
// target's entry of P is c expm1(-loss). (Off by some 10^-4 in p - 1 at
// K = 4096 as exp(z_t - lse) - 1 of two unlike sums, by the product's own
// relative error this way.)
//
// A token whose target is ignore_index bears no loss and passes no gradient,
// whatever its hidden state holds: its rows of P and of the x that dW reads
// are zeros. A token or a few are scored on the FP32 units (lwc_few.cuh).
#include <algorithm>
#include <initializer_list>

#include "lwc_few.cuh"
#include "lwc_tc.cuh"

namespace lwc {
namespace {

using tc::Product;

constexpr float kLog2e = 1.4426950408889634f;
// P in FP16 is scaled by this power of two: |P| <= 1 before (but for roundings), so nothing
// overflows, and a probability is kept to full precision down to 4e-9 (without
// it a uniform distribution over 128256 words would be subnormal).
constexpr float kFp16Scale = 16384.0f;
// Bytes of P per piece of the vocabulary. Gradients of 4096 tokens x 128256 words
// x 4096: 11.7, 10.9, 10.4, 10.1 and 10.0 ms for 48, 96, 192, 384 and 800 MB (each
// piece adds to dx in 32 bits and ends in incomplete waves of tiles).
constexpr uint64_t kPieceBytes = 384ull << 20;

// 2^v, off by at most 2^-22 of it; 0 below 2^-126.
__device__ __forceinline__ float pow2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The target's column, or -1 where it is ignored, or -2 where it is no column.
__device__ __forceinline__ int64_t target_of(int64_t t, int64_t ignore, uint64_t vocab) {
    if (t == ignore) return -1;
    return t >= 0 && (uint64_t)t < vocab ? t : -2;
}

// The tensor cores' FP32 sums are cut off rather than rounded, always towards
// zero, so a long sum drifts: 3e-6 of the loss at K = 4096. The logits are
// therefore summed a chunk of 64-term steps at a time and the parts added,
// rounded, in registers (16 columns of 8 chunks a thread). 8 steps leave
// 3.5e-7; 4 steps would leave two thirds of it, but take 2.26 ms instead of 1.55
// where the products bound the time (2048 tokens x 128256 words; 1.36 in one
// run, with eight times the error), and nothing for few rows, where W's way from
// memory does. Backward, 4096 tokens: 10.9, 9.65 and 9.46 ms for 4, 8 and one run.
constexpr uint32_t kChunkSteps = 8, kChunkStepsFewRows = 4;
uint32_t chunk_steps(uint64_t tokens) { return tokens > tc::kRows ? kChunkSteps : kChunkStepsFewRows; }

// A thread's logits of a tile: its row, the columns 32 i + 16 side + j.
struct Logits {
    float z[8][16];
    __device__ __forceinline__ Logits() {
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 16; j++) z[i][j] = 0.0f;
    }
    // adds an accumulator
    __device__ __forceinline__ void add(const tc::Tile &t) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t c = 32 * i + 16 * t.side;
            if (c < t.n_tile) {
                uint32_t raw[16];
                umma::tmem_ld16(t.taddr + c, raw);
#pragma unroll
                for (int j = 0; j < 16; j++) z[i][j] += __uint_as_float(raw[j]);
            }
        }
    }
};

struct XentStats : Logits {
    struct Args {
        float2 *part;   // rows x 2 n_tiles: (largest logit, sum of exp under it), without the target
        float *zt;      // the target's logit
        const int64_t *targets;
        int64_t ignore;
        uint32_t rows, cols, n_tiles;
    };
    __device__ __forceinline__ XentStats(const Args &, const tc::Tile &) {}
    __device__ __forceinline__ void take(const Args &, const tc::Tile &t, bool) { add(t); }
    __device__ __forceinline__ void finish(const Args &E, const tc::Tile &t) {
        if (t.row >= E.rows) return;
        const uint32_t n0 = t.n * t.n_tile, width = min(t.n_tile, E.cols - n0);
        const int64_t tgt = target_of(E.targets[t.row], E.ignore, E.cols);
        const uint32_t at = tgt >= (int64_t)n0 && tgt < (int64_t)(n0 + width) ? (uint32_t)(tgt - n0) : 0xFFFFFFFFu;
        float z_t = 0.0f;
        // four maxima and sums, so that no addition waits for the one before it
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, sum[4] = {};
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const uint32_t c = 32 * i + 16 * t.side + j;
                if (c == at) z_t = z[i][j];
                if (c >= width || c == at) z[i][j] = -INFINITY;
                top[j & 3] = fmaxf(top[j & 3], z[i][j]);
            }
        if (at != 0xFFFFFFFFu && ((at >> 4) & 1u) == t.side) E.zt[t.row] = z_t;
        const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // nothing but -infinity: any finite base gives a sum of 0
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 16; j++) sum[j & 3] += pow2((z[i][j] - base) * kLog2e);
        const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        E.part[((uint64_t)t.row * E.n_tiles + t.n) * 2 + t.side] = make_float2(m, s);
    }
};

struct XentGrad : Logits {
    struct Args {
        const float *lse, *loss, *coef;
        const int64_t *targets;
        uint16_t *p;    // rows x cols, in panels
        int64_t first;  // the piece's first column of the vocabulary
        uint32_t rows, cols, padded, fp16;   // padded: cols filled up to whole panels, with zeros
    };
    __device__ __forceinline__ XentGrad(const Args &, const tc::Tile &) {}
    __device__ __forceinline__ void take(const Args &, const tc::Tile &t, bool) { add(t); }
    __device__ __forceinline__ void finish(const Args &E, const tc::Tile &t) {
        if (t.row >= E.rows) return;
        const uint32_t n0 = t.n * t.n_tile, end = min(E.padded, n0 + t.n_tile);
        const float c_i = E.coef[t.row], lse = E.lse[t.row], hot = expm1f(-E.loss[t.row]);
        const int64_t at = E.targets[t.row] - E.first;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t c = n0 + 32 * i + 16 * t.side;
            if (c >= end) break;
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const float p = at == (int64_t)(c + j) ? hot : pow2((z[i][j] - lse) * kLog2e);
                v[j] = c_i == 0.0f || c + j >= E.cols ? 0.0f : p * c_i;
            }
            tc::store_panel(E.p, E.rows, t.row, c, end, E.fp16, v);
        }
    }
};

// The statistics of kRows tokens on the FP32 units (see lwc_few.cuh): a
// warp takes every so-many-th word; lane r keeps token r's largest logit and
// sum. One part per token and block.
template <int kRows>
__global__ void __launch_bounds__(few::kWarps * 32)
    xent_few_kernel(const lwc_xent x, float2 *__restrict__ part, float *__restrict__ zt) {
    __shared__ float2 sums[few::kWarps][kRows];
    tc::wait_for_stream();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
    constexpr uint32_t rows = kRows;
    const bool fp16 = x.elem == LWC_ELEM_FP16;
    const int64_t target = lane < rows ? target_of(x.targets[lane], x.ignore_index, x.vocab) : -1;
    float m = -INFINITY, s = 0.0f;
    const uint64_t warps = gridDim.x * (uint64_t)few::kWarps;
    // two words at a time, for twice the bytes in flight (past the last one: itself again, not counted)
    for (uint64_t v = blockIdx.x * (uint64_t)few::kWarps + warp; v < x.vocab; v += 2 * warps) {
        const uint64_t v2 = v + warps < x.vocab ? v + warps : v;
        const uint16_t *head = static_cast<const uint16_t *>(x.head);
        const uint16_t *const w[2] = {head + v * x.ld_head, head + v2 * x.ld_head};
        float acc[2][kRows] = {}, z[2] = {0.0f, 0.0f};
        few::dot_rows<2, kRows>(acc, w, static_cast<const uint16_t *>(x.x), x.ld_x, (uint32_t)x.tokens, x.hidden, 0, 1, fp16);
#pragma unroll
        for (int r = 0; r < kRows; r++)
            if (lane == (uint32_t)r) {
                z[0] = acc[0][r];
                z[1] = v2 != v ? acc[1][r] : -INFINITY;
            }
        if (lane < rows && target == (int64_t)v) {
            zt[lane] = z[0];
            z[0] = -INFINITY;
        }
        if (lane < rows && v2 != v && target == (int64_t)v2) {
            zt[lane] = z[1];
            z[1] = -INFINITY;
        }
        const float top = fmaxf(m, fmaxf(z[0], z[1])), base = top == -INFINITY ? 0.0f : top;
        s = s * pow2((m - base) * kLog2e) + pow2((z[0] - base) * kLog2e) + pow2((z[1] - base) * kLog2e);
        m = top;
    }
    if (lane < kRows) sums[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp == 0 && lane < rows) {
        for (uint32_t o = 1; o < few::kWarps; o++) {
            const float2 v = sums[o][lane];
            const float top = fmaxf(m, v.x), base = top == -INFINITY ? 0.0f : top;
            s = s * exp2f((m - base) * kLog2e) + v.y * exp2f((v.x - base) * kLog2e);
            m = top;
        }
        part[(uint64_t)lane * gridDim.x + blockIdx.x] = make_float2(m, s);
    }
}

// One warp per token: joins the maxima and sums of the vocabulary's parts.
__global__ void xent_join_kernel(const float2 *__restrict__ part, uint32_t parts, const float *__restrict__ zt,
                                 const int64_t *__restrict__ targets, int64_t ignore, uint64_t rows, uint64_t vocab,
                                 float *__restrict__ loss, float *__restrict__ lse, uint32_t *status) {
    tc::wait_for_stream();
    const uint32_t lane = threadIdx.x & 31u;
    const uint64_t warps = (uint64_t)gridDim.x * (blockDim.x >> 5);
    for (uint64_t row = blockIdx.x * (uint64_t)(blockDim.x >> 5) + (threadIdx.x >> 5); row < rows; row += warps) {
        const float2 *p = part + row * parts;
        float m = -INFINITY, s = 0.0f;
        for (uint32_t i = lane; i < parts; i += 32) {
            const float2 v = p[i];
            const float top = fmaxf(m, v.x), base = top == -INFINITY ? 0.0f : top;
            s = s * expf(m - base) + v.y * expf(v.x - base);
            m = top;
        }
        for (uint32_t d = 16; d; d >>= 1) {
            const float om = __shfl_xor_sync(0xFFFFFFFFu, m, d), os = __shfl_xor_sync(0xFFFFFFFFu, s, d);
            const float top = fmaxf(m, om), base = top == -INFINITY ? 0.0f : top;
            s = s * expf(m - base) + os * expf(om - base);
            m = top;
        }
        if (lane == 0) {
            const int64_t t = target_of(targets[row], ignore, vocab);
            const float z_t = t >= 0 ? zt[row] : -INFINITY;
            const float top = fmaxf(m, z_t), base = top == -INFINITY ? 0.0f : top;
            const float l = base + logf(s * expf(m - base) + (t >= 0 ? expf(z_t - base) : 0.0f));
            lse[row] = l;
            // from differences of logits: both are of one product, so their common part cancels exactly
            const float d = m - z_t;
            const float v = d <= 0.0f ? log1pf(s * expf(d)) : d + logf(s + expf(-d));
            loss[row] = t == -1 ? 0.0f : t == -2 || !isfinite(l) ? NAN : v;
            if (t == -2 && status) atomicOr(status, (uint32_t)LWC_DEVICE_BAD_TARGET);
        }
    }
}

// The sum of the losses and that over max(tokens that bear one, 1), where asked;
// one block, fixed order, sums in 64 bits.
__global__ void xent_total_kernel(const float *__restrict__ loss, const int64_t *__restrict__ targets, int64_t ignore,
                                  uint64_t rows, float *__restrict__ sum, float *__restrict__ mean) {
    __shared__ double sums[32];
    __shared__ unsigned long long counts[32];
    tc::wait_for_stream();
    double s = 0.0;
    unsigned long long n = 0;
    for (uint64_t i = threadIdx.x; i < rows; i += blockDim.x) {
        s += (double)loss[i];
        n += targets[i] != ignore;
    }
    for (uint32_t d = 16; d; d >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    }
    if ((threadIdx.x & 31u) == 0) {
        sums[threadIdx.x >> 5] = s;
        counts[threadIdx.x >> 5] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t w = 1; w < blockDim.x >> 5; w++) {
            s += sums[w];
            n += counts[w];
        }
        if (sum) *sum = (float)s;
        if (mean) *mean = (float)(s / (double)(n ? n : 1));
    }
}

// coef_i = c_i / unit (times kFp16Scale for FP16), alpha = unit (over it), with
// unit the largest entry of c P, c_i (1 - p_i) of one of the targets: P lies in
// [-1, 1] whatever the loss is divided by and however sure the tokens are, and
// the entry that weighs most, alone where there is one token, is not rounded
// (scaled by max |c| instead, one token's gradients were off by up to 2^-8 as a
// whole). At least 2^-64 of max |c|, so that coef stays finite.
// Only finite values count: an infinite or NaN gradient spoils its own token's
// row of dx (and dW), not the scale of the others.
// FP16: entries below 2^-28 of the largest are subnormal numbers (steps of
// 2^-38 of it): those of a token whose |c| is small, or whose tail is thin.
// One block.
__global__ void xent_coef_kernel(const float *__restrict__ grad, uint64_t grad_stride,
                                 const float *__restrict__ loss, const int64_t *__restrict__ targets, int64_t ignore,
                                 uint64_t rows, uint64_t vocab, uint32_t mean, uint32_t fp16, float *__restrict__ coef,
                                 float *__restrict__ alpha) {
    __shared__ float2 tops[32];
    __shared__ unsigned long long counts[32];
    tc::wait_for_stream();
    float2 top = {0.0f, 0.0f};   // of |c|, of the targets' entries
    unsigned long long n = 0;
    for (uint64_t i = threadIdx.x; i < rows; i += blockDim.x) {
        const int64_t t = target_of(targets[i], ignore, vocab);
        n += t != -1;
        const float c = t >= 0 ? fabsf(grad[i * grad_stride]) : 0.0f, e = t >= 0 ? -expm1f(-loss[i]) * c : 0.0f;
        if (isfinite(c)) top.x = fmaxf(top.x, c);
        if (isfinite(e)) top.y = fmaxf(top.y, e);
    }
    for (uint32_t d = 16; d; d >>= 1) {
        top.x = fmaxf(top.x, __shfl_xor_sync(0xFFFFFFFFu, top.x, d));
        top.y = fmaxf(top.y, __shfl_xor_sync(0xFFFFFFFFu, top.y, d));
        n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    }
    if ((threadIdx.x & 31u) == 0) {
        tops[threadIdx.x >> 5] = top;
        counts[threadIdx.x >> 5] = n;
    }
    __syncthreads();
    top = make_float2(0.0f, 0.0f);
    n = 0;
    for (uint32_t w = 0; w < blockDim.x >> 5; w++) {
        top.x = fmaxf(top.x, tops[w].x);
        top.y = fmaxf(top.y, tops[w].y);
        n += counts[w];
    }
    const float div = mean ? (float)(n ? n : 1) : 1.0f;
    const float most = fmaxf(top.y, top.x * 0x1p-64f) / div, unit = most > 0.0f ? most : 1.0f;
    const float scale = fp16 ? kFp16Scale : 1.0f;
    for (uint64_t i = threadIdx.x; i < rows; i += blockDim.x) {
        const bool on = target_of(targets[i], ignore, vocab) >= 0;
        coef[i] = on ? grad[i * grad_stride] / div / unit * scale : 0.0f;
    }
    if (threadIdx.x == 0) *alpha = unit / scale;
}

bool rows16(const void *p, uint64_t ld) { return aligned16(p) && ld % 8 == 0; }

lwc_status check(const lwc_xent *x) {
    if (!x) return fail(LWC_ERR_INVALID_ARG, "NULL problem");
    if (x->elem != LWC_ELEM_BF16 && x->elem != LWC_ELEM_FP16)
        return fail(LWC_ERR_UNSUPPORTED, "element type %u (BF16 and FP16 are taken)", x->elem);
    if (x->vocab == 0 || x->hidden == 0) return fail(LWC_ERR_INVALID_ARG, "vocab and hidden must be at least 1");
    if (x->tokens > 0x7FFFFFFFull || x->vocab > 0x7FFFFFFFull || x->hidden > 0x7FFFFFFFull)
        return fail(LWC_ERR_UNSUPPORTED, "sizes above 2^31 - 1");
    if (x->ld_x < x->hidden || x->ld_head < x->hidden)
        return fail(LWC_ERR_INVALID_ARG, "a row stride is below hidden");
    if (!x->head || (x->tokens && (!x->x || !x->targets))) return fail(LWC_ERR_INVALID_ARG, "NULL device pointer");
    if (!rows16(x->head, x->ld_head) || (x->tokens && !rows16(x->x, x->ld_x)))
        return fail(LWC_ERR_MISALIGNED, "x and head need 16-byte aligned rows (base and 2 x row stride)");
    if (reinterpret_cast<uintptr_t>(x->targets) & 7u) return fail(LWC_ERR_MISALIGNED, "targets must be 8-byte aligned");
    return LWC_OK;
}

lwc_status check_words(std::initializer_list<const float *> words, const uint32_t *d_status, const void *work) {
    for (const float *p : words)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(LWC_ERR_MISALIGNED, "FP32 arrays must be 4-byte aligned");
    if (reinterpret_cast<uintptr_t>(d_status) & 3u)
        return fail(LWC_ERR_MISALIGNED, "status word must be 4-byte aligned");
    if (!work || (reinterpret_cast<uintptr_t>(work) & 255u))
        return fail(LWC_ERR_MISALIGNED, "the workspace must be 256-byte aligned");
    return LWC_OK;
}

// Whether the FP32 units take a forward call (compare the gated block's rule).
// us on the FP32 units / the tensor cores, V x K: 1000 x 256: 4.3 / 14 (1 token),
// 4.8 / 14 (4); 32000 x 2048: 28 / 35 (1), 38 / 35 (2), 44 / 35 (4); 128256 x 4096:
// 163 / 172 (1), 215 / 177 (2).
bool is_few(const lwc_xent *x) {
    const uint64_t m = x->tokens;
    return m == 1 || (m <= 4 && m * m <= 200000000ull / x->vocab / x->hidden);
}

// Forward workspace: statistics of the vocabulary's parts, target logits.
struct ForwardPlan {
    Product z;
    uint32_t few_blocks = 0;   // on the FP32 units; else z
    uint64_t zt_off, total;
};

lwc_status plan_forward(const lwc_xent *x, uint32_t *d_status, ForwardPlan &f) {
    if (is_few(x)) {
        int sms = 0;
        const lwc_status st = tc::device_sms(sms);
        if (st) return st;
        f.few_blocks = (uint32_t)std::min<uint64_t>((x->vocab + few::kWarps - 1) / few::kWarps, 4ull * sms);
        f.zt_off = round_up(x->tokens * f.few_blocks * sizeof(float2), 256);
        f.total = f.zt_off + round_up(x->tokens * 4, 256);
        return LWC_OK;
    }
    Product &p = f.z;
    p = Product();
    p.a[0] = {x->x, x->tokens, x->hidden, x->ld_x};
    p.b[0] = {x->head, x->vocab, x->hidden, x->ld_head};
    p.m = x->tokens;
    p.n = x->vocab;
    p.k = x->hidden;
    p.fp16 = x->elem == LWC_ELEM_FP16;
    p.chunk = chunk_steps(x->tokens);
    p.status = d_status;
    const lwc_status st = tc::plan_product(p, false);
    if (st) return st;
    f.zt_off = round_up(x->tokens * p.n_tiles * 2 * sizeof(float2), 256);
    f.total = f.zt_off + round_up(x->tokens * 4, 256);
    return LWC_OK;
}

// Backward workspace: coef, the losses and lse of a forward pass (where the
// caller has no losses), alpha, x transposed (zeros where a token bears no
// loss), a piece of P (both in panels; before it, in its place, the forward
// pass's workspace), dx in FP32, parts of split products.
struct BackwardPlan {
    uint64_t piece;
    uint32_t dx_width = 0;   // the tiles of dx: the same for every piece, since they share its sum
    uint64_t loss_off, lse_off, alpha_off, xt_off, p_off, acc_off, part_off, total;
    ForwardPlan forward;
};

// One piece: columns first .. first + width - 1 of the vocabulary.
lwc_status plan_piece(const lwc_xent *x, const BackwardPlan &b, const uint8_t *work, uint64_t first, uint64_t width,
                      uint32_t *d_status, Product *z, Product *dw, Product *dx) {
    const bool fp16 = x->elem == LWC_ELEM_FP16;
    const void *head = static_cast<const uint16_t *>(x->head) + first * x->ld_head;
    const tc::Matrix w = {head, width, x->hidden, x->ld_head}, p = {work + b.p_off, x->tokens, width, 0};
    lwc_status st = LWC_OK;
    if (z) {
        *z = Product();
        z->a[0] = {x->x, x->tokens, x->hidden, x->ld_x};
        z->b[0] = w;
        z->m = x->tokens;
        z->n = round_up(width, 64);   // whole panels
        z->k = x->hidden;
        z->fp16 = fp16;
        z->chunk = chunk_steps(x->tokens);   // the forward pass's sums: what they are off by cancels in z - lse
        z->status = d_status;
        st = tc::plan_product(*z, false);
    }
    if (!st && dw) {
        *dw = Product();
        // its transpose, x^T P: a K-major A operand
        dw->a[0] = {work + b.xt_off, x->hidden, x->tokens, 0};
        dw->b[0] = p;
        dw->b_mn = true;
        dw->m = x->hidden;
        dw->n = width;
        dw->k = x->tokens;
        dw->fp16 = fp16;
        dw->status = d_status;
        st = tc::plan_product(*dw, true);
    }
    if (!st && dx) {
        *dx = Product();
        dx->a[0] = p;
        dx->b[0] = w;
        dx->b_mn = true;
        dx->m = x->tokens;
        dx->n = x->hidden;
        dx->k = width;
        dx->fp16 = fp16;
        dx->width = b.dx_width;
        dx->status = d_status;
        st = tc::plan_product(*dx, true);
    }
    return st;
}

lwc_status plan_backward(const lwc_xent *x, bool want_dx, bool want_dw, bool have_loss, BackwardPlan &b) {
    const uint64_t M = x->tokens, V = x->vocab, K = x->hidden;
    // pieces of equal width, a multiple of the widest tile
    const uint64_t pieces = std::max<uint64_t>(1, (2 * M * V + kPieceBytes - 1) / kPieceBytes);
    b.piece = std::min(V, round_up((V + pieces - 1) / pieces, tc::kMaxCols));
    lwc_status st = LWC_OK;
    b.forward.total = 0;
    b.loss_off = b.alpha_off = round_up(M * 4, 256);
    if (!have_loss) {
        st = plan_forward(x, nullptr, b.forward);
        if (st) return st;
        b.lse_off = 2 * b.loss_off;
        b.alpha_off = 3 * b.loss_off;
    }
    b.xt_off = b.alpha_off + 256;
    b.p_off = b.xt_off + (want_dw ? round_up(tc::panel_bytes(K, M), 256) : 0);
    b.acc_off = b.p_off + std::max(round_up(tc::panel_bytes(M, b.piece), 256), b.forward.total);
    uint64_t part = 0, acc = 0;
    // the widths that occur: a full piece and the last one
    for (const uint64_t width : {b.piece, V % b.piece}) {
        if (width == 0) break;
        Product dw, dx;
        st = plan_piece(x, b, nullptr, 0, width, nullptr, nullptr, want_dw ? &dw : nullptr, want_dx ? &dx : nullptr);
        if (st) return st;
        if (want_dw) part = std::max(part, dw.part_bytes);
        if (want_dx) part = std::max(part, dx.part_bytes);
        if (want_dx && b.piece < V) {
            b.dx_width = dx.n_tile;
            acc = dx.acc_bytes;
        }
    }
    b.part_off = b.acc_off + round_up(acc, 256);
    b.total = b.part_off + round_up(part, 256);
    return LWC_OK;
}

lwc_status launched(const char *what, cudaError_t err) {
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(err));
    return LWC_OK;
}

// The forward pass's launches; d_bad: where targets that are no words are reported, or NULL.
lwc_status run_forward(const lwc_xent *x, const ForwardPlan &f, float *d_loss, float *d_lse, float *d_sum,
                       float *d_mean, uint8_t *work, uint32_t *d_bad, cudaStream_t s) {
    float2 *part = reinterpret_cast<float2 *>(work);
    float *zt = reinterpret_cast<float *>(work + f.zt_off);
    uint32_t parts = f.few_blocks;
    lwc_status st = LWC_OK;
    if (f.few_blocks) {
        const dim3 grid(f.few_blocks);
        const uint32_t threads = few::kWarps * 32;
        st = launched("loss", x->tokens == 1   ? tc::launch_next(xent_few_kernel<1>, grid, threads, 0, 1, s, *x, part, zt)
                              : x->tokens == 2 ? tc::launch_next(xent_few_kernel<2>, grid, threads, 0, 1, s, *x, part, zt)
                              : x->tokens == 3 ? tc::launch_next(xent_few_kernel<3>, grid, threads, 0, 1, s, *x, part, zt)
                                               : tc::launch_next(xent_few_kernel<4>, grid, threads, 0, 1, s, *x, part, zt));
    } else {
        XentStats::Args e;
        e.part = part;
        e.zt = zt;
        e.targets = x->targets;
        e.ignore = x->ignore_index;
        e.rows = (uint32_t)x->tokens;
        e.cols = (uint32_t)x->vocab;
        e.n_tiles = f.z.n_tiles;
        parts = 2 * e.n_tiles;
        st = tc::launch_product<XentStats, false>(f.z, e, s);
    }
    if (st) return st;
    const uint64_t blocks = std::min<uint64_t>((x->tokens + 7) / 8, 148 * 8);
    st = launched("loss join",
                  tc::launch_next(xent_join_kernel, dim3((unsigned)blocks), 256, 0, 1, s, part, parts, zt,
                                  x->targets, x->ignore_index, x->tokens, x->vocab, d_loss, d_lse, d_bad));
    if (!st && (d_sum || d_mean))
        st = launched("loss total", tc::launch_next(xent_total_kernel, dim3(1), 1024, 0, 1, s, d_loss, x->targets,
                                                    x->ignore_index, x->tokens, d_sum, d_mean));
    return st;
}

// d_loss: the forward pass's losses, or NULL (computed again).
lwc_status backward(const lwc_xent *x, const float *d_lse, const float *d_loss, const float *d_grad,
                    uint64_t grad_stride, int mean, void *d_dx, void *d_dhead, void *d_work, uint64_t work_bytes,
                    uint32_t *d_status, cudaStream_t s) {
    lwc_status st = check(x);
    if (st) return st;
    if ((reinterpret_cast<uintptr_t>(d_dx) | reinterpret_cast<uintptr_t>(d_dhead)) & 1u)
        return fail(LWC_ERR_MISALIGNED, "odd device pointer");
    if (x->tokens == 0) {
        if (d_dhead) {
            const cudaError_t err = cudaMemsetAsync(d_dhead, 0, 2 * x->vocab * x->hidden, s);
            if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "output fill: %s", cudaGetErrorString(err));
        }
        clear_error();
        return LWC_OK;
    }
    if (!d_dx && !d_dhead) {
        clear_error();
        return LWC_OK;
    }
    if (!d_lse || !d_grad) return fail(LWC_ERR_INVALID_ARG, "NULL device pointer");
    st = check_words({d_lse, d_loss, d_grad}, d_status, d_work);
    if (st) return st;
    BackwardPlan b;
    st = plan_backward(x, d_dx != nullptr, d_dhead != nullptr, d_loss != nullptr, b);
    if (st) return st;
    if (work_bytes < b.total)
        return fail(LWC_ERR_INVALID_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)work_bytes,
                    (unsigned long long)b.total);
    uint8_t *work = static_cast<uint8_t *>(d_work);
    float *coef = reinterpret_cast<float *>(work), *alpha = reinterpret_cast<float *>(work + b.alpha_off);
    uint8_t *xt = work + b.xt_off;
    float *acc = reinterpret_cast<float *>(work + b.acc_off), *part = reinterpret_cast<float *>(work + b.part_off);
    const uint32_t fp16 = x->elem == LWC_ELEM_FP16;

    if (!d_loss) {
        float *loss = reinterpret_cast<float *>(work + b.loss_off);
        b.forward.z.status = d_status;
        st = run_forward(x, b.forward, loss, reinterpret_cast<float *>(work + b.lse_off), nullptr, nullptr,
                         work + b.p_off, nullptr, s);
        if (st) return st;
        d_loss = loss;
    }
    st = launched("loss coefficients",
                  tc::launch_next(xent_coef_kernel, dim3(1), 1024, 0, 1, s, d_grad, grad_stride, d_loss,
                                  x->targets, x->ignore_index, x->tokens, x->vocab, (uint32_t)(mean != 0), fp16, coef,
                                  alpha));
    if (!st && d_dhead) st = tc::launch_transpose(x->x, x->ld_x, x->tokens, x->hidden, coef, xt, s);
    for (uint64_t first = 0; first < x->vocab && !st; first += b.piece) {
        const uint64_t width = std::min(b.piece, x->vocab - first);
        Product z, dw, dx;
        st = plan_piece(x, b, work, first, width, d_status, &z, d_dhead ? &dw : nullptr, d_dx ? &dx : nullptr);
        if (st) break;
        XentGrad::Args e;
        e.lse = d_lse;
        e.loss = d_loss;
        e.coef = coef;
        e.targets = x->targets;
        e.p = reinterpret_cast<uint16_t *>(work + b.p_off);
        e.first = (int64_t)first;
        e.rows = (uint32_t)x->tokens;
        e.cols = (uint32_t)width;
        e.fp16 = fp16;
        e.padded = (uint32_t)z.n;
        st = tc::launch_product<XentGrad, false>(z, e, s);
        tc::OutEpi::Args o = {};
        o.part = part;
        o.alpha = alpha;
        o.ld = x->hidden;
        o.fp16 = fp16;
        if (!st && d_dhead) {
            o.out[0] = static_cast<uint16_t *>(d_dhead) + first * x->hidden;
            o.rows = (uint32_t)x->hidden;
            o.cols = (uint32_t)width;
            o.transposed = 1;
            o.wide = rows16(o.out[0], x->hidden);
            o.tile_rows = dw.tile_rows();
            st = tc::launch_product<tc::OutEpi, true>(dw, o, s);
        }
        if (!st && d_dx) {
            o.out[0] = static_cast<uint16_t *>(d_dx);
            o.rows = (uint32_t)x->tokens;
            o.cols = (uint32_t)x->hidden;
            o.wide = rows16(d_dx, x->hidden);
            o.transposed = 0;
            o.tile_rows = dx.tile_rows();
            o.acc = acc;
            o.add_in = first != 0;
            o.keep_acc = first + width < x->vocab;
            st = tc::launch_product<tc::OutEpi, true>(dx, o, s);
        }
    }
    if (st) return st;
    clear_error();
    return LWC_OK;
}

}  // namespace
}  // namespace lwc

using namespace lwc;

extern "C" {

uint64_t lwc_xent_forward_workspace_bytes(const lwc_xent *x) {
    ForwardPlan f;
    if (check(x) || x->tokens == 0 || plan_forward(x, nullptr, f)) return 0;
    clear_error();
    return f.total;
}

lwc_status lwc_xent_forward(const lwc_xent *x, float *d_loss, float *d_lse, float *d_sum, float *d_mean, void *d_work,
                            uint64_t work_bytes, uint32_t *d_status, lwc_stream_t stream) {
    lwc_status st = check(x);
    if (st) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (x->tokens == 0) {
        for (float *p : {d_sum, d_mean}) {
            const cudaError_t err = p ? cudaMemsetAsync(p, 0, sizeof(float), s) : cudaSuccess;
            if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "output fill: %s", cudaGetErrorString(err));
        }
        clear_error();
        return LWC_OK;
    }
    if (!d_loss || !d_lse) return fail(LWC_ERR_INVALID_ARG, "NULL device pointer");
    st = check_words({d_loss, d_lse, d_sum, d_mean}, d_status, d_work);
    if (st) return st;
    ForwardPlan f;
    st = plan_forward(x, d_status, f);
    if (st) return st;
    if (work_bytes < f.total)
        return fail(LWC_ERR_INVALID_ARG, "workspace of %llu bytes, %llu needed", (unsigned long long)work_bytes,
                    (unsigned long long)f.total);
    st = run_forward(x, f, d_loss, d_lse, d_sum, d_mean, static_cast<uint8_t *>(d_work), d_status, s);
    if (st) return st;
    clear_error();
    return LWC_OK;
}

uint64_t lwc_xent_backward_workspace_bytes(const lwc_xent *x, int want_dx, int want_dhead) {
    BackwardPlan b;
    if (check(x) || x->tokens == 0 || plan_backward(x, want_dx != 0, want_dhead != 0, false, b)) return 0;
    clear_error();
    return b.total;
}

lwc_status lwc_xent_backward(const lwc_xent *x, const float *d_lse, const float *d_grad, uint64_t grad_stride,
                             int mean, void *d_dx, void *d_dhead, void *d_work, uint64_t work_bytes,
                             uint32_t *d_status, lwc_stream_t stream) {
    return backward(x, d_lse, nullptr, d_grad, grad_stride, mean, d_dx, d_dhead, d_work, work_bytes, d_status,
                    reinterpret_cast<cudaStream_t>(stream));
}

lwc_status lwc_xent_backward_losses(const lwc_xent *x, const float *d_lse, const float *d_loss, const float *d_grad,
                                    uint64_t grad_stride, int mean, void *d_dx, void *d_dhead, void *d_work,
                                    uint64_t work_bytes, uint32_t *d_status, lwc_stream_t stream) {
    const lwc_status st = check(x);
    if (st) return st;
    if (x->tokens && (d_dx || d_dhead) && !d_loss) return fail(LWC_ERR_INVALID_ARG, "NULL device pointer");
    return backward(x, d_lse, d_loss, d_grad, grad_stride, mean, d_dx, d_dhead, d_work, work_bytes, d_status,
                    reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
