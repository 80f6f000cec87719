// Host side of the dense product core (lwc_tc.cuh): tile and split choice,
// tensor maps, and the kernel that joins the parts of a split contraction.
#include <algorithm>
#include <mutex>
#include <vector>

#include "lwc_tc.cuh"

namespace lwc {
namespace tc {
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Device {
    int sms = 0, max_smem = 0;
    bool ready = false;
};
std::mutex g_mutex;
std::vector<Device> g_dev;
EncodeTiledFn g_encode = nullptr;

lwc_status device(Device &out, bool bind = false) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    // binds the device's context to this host thread, which may have made no
    // CUDA call yet (an autograd worker): the tensor map calls need one
    if (err == cudaSuccess && bind) err = cudaSetDevice(dev);
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "current device: %s", cudaGetErrorString(err));
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (err != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
            return fail(LWC_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
        g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    if ((int)g_dev.size() <= dev) g_dev.resize(dev + 1);
    Device &c = g_dev[dev];
    if (!c.ready) {
        int major = 0;
        err = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (err == cudaSuccess && major != 10)
            return fail(LWC_ERR_UNSUPPORTED, "the tensor-core product needs an sm_100 device (compute capability %d.x)",
                        major);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, dev);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&c.max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "device setup: %s", cudaGetErrorString(err));
        c.ready = true;
    }
    out = c;
    return LWC_OK;
}

// Bytes of one operand that are counted on to stay in L2 (126 MB in all).
constexpr uint64_t kResidentBytes = 56ull << 20;

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// blocks: columns are indexed by 64s (the third index), `boxed` of them a copy.
lwc_status encode_map(CUtensorMap *map, bool fp16, const Matrix &m, uint32_t box_outer, bool blocks, uint32_t boxed) {
    const uint64_t ld = m.ld ? m.ld : 64, n_blocks = ceil_div(m.cols, 64);
    const cuuint64_t gdim[3] = {blocks ? 64 : m.cols, m.rows, blocks ? n_blocks : 1};
    const cuuint64_t gstride[2] = {ld * 2, m.ld ? 128 : m.rows * 128};
    const cuuint32_t box[3] = {64, box_outer, boxed};
    const cuuint32_t estride[3] = {1, 1, 1};
    const CUresult r = g_encode(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                                const_cast<void *>(m.p), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(LWC_ERR_CUDA, "tensor map: driver error %d", (int)r);
    return LWC_OK;
}

// Joins the parts of the split tiles: adds them in ascending order, so that a
// result repeats bit for bit, and hands the sum to the epilogue's own ending.
// One block per 8 columns of a tile, a thread per row.
__global__ void join_kernel(const __grid_constant__ TcArgs P, const __grid_constant__ OutEpi::Args E) {
    wait_for_stream();
    const uint32_t rows = blockDim.x, local = threadIdx.x, c = blockIdx.x * 8;
    const uint32_t index = blockIdx.y, splits = P.splits;
    const Unit t = unit_of(P, P.whole + index * splits);
    const float *part = E.part + ((uint64_t)index * splits * P.n_tile + c) * rows + local;
    float v[8] = {};
    for (uint32_t k = 0; k < splits; k++)
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) v[j] += part[((uint64_t)k * P.n_tile + j) * rows];
    OutEpi::end<8>(E, v, t.batch, t.m * rows + local, t.n * P.n_tile + c,
                   ((uint64_t)t.tile * P.n_tile + c) * rows + local, rows);
}

}  // namespace

lwc_status device_sms(int &sms) {
    Device d;
    const lwc_status st = device(d);
    sms = d.sms;
    return st;
}

lwc_status plan_product(Product &p, bool may_split) {
    Device d;
    const lwc_status st = device(d);
    if (st) return st;
    const bool halves = p.b_pick == kHalves;
    // More than one tile of rows: CTA pairs, 256 rows a tile. Their tiles take
    // half the bytes from L2 for the same products.
    p.pair = p.m > kRows;
    const uint32_t ctas = p.pair ? 2 : 1;
    const uint64_t workers = (uint64_t)d.sms / ctas;
    const uint64_t m_tiles = ceil_div(p.m, kRows * ctas);
    // widths the MMA and the operand boxes take
    const uint32_t unit = p.b_mn ? 64u * ctas : 16u * ctas;
    const uint64_t steps = ceil_div(p.k, kStepK) + (p.a_pick == kSegments ? ceil_div(p.k2, kStepK) : 0);
    // Tiles are walked in waves of one per worker, and the last wave is rarely full.
    // Where parts of a contraction may be joined afterwards, its tiles (all tiles,
    // if there is no full wave) may be split into s parts that fill it better.
    // Cycles of a step of a tile: its MMAs (2 a column) and what narrower tiles load
    // more often; no less than the copies take to come round, whatever their size
    // (1000 x 2048 x 32003 in tiles of 128 columns: 530). The joining costs about
    // 10000 cycles and the parts' traffic. A tile's epilogue, 30 cycles a column and
    // 1500, runs under the next tile's products if those take as long, the last
    // tile's under nothing. With one tile of rows, B's way from memory is what
    // counts: as even a share of it for every worker as there is, in wide tiles
    // (32000 x 2048, 9 rows: 31 us as one wave of 224 columns, 52 us as two of 112).
    const bool few = m_tiles == 1;
    auto step = [&](uint32_t w) { return few ? w + 24.0 : std::max(500.0, 2.0 * w + 160.0); };
    double best = 0.0;
    uint64_t units = 0, rest = 0;
    p.n_tile = 0;
    for (uint32_t w = unit; w <= kMaxCols; w += unit) {
        if (p.width && w != p.width) continue;
        const uint64_t n_tiles = ceil_div(p.n, halves ? w / 2 : w), tiles = m_tiles * n_tiles * p.batch;
        const uint64_t over = tiles % workers;
        const double end = few ? 0.0 : 30.0 * w + 1500.0, wave = std::max((double)steps * step(w), end);
        const double full = (double)(tiles / workers) * wave + end;
        double least = full + (over ? wave : 0.0);
        uint32_t splits = 1;
        for (uint64_t s = 2; may_split && !few && over && s <= 32 && s * 8 <= steps; s++) {
            const double cost = full + (double)ceil_div(over * s, workers) / (double)s * wave + 10000.0 +
                                (double)(over * s * w * kRows * ctas) / 300.0;
            if (cost < least) {
                least = cost;
                splits = (uint32_t)s;
            }
        }
        if (!p.n_tile || least <= best) {
            best = least;
            p.n_tile = w;
            p.n_tiles = (uint32_t)n_tiles;
            p.splits = splits;
            units = tiles;
            rest = over;
        }
    }
    if (may_split && few && rest) {
        // more parts have to be worth their traffic (a fifth), all of it the joining
        double least = 1.0;
        for (uint64_t s = 2; s <= 32 && s * 8 <= steps; s++) {
            const double wave = (double)ceil_div(rest * s, workers) / (double)s;
            if (wave < 0.8 * least) {
                least = wave;
                p.splits = (uint32_t)s;
            }
        }
        if ((1.0 - least) * (double)steps * (2.0 * p.n_tile + 100.0) < 10000.0) p.splits = 1;
    }
    // no part may be empty
    if (p.splits > 1) p.splits = (uint32_t)ceil_div(steps, ceil_div(steps, p.splits));
    p.whole = p.splits > 1 ? units - rest : units;
    p.part_bytes = p.splits > 1 ? 4 * rest * p.splits * p.n_tile * kRows * ctas : 0;
    p.acc_bytes = 4 * units * p.n_tile * kRows * ctas;
    if (m_tiles * p.n_tiles * (uint64_t)p.batch * p.splits > 0xFFFFFFFFull || p.m > 0x7FFFFFFFull || p.n > 0x7FFFFFFFull ||
        p.k > 0x7FFFFFFFull || p.k2 > 0x7FFFFFFFull)
        return fail(LWC_ERR_UNSUPPORTED, "sizes above 2^31 - 1");
    return LWC_OK;
}

lwc_status marshal_product(const Product &p, TcArgs &P, uint32_t &grid, uint32_t &smem) {
    Device d;
    lwc_status st = device(d, true);
    if (st) return st;
    const bool halves = p.b_pick == kHalves;
    const uint32_t ctas = p.pair ? 2 : 1;
    const uint32_t a_box = p.pair ? kRows : (uint32_t)std::min<uint64_t>(kRows, round_up(p.m, 8));
    const uint32_t w = p.n_tile / ctas;
    const uint32_t b_box = p.b_mn ? 64 : halves ? p.n_tile / 2 : w;
    // Blocks of 64 columns as an index of their own: in panels, and in rows that
    // are whole blocks, where an MN-major stage is then one copy instead of one a
    // block (gradients of 4001 x 14336 x 4096: 2.29 ms with two, 2.22 with one).
    const bool whole_b = p.b_mn && p.b[0].cols % 64 == 0 && (p.b_pick == kOne || p.b[1].cols % 64 == 0);
    P.a_panels = p.a[0].ld == 0;
    P.b_panels = p.b[0].ld == 0 || whole_b;
    const uint32_t boxed = p.b_mn && P.b_panels ? w / 64 : 1;
    P.b_boxes = p.b_mn ? w / 64 / boxed : 1;
    for (uint32_t i = 0; i < 2 && !st; i++) {
        if (i == 0 || p.a_pick != kOne) st = encode_map(&P.a[i], p.fp16, p.a[i], a_box, P.a_panels, 1);
        else P.a[i] = P.a[0];
        if (st) break;
        if (i == 0 || p.b_pick != kOne) st = encode_map(&P.b[i], p.fp16, p.b[i], b_box, P.b_panels, boxed);
        else P.b[i] = P.b[0];
    }
    if (st) return st;
    P.a_pick = p.a_pick;
    P.b_pick = p.b_pick;
    P.m_tiles = (uint32_t)ceil_div(p.m, kRows * ctas);
    P.n_tiles = p.n_tiles;
    P.batch = p.batch;
    P.splits = p.splits;
    P.n_tile = p.n_tile;
    P.steps0 = (uint32_t)ceil_div(p.k, kStepK);
    P.steps = P.steps0 + (p.a_pick == kSegments ? (uint32_t)ceil_div(p.k2, kStepK) : 0u);
    P.steps_per_split = (uint32_t)ceil_div(P.steps, p.splits);
    P.chunk = p.chunk ? p.chunk : P.steps;
    // m tiles walked together: all of them where A stays in L2 while B, which does
    // not, is read once (4096 tokens' losses over 128256 words, 33 MB of A in 16 m
    // tiles: 3.72, 3.55, 3.54, 3.59, 3.62 and 3.40 ms for groups of 2, 4, 6, 8, 12 and
    // 16; the gated product of 13, 16, 20 and 24 m tiles by 14336 x 4096 takes the same
    // time, within 1 %, for 7, 8, 10, 12 and all); else as many as make the tiles that
    // run at a time about square.
    const uint64_t a_bytes = 2 * p.m * (p.k + p.k2), b_bytes = 2 * p.n * (p.k + p.k2) * (halves ? 2 : 1);
    const bool resident = a_bytes <= kResidentBytes && b_bytes > kResidentBytes;
    P.group = resident ? P.m_tiles : std::min<uint32_t>(P.m_tiles, 8);
    P.whole = (uint32_t)p.whole;
    P.units = P.whole + (P.m_tiles * P.n_tiles * p.batch - P.whole) * p.splits;
    P.stage_bytes = kABytes + w * 128u;
    // a pair's barrier counts the bytes of both CTAs
    P.tx_bytes = ctas * (a_box + w) * 128u;
    // 1 KB for alignment
    P.stages = std::min<uint32_t>(kMaxStages, ((uint32_t)d.max_smem - kCtlBytes - 1024u) / P.stage_bytes);
    P.idesc = umma::instr_desc_f16(p.fp16, false, p.b_mn, kRows * ctas, p.n_tile);
    P.status = p.status;
    grid = ctas * std::min<uint32_t>(P.units, (uint32_t)d.sms / ctas);
    smem = P.stages * P.stage_bytes + kCtlBytes + 1024u;
    return LWC_OK;
}

lwc_status allow_smem(const void *kernel, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (err == cudaSuccess && (done.load(std::memory_order_acquire) & bit)) return LWC_OK;
    Device d;
    const lwc_status st = device(d);
    if (st) return st;
    if (err == cudaSuccess) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, d.max_smem);
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "device setup: %s", cudaGetErrorString(err));
    done.fetch_or(bit, std::memory_order_release);
    return LWC_OK;
}

lwc_status launch_join(const TcArgs &args, const OutEpi::Args &e, bool pair, cudaStream_t s) {
    const uint32_t tiles = (args.units - args.whole) / args.splits;
    const cudaError_t err =
        launch_next(join_kernel, dim3(args.n_tile / 8, tiles), kRows * (pair ? 2 : 1), 0, 1, s, args, e);
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "join launch: %s", cudaGetErrorString(err));
    return LWC_OK;
}

// One 64 x 64 tile a block, through shared memory in 4-byte words; a tile of
// dst is 8 KB of one panel.
__global__ void transpose_kernel(const uint16_t *__restrict__ src, uint64_t ld_src, uint64_t rows, uint64_t cols,
                                 const float *__restrict__ keep, uint16_t *__restrict__ dst) {
    __shared__ uint16_t tile[64][66];
    wait_for_stream();
    const uint64_t r0 = blockIdx.x * 64ull, c0 = blockIdx.y * 64ull;
    for (uint32_t i = threadIdx.x; i < 64 * 8; i += blockDim.x) {
        const uint32_t r = i >> 3, c = (i & 7u) * 8;
        uint32_t w[4] = {0, 0, 0, 0};
        if (r0 + r < rows && !(keep && keep[r0 + r] == 0.0f)) {
            const uint16_t *p = src + (r0 + r) * ld_src + c0 + c;
            if (c0 + c + 8 <= cols) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
                for (uint32_t j = 0; j < 8; j++)
                    if (c0 + c + j < cols) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1u));
            }
        }
        for (uint32_t j = 0; j < 4; j++) *reinterpret_cast<uint32_t *>(&tile[r][c + 2 * j]) = w[j];
    }
    __syncthreads();
    // rows past the last one fill up the panel with zeros
    uint16_t *out = dst + panel_at(cols, c0, r0);
    for (uint32_t i = threadIdx.x; i < 64 * 8; i += blockDim.x) {
        const uint32_t c = i >> 3, r = (i & 7u) * 8;
        if (c0 + c >= cols) continue;
        uint32_t w[4];
        for (uint32_t j = 0; j < 4; j++) w[j] = tile[r + 2 * j][c] | (uint32_t)tile[r + 2 * j + 1][c] << 16;
        dev::st_v4(out + c * 64 + r, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

lwc_status launch_transpose(const void *src, uint64_t ld_src, uint64_t rows, uint64_t cols, const float *keep,
                            void *dst, cudaStream_t s) {
    if (ceil_div(cols, 64) > 65535) return fail(LWC_ERR_UNSUPPORTED, "hidden above 4194240");
    const cudaError_t err =
        launch_next(transpose_kernel, dim3((unsigned)ceil_div(rows, 64), (unsigned)ceil_div(cols, 64)), 256, 0, 1, s,
                    static_cast<const uint16_t *>(src), ld_src, rows, cols, keep, static_cast<uint16_t *>(dst));
    if (err != cudaSuccess) return fail(LWC_ERR_CUDA, "transpose launch: %s", cudaGetErrorString(err));
    return LWC_OK;
}

}  // namespace tc
}  // namespace lwc
