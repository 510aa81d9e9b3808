// ecc_gemm.cu -- the matrix products' launches: the shape of a launch, tensor
// maps, and the kernels of the plain linear operators (ecc_gemm.cuh).

#include <algorithm>
#include <cmath>

#include "ecc_gemm.cuh"

namespace ecc {

// ---------------------------------------------------------------- host side
namespace {

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled()
{
    static EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return (EncodeTiled)f;
    }();
    return fn;
}

CUtensorMapDataType map_type(uint32_t type)
{
    return type == ECC_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
           : type == ECC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}

// map of an operand: boxes of 128 bytes x `box_rows`
bool make_map(CUtensorMap *map, const Operand &o, uint64_t rows, uint64_t K, uint32_t type, uint32_t box_rows)
{
    const uint32_t size = type_bytes(type);
    const uint64_t inner = o.mn ? rows : K, outer = o.mn ? K : rows;
    const cuuint64_t dims[2] = {inner, outer};
    // the stride of a single row is never used, but has to be a multiple of 16 bytes
    const cuuint64_t stride[1] = {outer > 1 ? o.ld * size : (inner * size + 15) / 16 * 16};
    const cuuint32_t box[2] = {kTileBytes / size, box_rows}, one[2] = {1, 1};
    return encode_tiled()(map, map_type(type), 2, const_cast<void *>(o.p), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// map of an operand down its columns, in groups of 64 rows: boxes of `groups`
// of them by 64 reduction indices
bool make_wide_map(CUtensorMap *map, const Operand &o, uint64_t rows, uint64_t K, uint32_t type, uint32_t groups)
{
    if (rows % 64)
        return false;
    const uint32_t size = type_bytes(type);
    const cuuint64_t dims[3] = {64, K, rows / 64}, stride[2] = {K > 1 ? o.ld * size : rows * size, 64 * size};
    const cuuint32_t box[3] = {64, 64, groups}, one[3] = {1, 1, 1};
    return encode_tiled()(map, map_type(type), 3, const_cast<void *>(o.p), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// map of an output [rows, cols]: boxes of `across` x 32 values
bool make_out_map(CUtensorMap *map, void *p, uint64_t ld, uint64_t rows, uint64_t cols, uint32_t type, uint32_t across,
                  bool swizzled = false)
{
    const uint32_t size = type_bytes(type);
    const cuuint64_t dims[2] = {cols, rows}, stride[1] = {rows > 1 ? ld * size : (cols * size + 15) / 16 * 16};
    const cuuint32_t box[2] = {across, 32}, one[2] = {1, 1};
    const CUtensorMapDataType t = type == ECC_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : map_type(type);
    return encode_tiled()(map, t, 2, p, dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzled ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One map over two matrices of `rows` rows of one stride, 16 rows of each in
// turns: the second one's distance is a stride.  Whether there can be one.
bool make_turns_map(CUtensorMap *map, const Operand &lower, const Operand &upper, uint64_t rows, uint64_t K, uint32_t type)
{
    const uint32_t size = type_bytes(type);
    const uint64_t apart = (const uint8_t *)upper.p - (const uint8_t *)lower.p;
    if (rows % 16 || lower.ld != upper.ld || !apart || apart % 16 || apart >= 1ull << 40 || lower.ld * size >= 1ull << 36)
        return false;
    const cuuint64_t dims[4] = {K, 16, 2, rows / 16}, stride[3] = {lower.ld * size, apart, 16 * lower.ld * size};
    const cuuint32_t box[4] = {kTileBytes / size, 16, 2, kPTile / 32}, one[4] = {1, 1, 1, 1};
    return encode_tiled()(map, map_type(type), 4, const_cast<void *>(lower.p), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t up(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

struct Shape {
    bool pair;
    uint32_t bn, split;
};

// The launch shape with the least estimated time, in SM cycles.  What the
// estimate is made of was fitted to 48 products of 1 to 8192 rows, 100 to
// 16384 columns and reductions of 256 to 16384, bf16 and e4m3, each in every
// shape; the chosen shape was within 8% of the best of its product for 46.
// - a reduction block costs its products (128 bn 64 multiply-adds at 4096 a
//   cycle, 8-bit operands twice that) or its loads, whichever is more: 49
//   bytes a cycle for pairs, for single CTAs 70 on a full GPU, 62 below, 48
//   where the operands are streamed once (few rows);
// - a wave is one CTA an SM (two of the single ones share an SM's time), and
//   the operands cannot arrive faster than HBM gives them;
// - an epilogue, and joining a shared reduction.
// So 8 x 16384 x 4096 takes 26.8 us in 16-row tiles (28 in 64-row ones), 128
// x 4096 x 4096 15.5 us as 64-row tiles of four CTAs each (25 as pairs, 18 as
// 64-row tiles of two), 1024 x 4096 x 4096 28.5 us as pairs (32 as 128-row
// tiles).
Shape choose_shape(uint64_t rows, uint64_t cols, uint64_t K, uint32_t kblocks, bool q_mn, bool f8, int sms)
{
    Shape best{false, rows <= 16 && !q_mn ? 16u : 64u, 1};
    if (!kblocks)
        return best;
    const double hbm = (double)(rows + cols) * K * (f8 ? 1 : 2) / 3500;
    double least = 1e30;
    auto consider = [&](bool pair, uint32_t bn, uint32_t split, double t) {
        if (t < least) {
            least = t;
            best = {pair, bn, split};
        }
    };
    for (uint32_t bn : {256u, 128u}) {
        const double waves = std::ceil(2.0 * up(cols, 256) * up(rows, bn) / sms), bytes = kPBytes + bn / 2 * kTileBytes;
        const double work = waves * kblocks * std::max(bytes / 49, bn * 2.0);
        consider(true, bn, 1, std::max(work, hbm) + 5500 + 12 * bn + 0.01 * work);
    }
    for (uint32_t bn : {128u, 64u, 32u, 16u}) {
        if ((bn < 128 && rows > 4 * bn) || (bn > 16 && 2 * rows <= bn) || (q_mn && bn < 64))
            continue;
        for (uint32_t split = 1; split <= 8; split *= 2) {
            const double ctas = (double)up(cols, 128) * up(rows, bn) * split, bytes = kPBytes + bn * kTileBytes;
            if (split > 1 && (ctas > 2.0 * sms || kblocks < 2 * split))
                break;
            const double waves = ctas <= 2.0 * sms ? std::max(1.0, ctas / sms) : std::ceil(ctas / sms);
            const double rate = ctas > sms ? 70 : rows <= 128 ? 48 : 62;
            const double work = (double)up(kblocks, split) * waves * std::max(bytes / rate, bn * 2.0);
            const double join = split > 1 ? 2500 + 25.0 * bn * waves : 0;
            consider(false, bn, split, std::max(work, hbm) + 3000 + 12 * bn * waves + join + 0.01 * work);
        }
    }
    return best;
}

// Reductions of up to this many blocks hide no epilogue.
constexpr uint32_t kStagedBlocks = 16;

// A product made ready: its maps, its arguments.
struct Plan {
    CUtensorMap pm{}, pm2{}, qm{}, om{}, om2{}, om3{};
    GemmArgs g{};
    bool pair = false;
    uint32_t stage_bytes = 0;
    uint32_t tiles() const { return g.ptiles * g.qtiles; }
};

Shape shape_of(const Product &x, uint32_t type, int sms)
{
    const uint32_t per = type == ECC_E4M3 ? 128 : 64;
    Shape s = choose_shape(x.rows, x.mode == kGated ? 2 * x.cols : x.cols, x.K, (uint32_t)up(x.K, per), x.Q.mn, type == ECC_E4M3,
                           sms);
    // Logits: pairs on 256 x 256 tiles as soon as every pair has one.
    if ((x.mode == kStats || x.mode == kSlopes) && x.K && (s.pair || 2 * up(x.cols, 256) * up(x.rows, 256) >= (uint64_t)sms))
        s = {true, 256, 1};
    return s;
}

ecc_status make_plan(Plan &plan, const Product &x, const Shape &shape, uint32_t type, uint32_t *status, bool clear_status)
{
    const bool gated = x.mode == kGated;
    const uint32_t pcols = gated ? kPCols<kGated> : kPTile;
    const uint64_t ptiles = up(x.cols, shape.pair ? 2 * pcols : pcols), qtiles = up(x.rows, shape.bn);
    if (ptiles * qtiles >= (1u << 27))
        return ECC_ERR_ARG;
    GemmArgs &g = plan.g;
    g.e = x.e;
    g.rows = x.rows;
    g.cols = x.cols;
    g.kblocks = (uint32_t)up(x.K, type == ECC_E4M3 ? 128 : 64);
    g.kswitch = (uint32_t)(x.kswitch / 64);
    g.status = status;
    g.clear_status = clear_status;
    g.limit_ns = kWaitLimitNs + 1000ull * g.kblocks; // an epilogue waits for a whole reduction
    g.bn = shape.bn;
    g.split = shape.split;
    g.ptiles = (uint32_t)ptiles;
    g.qtiles = (uint32_t)qtiles;
    g.idesc = product_desc(type, x.P.mn, x.Q.mn, shape.pair ? 256 : 128, g.bn);
    plan.pair = shape.pair;
    const uint32_t qn = shape.pair ? g.bn / 2 : g.bn;
    plan.stage_bytes = kPBytes + qn * kTileBytes;
    if (!x.K)
        return ECC_OK;
    // (kDual: the first matrix's reduction ends somewhere in its last block, whose rest reads as zeros)
    const uint32_t box = gated ? 16 : x.P.mn ? 64 : kPTile;
    const uint64_t k1 = x.mode == kDual ? x.kfirst : x.K;
    // results through shared memory: of reductions that are shorter than the epilogue
    const Epilogue &e = x.e;
    if (shape.pair && g.kblocks <= kStagedBlocks && x.mode == kSlopes) { // (t is the workspace's: tokens by the vocabulary's part)
        if (encode_tiled() && make_out_map(&plan.om, e.out, e.ldout, x.cols, x.rows, e.out_type, 32, true))
            g.staged = 2048;
    } else if (shape.pair && g.kblocks <= kStagedBlocks && encode_tiled() && tma_rows(e.out, e.ldout, e.out_type, e.rswitch ? e.rows2 : x.rows)) {
        if (x.mode == kPlain && e.out_type != ECC_E4M3 && !e.pre && !e.residual) {
            const uint64_t rows = e.rswitch ? e.rows2 : x.rows;
            if (make_out_map(&plan.om, e.out, e.ldout, rows, x.cols, e.out_type, 32) &&
                (!e.rswitch || (tma_rows(e.out2, e.ldout2, e.out_type, rows) &&
                                make_out_map(&plan.om2, e.out2, e.ldout2, rows, x.cols, e.out_type, 32))))
                g.staged = 1024 * type_bytes(e.out_type);
        } else if (gated && e.pre) { // (the output alone gains nothing: 8192 x 8192 x 256 87 us, 85 by store_rows; with g and u 134, 154)
            const uint32_t bytes = 512 * (type_bytes(e.out_type) + 2 * type_bytes(e.pre_type));
            if (bytes <= 4096 && tma_rows(e.pre, e.ldpre, e.pre_type, x.rows) && tma_rows(e.pre2, e.ldpre2, e.pre_type, x.rows) &&
                make_out_map(&plan.om, e.out, e.ldout, x.rows, x.cols, e.out_type, 16) &&
                make_out_map(&plan.om2, e.pre, e.ldpre, x.rows, x.cols, e.pre_type, 16) &&
                make_out_map(&plan.om3, e.pre2, e.ldpre2, x.rows, x.cols, e.pre_type, 16))
                g.staged = (bytes + 127) / 128 * 128;
        }
    }
    const uint32_t last = (uint32_t)(x.rows - (qtiles - 1) * g.bn), half = g.bn / 2; // rows of the last tile
    g.odd = (up(std::min(last, half), 32) & 1) | (last > half ? (up(last - half, 32) & 1) << 1 : 0);
    if (!encode_tiled())
        return ECC_ERR_CUDA;
    g.qwide = x.Q.mn && make_wide_map(&plan.qm, x.Q, g.rows, x.K, type, qn / 64);
    if (!g.qwide && !make_map(&plan.qm, x.Q, g.rows, x.K, type, x.Q.mn ? 64 : qn))
        return ECC_ERR_CUDA;
    if (gated) {
        g.e.swapped = x.P2.p < x.P.p;
        if ((g.one_box = make_turns_map(&plan.pm, g.e.swapped ? x.P2 : x.P, g.e.swapped ? x.P : x.P2, g.cols, x.K, type)))
            return ECC_OK;
        g.e.swapped = false;
    }
    g.pwide = x.P.mn && make_wide_map(&plan.pm, x.P, g.cols, k1, type, kPTile / 64) &&
              (x.mode != kDual || make_wide_map(&plan.pm2, x.P2, g.cols, k1, type, kPTile / 64));
    if (!g.pwide && (!make_map(&plan.pm, x.P, g.cols, k1, type, box) ||
                     ((gated || x.mode == kDual) && !make_map(&plan.pm2, x.P2, g.cols, k1, type, box))))
        return ECC_ERR_CUDA;
    return ECC_OK;
}

// stages and shared memory of a launch of `ctas` CTAs
size_t stage_memory(Plan &plan, uint32_t ctas, int sms)
{
    const bool alone = plan.pair || ctas <= (uint32_t)sms; // one CTA an SM
    const uint32_t out = plan.g.staged * 2 * 8; // two stages for each of eight warps
    const uint32_t budget = (alone ? kAloneSmem : kSharedSmem) - kSmemHead - (uint32_t)sizeof(GemmBars) - out;
    plan.g.stages = std::min(kMaxStages, budget / plan.stage_bytes);
    return kSmemHead + (size_t)plan.g.stages * plan.stage_bytes + out;
}

ecc_status launch_plan(const void *f, int threads, uint32_t ctas, uint32_t cluster, size_t smem, void **args, bool behind,
                       cudaStream_t st)
{
    if (occupancy(f, threads, smem) <= 0)
        return ECC_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = behind ? 2 : 1;
    return launch_status(cudaLaunchKernelExC(&cfg, f, args));
}

// Whether a few tokens' statistics stream the head (P: tokens, Q: the head)
// through a persistent CTA an SM: with tiles for most of them.
bool streams(const Product &x, int sms) { return x.mode == kStats && x.K && x.cols <= 64 && 2 * up(x.rows, kPTile) >= (uint64_t)sms; }

uint32_t stream_ctas(const Product &x, int sms) { return (uint32_t)std::min<uint64_t>(up(x.rows, kPTile), sms); }

ecc_status stream_stats(const Product &x, uint32_t type, uint32_t *status, bool behind, int sms, cudaStream_t st)
{
    CUtensorMap wm, xm;
    StreamArgs g{};
    g.e = x.e;
    g.vocab = x.rows;
    g.tokens = x.cols;
    g.kblocks = (uint32_t)up(x.K, type == ECC_E4M3 ? 128 : 64);
    g.tiles = (uint32_t)up(x.rows, kPTile);
    g.bn = x.cols <= 16 ? 16 : x.cols <= 32 ? 32 : 64;
    g.segs = std::min(256 / g.bn, (g.kblocks + kSegment - 1) / kSegment);
    const uint32_t stage_bytes = kPBytes + g.bn * kTileBytes;
    g.stages = std::min(kMaxStages, (kAloneSmem - kSmemHead - (uint32_t)sizeof(StreamBars)) / stage_bytes);
    g.idesc = product_desc(type, false, false, 128, g.bn);
    g.status = status;
    g.limit_ns = kWaitLimitNs + 1000ull * g.kblocks;
    if (!encode_tiled() || !make_map(&wm, x.Q, x.rows, x.K, type, kPTile) || !make_map(&xm, x.P, x.cols, x.K, type, g.bn))
        return ECC_ERR_CUDA;
    void *args[] = {&wm, &xm, &g};
    return launch_plan(stats_stream(type == ECC_E4M3), kStreamThreads, stream_ctas(x, sms), 1,
                       kSmemHead + (size_t)g.stages * stage_bytes, args, behind, st);
}

// Whether a kernel is launched with `n` registers a thread: one whose warps
// share them out differently would wait forever if there were fewer.
bool registers_of(const void *f, int n)
{
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, f) == cudaSuccess && a.numRegs == n;
}

const void *kernel_of(const Product &x, bool f8, bool pair)
{
    if (x.mode == kGated)
        return gated_kernel(f8, pair);
    if (x.mode == kDual)
        return dual_kernel(pair);
    if (x.mode == kStats)
        return stats_kernel(f8, pair);
    if (x.mode == kSlopes)
        return slopes_kernel(pair);
    return f8                     ? gemm_kernel<false, false, true, kPlain>(pair)
           : x.P.mn && x.Q.mn     ? gemm_kernel<true, true, false, kPlain>(pair)
           : x.P.mn               ? gemm_kernel<true, false, false, kPlain>(pair)
                                  : gemm_kernel<false, false, false, kPlain>(pair);
}

} // namespace

bool tma_rows(const void *p, uint64_t ld, uint32_t type, uint64_t rows)
{
    const uint64_t bytes = ld * type_bytes(type);
    return ((uintptr_t)p & 15) == 0 && (rows <= 1 || ((bytes & 15) == 0 && bytes < (1ull << 40)));
}

uint32_t stats_parts(const Product &x, uint32_t type)
{
    const int sms = sm_count();
    if (sms <= 0)
        return 0;
    if (streams(x, sms))
        return 4 * stream_ctas(x, sms);
    const Shape s = shape_of(x, type, sms);
    return (uint32_t)up(x.rows, s.bn) * (s.pair ? 2 : s.split);
}

ecc_status gemm(const Product &x, uint32_t type, uint32_t *status, bool clear_status, bool behind, cudaStream_t st)
{
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    if (streams(x, sms))
        return stream_stats(x, type, status, behind, sms, st);
    Plan plan;
    const ecc_status rc = make_plan(plan, x, shape_of(x, type, sms), type, status, clear_status);
    if (rc != ECC_OK)
        return rc;
    const bool pair = plan.pair;
    const uint32_t ctas = pair ? 2 * std::min<uint32_t>(plan.tiles(), sms / 2) : plan.tiles() * plan.g.split;
    const size_t smem = stage_memory(plan, ctas, sms);
    const void *f = kernel_of(x, type == ECC_E4M3, pair);
    void *pair_args[] = {&plan.pm, &plan.pm2, &plan.qm, &plan.om, &plan.om2, &plan.om3, &plan.g};
    void *split_args[] = {&plan.pm, &plan.pm2, &plan.qm, &plan.g};
    void **args = pair ? pair_args : split_args;
    if (pair && x.mode == kStats && !registers_of(f, kStatsRegisters))
        return ECC_ERR_CUDA;
    return launch_plan(f, pair ? (x.mode == kStats ? kStatsThreads : kPairThreads) : kSplitThreads, ctas, pair ? 2 : plan.g.split, smem, args, behind, st);
}

ecc_status gemm_backward(const Product &dx, const Product &dw, uint32_t type, uint32_t *status, bool clear_status, bool behind,
                         cudaStream_t st)
{
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    Shape s1 = shape_of(dx, type, sms), s2 = shape_of(dw, type, sms);
    // In one launch where neither fills the GPU by itself and both fit it, two
    // CTAs an SM, with their reductions shared out less if need be; or, as they
    // are, where they make two such fillings at most: the second product's CTAs
    // start as the first one's end (linear gradient of 512 x 2048 x 2048 34.5 us,
    // 46.8 in two launches; 333 x 8001 x 515 52.9 and 62.1).
    // (dx is kPlain or kDual, dw kPlain: 128 columns a tile)
    const uint64_t t1 = up(dx.cols, kPTile) * up(dx.rows, s1.bn), t2 = up(dw.cols, kPTile) * up(dw.rows, s2.bn);
    const Shape o1 = s1, o2 = s2;
    while (t1 * s1.split + t2 * s2.split > 2ull * sms && (s1.split > 1 || s2.split > 1)) {
        uint32_t &s = t1 * s1.split > t2 * s2.split ? (s1.split > 1 ? s1.split : s2.split) : (s2.split > 1 ? s2.split : s1.split);
        s /= 2;
    }
    if (t1 * s1.split + t2 * s2.split > 2ull * sms) {
        s1 = o1;
        s2 = o2;
    }
    if (s1.pair || s2.pair || !dx.K || !dw.K || t1 * s1.split + t2 * s2.split > 4ull * sms) {
        const ecc_status rc = gemm(dx, type, status, clear_status, behind, st); // (each in its own shape)
        return rc == ECC_OK ? gemm(dw, type, status, false, true, st) : rc;
    }
    Plan a, b;
    ecc_status rc = make_plan(a, dx, s1, type, status, clear_status);
    if (rc == ECC_OK)
        rc = make_plan(b, dw, s2, type, status, false);
    if (rc != ECC_OK)
        return rc;
    const uint32_t cluster = std::max(s1.split, s2.split);
    uint32_t n1 = (uint32_t)up(a.tiles() * s1.split, cluster) * cluster;
    const uint32_t ctas = n1 + (uint32_t)up(b.tiles() * s2.split, cluster) * cluster;
    const size_t m1 = stage_memory(a, ctas, sms), m2 = stage_memory(b, ctas, sms);
    void *args[] = {&a.pm, &a.pm2, &a.qm, &a.g, &b.pm, &b.qm, &b.g, &n1};
    return launch_plan(dx.mode == kDual ? dual_both_kernel() : (const void *)gemm_both_kernel<kPlain>, kSplitThreads, ctas, cluster, std::max(m1, m2), args, behind, st);
}

} // namespace ecc
