// ecc_gemm.cu -- matrix products on the tensor cores (tcgen05, operands by
// tiled TMA, accumulators in tensor memory) with the linear operators'
// epilogue.
//
// out[r, c] = act(scale * sum_k Q[r, k] P[c, k] + bias[c]) + residual[r, c].
// P, whose rows are the output's columns, is the product's 128-row side, so
// that a lane of tensor memory is a column of the output: a warp stores 32
// neighbouring values of a row at once, whatever the rows' alignment, and a
// thread needs one bias value a tile.  The other side, Q, gives the tile's
// width: 16 for a few tokens up to 256 for a training batch.
//
// gemm_pair_kernel: pairs of CTAs (tcgen05 cta_group::2) on 256 x `bn` tiles;
// per CTA a TMA warp, a product warp (of the pair's first CTA) and four
// or eight epilogue warps.  The pairs are persistent, and the epilogue works on one
// accumulator while the products fill the other.  For many tiles.
// gemm_split_kernel: one 128 x `bn` tile a cluster of up to 8 CTAs that share
// its reduction, for few tiles: the parts are joined through distributed
// shared memory, in the order of the CTAs' ranks.  Two CTAs an SM, or one
// with twice the stages where there are no more CTAs than SMs.

#include <algorithm>
#include <cmath>

#include "ecc_act.cuh"
#include "ecc_gemm.h"
#include "ecc_tensor.cuh"

namespace ecc {

constexpr int kSplitThreads = 192; // TMA warp, product warp, 4 epilogue warps
constexpr int kPairThreads = 320;  // 8 of them: half a tile's rows each (reductions of 1024 are shorter than an epilogue)
constexpr uint32_t kPTile = 128;  // P rows of a CTA
constexpr uint32_t kMaxStages = 12;
constexpr uint32_t kPBytes = kPTile * kTileBytes;
constexpr uint32_t kAloneSmem = 226 * 1024, kSharedSmem = 112 * 1024; // of a CTA that has an SM to itself, or half of it
constexpr uint32_t kSmemHead = 1024; // room to align the stages to 1024 bytes

struct GemmArgs {
    Epilogue e;
    uint64_t rows, cols;
    uint32_t kblocks; // reduction blocks of 128 bytes (64 reduction indices for MN-major operands)
    uint32_t ptiles, qtiles, bn, stages, idesc, split;
    uint32_t *status;
    bool clear_status;
    uint64_t limit_ns;
};

struct GemmBars {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2];
    uint32_t tmem;
};

// ---------------------------------------------------------------- epilogue
template <uint32_t ACT, int W> __device__ __forceinline__ void activate(float (&a)[W])
{
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        const float2 v = act_value2<ACT>(make_float2(a[j], a[j + 1]));
        a[j] = v.x;
        a[j + 1] = v.y;
    }
}

// W rows of a column, the first n of them in range.  The rows' addresses are
// the same for the whole warp (uniform registers); a lane adds its column.
// A reduction of less than about 1024 takes as long as this does, 3.8 us a tile
// of 256 x 256 (8192 x 16384 x 64: 107 us, 2.5 TB/s, and as long with float32 or e4m3
// results).  Slower: four values a store, lanes' rows exchanged for columns by
// shuffles, 119 us; whole rows by four warps through shared memory, 195; eight
// warps of 16 rows at a time, 125.  Sixteen such warps: 103, but 168 instead
// of 163 at a reduction of 1024.
template <typename T, int W>
__device__ __forceinline__ void store_rows(void *base, uint64_t ld, uint64_t r0, uint32_t n, uint32_t c, const float (&a)[W],
                                           float s)
{
    T *row = static_cast<T *>(base) + r0 * ld;
    if (n == W) {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            row[c] = from_f32<T>(sizeof(T) == 1 ? a[j] * s : a[j]);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            if (j < n)
                row[c] = from_f32<T>(sizeof(T) == 1 ? a[j] * s : a[j]);
    }
}
// The residual of W rows of a column, as it is stored: asked for before the
// products are waited for (with the loads after them a 8192 x 16384 x 4096
// product took 906 us instead of 560).
template <typename T, int W>
__device__ __forceinline__ void load_rows(const void *base, uint64_t ld, uint64_t r0, uint32_t n, uint32_t c, uint32_t (&v)[W])
{
    const T *row = static_cast<const T *>(base) + r0 * ld;
    if (n == W) {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            v[j] = row[c];
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j, row += ld)
            if (j < n)
                v[j] = row[c];
    }
}
template <int W>
__device__ __forceinline__ void ask_residual(const Epilogue &e, uint32_t (&v)[W], uint64_t r0, uint32_t n, uint32_t c)
{
    if (!e.residual)
        return;
    if (e.res_type == ECC_F32)
        load_rows<uint32_t>(e.residual, e.ldres, r0, n, c, v);
    else
        load_rows<uint16_t>(e.residual, e.ldres, r0, n, c, v);
}
template <int W> __device__ __forceinline__ void add_residual(uint32_t type, const uint32_t (&v)[W], float (&a)[W])
{
    if (type == ECC_F32) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            a[j] += __uint_as_float(v[j]);
    } else if (type == ECC_BF16) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            a[j] += __uint_as_float(v[j] << 16);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            a[j] += __half2float(__ushort_as_half((unsigned short)v[j]));
    }
}

// W rows from row `r0` (the first n of them in range) of this thread's column c
template <int W>
__device__ __forceinline__ void finish(const Epilogue &e, float (&a)[W], const uint32_t (&res)[W], uint64_t r0, uint32_t n,
                                       uint32_t c, float bias)
{
#pragma unroll
    for (int j = 0; j < W; ++j)
        a[j] = a[j] * e.scale + bias;
    if (e.pre) {
        if (e.pre_type == ECC_F32)
            store_rows<float>(e.pre, e.ldpre, r0, n, c, a, 1.f);
        else if (e.pre_type == ECC_BF16)
            store_rows<bf16>(e.pre, e.ldpre, r0, n, c, a, 1.f);
        else
            store_rows<__half>(e.pre, e.ldpre, r0, n, c, a, 1.f);
    }
    if (e.act == ECC_ACT_RELU)
        activate<ECC_ACT_RELU>(a);
    else if (e.act == ECC_ACT_GELU)
        activate<ECC_ACT_GELU>(a);
    else if (e.act == ECC_ACT_GELU_TANH)
        activate<ECC_ACT_GELU_TANH>(a);
    else if (e.act == ECC_ACT_SILU)
        activate<ECC_ACT_SILU>(a);
    if (e.residual)
        add_residual(e.res_type, res, a);
    if (e.out_type == ECC_F32)
        store_rows<float>(e.out, e.ldout, r0, n, c, a, 1.f);
    else if (e.out_type == ECC_BF16)
        store_rows<bf16>(e.out, e.ldout, r0, n, c, a, 1.f);
    else if (e.out_type == ECC_F16)
        store_rows<__half>(e.out, e.ldout, r0, n, c, a, 1.f);
    else
        store_rows<e4m3>(e.out, e.ldout, r0, n, c, a, e.out_scale);
}

// This CTA's part of a tile, [column of tensor memory][lane], for the join.
template <int W> __device__ __forceinline__ void keep_part(float *parts, const float (&a)[W], uint32_t j, uint32_t row)
{
#pragma unroll
    for (int i = 0; i < W; ++i)
        parts[(j + i) * kPTile + row] = a[i];
}
// Share `share` of a tile's rows [r0, ...): the sum of the g.split CTAs'
// parts, eight rows at a time so that their loads are in flight together,
// then the epilogue.  `at`: this lane's first value in its CTA's part;
// `base`: the cluster's rank of the first of those CTAs.
__device__ __forceinline__ void join_parts(const GemmArgs &g, uint32_t at, uint32_t base, uint32_t share, uint64_t r0, uint32_t c)
{
    const uint32_t n = (uint32_t)min((uint64_t)g.bn, g.rows - r0), per = (n + g.split - 1) / g.split;
    const uint32_t j0 = share * per, j1 = min(n, j0 + per);
    if (c >= g.cols)
        return;
    const float bias = g.e.bias ? load_any(g.e.bias, c, g.e.bias_type) : 0.f;
    for (uint32_t j = j0; j < j1; j += 8) {
        float a[8] = {};
        uint32_t res[8];
        ask_residual(g.e, res, r0 + j, min(8u, j1 - j), c);
        for (uint32_t k = 0; k < g.split; ++k) {
            const uint32_t from = cluster_addr(at + j * kPTile * 4, base + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (j + i < j1)
                    a[i] += cluster_load(from + i * kPTile * 4);
        }
        finish(g.e, a, res, r0 + j, min(8u, j1 - j), c, bias);
    }
}

// ---------------------------------------------------------------- loads and products of a reduction block
// rows [r0, r0 + n) of reduction block kb -> dst
template <int CG, bool MN, bool F8>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, uint64_t r0, uint32_t n, uint32_t kb,
                                             uint32_t bar)
{
    constexpr int per = F8 ? 128 : 64; // reduction indices of a block
    if constexpr (MN) {
        for (uint32_t c = 0; c < n; c += 64)
            tma_load<CG>(dst + c * kTileBytes, map, (int)(r0 + c), (int)(kb * 64), bar);
    } else {
        tma_load<CG>(dst, map, (int)(kb * per), (int)r0, bar);
    }
}

template <int CG, bool PMN, bool QMN, bool F8>
__device__ __forceinline__ void multiply_block(uint32_t d, uint32_t pa, uint32_t qa, uint32_t idesc, bool first)
{
    const uint64_t a = operand_desc<PMN>(pa, 64 * kTileBytes), b = operand_desc<QMN>(qa, 64 * kTileBytes);
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k)
        tensor_product<CG, F8>(d, a + k * operand_step<PMN>(), b + k * operand_step<QMN>(), idesc, !first || k > 0);
}

// behind the launch's own preparation: wait for what it reads
__device__ __forceinline__ void begin(const GemmArgs &g)
{
    wait_for_previous();
    let_next_start();
    if (g.clear_status && blockIdx.x == 0 && threadIdx.x == 0) // waits that give up do so a second from now at the earliest
        *(volatile uint32_t *)g.status = ECC_OK;
}

// ---------------------------------------------------------------- pairs of CTAs, many tiles
// Tiles in groups of 8 column tiles, a group row tile by row tile: the tiles
// in work at a time form a block that shares its operands through L2.
struct TilePos {
    uint32_t p, q;
};
__device__ __forceinline__ TilePos tile_pos(uint32_t t, uint32_t ptiles, uint32_t qtiles)
{
    const uint32_t g = t / (8 * qtiles), p0 = g * 8, w = min(8u, ptiles - p0), r = t - g * 8 * qtiles;
    return {p0 + r % w, r / w};
}

template <bool PMN, bool QMN, bool F8>
__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_pair_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ GemmArgs g)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ GemmBars s;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t stage0 = (smem_u32(smem_raw) + kSmemHead - 1) & ~(kSmemHead - 1);
    const uint32_t qn = g.bn / 2, stage_bytes = kPBytes + qn * kTileBytes;
    const uint32_t tiles = g.ptiles * g.qtiles, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < g.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 16); // eight epilogue warps of each CTA
        }
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        prefetch_map(&pmap);
        prefetch_map(&qmap);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(&s.tmem), 512);
        tmem_fence_before();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&s.tmem;
    begin(g);

    if (warp == 0) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0, issued = 0;
            bool ok = true;
            for (uint32_t t = pair; t < tiles && ok; t += pairs) {
                const TilePos pos = tile_pos(t, g.ptiles, g.qtiles);
                const uint64_t p0 = (uint64_t)pos.p * 2 * kPTile + rank * kPTile, q0 = (uint64_t)pos.q * g.bn + rank * qn;
                for (uint32_t kb = 0; kb < g.kblocks; ++kb) {
                    if (!(ok = mbar_wait(&s.empty[st], ph ^ 1, g.limit_ns)))
                        break;
                    const uint32_t bar = cluster_addr(smem_u32(&s.full[st]), 0), at = stage0 + st * stage_bytes;
                    if (rank == 0)
                        mbar_expect_tx(&s.full[st], 2 * stage_bytes);
                    load_operand<2, PMN, F8>(at, &pmap, p0, kPTile, kb, bar);
                    load_operand<2, QMN, F8>(at + kPBytes, &qmap, q0, qn, kb, bar);
                    ++issued;
                    if (++st == g.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) { // give the copies in flight a last wait
                set_status(g.status, ECC_ERR_TIMEOUT);
                if (rank == 0)
                    for (uint32_t i = 0; i < min(issued, g.stages); ++i) {
                        if (st == 0) {
                            st = g.stages;
                            ph ^= 1;
                        }
                        --st;
                        (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                    }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t st = 0, ph = 0, acc = 0, aph = 0;
            bool ok = true;
            for (uint32_t t = pair; t < tiles && ok; t += pairs) {
                if (!(ok = mbar_wait(&s.tempty[acc], aph ^ 1, g.limit_ns)))
                    break;
                tmem_fence_after();
                for (uint32_t kb = 0; kb < g.kblocks; ++kb) {
                    if (!(ok = mbar_wait(&s.full[st], ph, g.limit_ns))) {
                        (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t at = stage0 + st * stage_bytes;
                    multiply_block<2, PMN, QMN, F8>(tmem + acc * g.bn, at, at + kPBytes, g.idesc, kb == 0);
                    tensor_commit<2>(smem_u32(&s.empty[st]));
                    if (++st == g.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                tensor_commit<2>(smem_u32(&s.tfull[acc]));
                if (acc)
                    aph ^= 1;
                acc ^= 1;
            }
            if (!ok)
                set_status(g.status, ECC_ERR_TIMEOUT);
        }
    } else {
        const uint32_t quad = warp & 3; // a warp reads the lanes of its number modulo 4
        const uint32_t j0 = warp < 6 ? 0 : g.bn / 2, j1 = j0 + g.bn / 2;
        uint32_t acc = 0, aph = 0;
        for (uint32_t t = pair; t < tiles; t += pairs) {
            const TilePos pos = tile_pos(t, g.ptiles, g.qtiles);
            const uint32_t c = pos.p * 2 * kPTile + rank * kPTile + quad * 32 + lane;
            const uint64_t r0 = (uint64_t)pos.q * g.bn;
            const bool col_ok = c < g.cols;
            const float bias = g.e.bias && col_ok ? load_any(g.e.bias, c, g.e.bias_type) : 0.f;
            const uint64_t left = g.rows - r0;
            uint32_t res[2][32]; // of this chunk of 32 rows and the next
            auto ask = [&](uint32_t j, uint32_t (&v)[32]) {
                if (col_ok && j < j1 && j < left)
                    ask_residual(g.e, v, r0 + j, (uint32_t)min((uint64_t)32, left - j), c);
            };
            ask(j0, res[0]);
            if (!__all_sync(~0u, mbar_wait(&s.tfull[acc], aph, g.limit_ns))) {
                if (lane == 0)
                    set_status(g.status, ECC_ERR_TIMEOUT);
                break;
            }
            tmem_fence_after();
            auto chunk = [&](uint32_t j, const uint32_t (&v)[32]) {
                float a[32];
                tmem_load32(tmem + (quad * 32 << 16) + acc * g.bn + j, a);
                if (j + 32 == j1) { // the accumulator is read: products may fill it again
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        cluster_arrive(cluster_addr(smem_u32(&s.tempty[acc]), 0));
                }
                if (col_ok && j < left)
                    finish(g.e, a, v, r0 + j, (uint32_t)min((uint64_t)32, left - j), c, bias);
            };
            for (uint32_t j = j0; j < j1; j += 64) { // (bn is 128 or 256)
                ask(j + 32, res[1]);
                chunk(j, res[0]);
                ask(j + 64, res[0]);
                chunk(j + 32, res[1]);
            }
            if (acc)
                aph ^= 1;
            acc ^= 1;
        }
    }
    __syncthreads();
    __syncwarp();
    tmem_fence_before();
    cluster_sync(); // both CTAs are done with each other's barriers and tensor memory
    tmem_fence_after();
    if (warp == 1)
        tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------- clusters that share a tile's reduction
// `wait` waits for the products (the first residual is asked for before)
template <int W, typename Wait>
__device__ __forceinline__ void split_columns(const GemmArgs &g, uint32_t tmem, uint32_t quad, uint32_t lane, uint32_t c,
                                              uint64_t r0, bool col_ok, float bias, bool direct, float *part, Wait wait)
{
    const uint64_t left = g.rows - r0;
    for (uint32_t j = 0; j < g.bn && j < left; j += W) {
        float a[W];
        uint32_t res[W];
        const uint32_t n = (uint32_t)min((uint64_t)W, left - j);
        if (direct && col_ok)
            ask_residual(g.e, res, r0 + j, n, c);
        if (j == 0 && g.kblocks && !wait())
            return;
        if (g.kblocks) {
            if constexpr (W == 32)
                tmem_load32(tmem + (quad * 32 << 16) + j, a);
            else
                tmem_load16(tmem + (quad * 32 << 16) + j, a);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                a[i] = 0.f;
        }
        if (direct) {
            if (col_ok)
                finish(g.e, a, res, r0 + j, n, c, bias);
        } else {
            keep_part(part, a, j, quad * 32 + lane);
        }
    }
}

// block: this CTA's number among the product's
template <bool PMN, bool QMN, bool F8>
__device__ __forceinline__ void split_tile(const CUtensorMap &pmap, const CUtensorMap &qmap, const GemmArgs &g, uint32_t block,
                                           uint8_t *smem_raw, GemmBars &s)
{
    // the CTAs that share a tile are g.split neighbours of the cluster, `base` the first of them
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, crank = cluster_rank();
    const uint32_t rank = crank & (g.split - 1), base = crank - rank;
    const uint32_t off = (kSmemHead - (smem_u32(smem_raw) & (kSmemHead - 1))) & (kSmemHead - 1);
    const uint32_t stage0 = smem_u32(smem_raw) + off;
    const uint32_t stage_bytes = kPBytes + g.bn * kTileBytes;
    const uint32_t tile = block / g.split;
    if (tile >= g.ptiles * g.qtiles) { // fills up the last cluster
        if (g.split > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }
    const uint64_t p0 = (uint64_t)(tile % g.ptiles) * kPTile, q0 = (uint64_t)(tile / g.ptiles) * g.bn;
    const uint32_t kb0 = (uint32_t)((uint64_t)g.kblocks * rank / g.split);
    const uint32_t kb1 = (uint32_t)((uint64_t)g.kblocks * (rank + 1) / g.split);
    const uint32_t tcols = g.bn < 32 ? 32 : g.bn;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < g.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        mbar_init(&s.tfull[0], 1);
        fence_mbar_init();
        fence_proxy_async();
    }
    if (threadIdx.x == 32 && g.kblocks) {
        prefetch_map(&pmap);
        prefetch_map(&qmap);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), tcols);
        tmem_fence_before();
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&s.tmem;
    begin(g);

    const uint32_t quad = warp & 3;
    const uint32_t c = (uint32_t)p0 + quad * 32 + lane;
    const bool col_ok = c < g.cols;
    float bias = 0.f;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!(ok = mbar_wait(&s.empty[st], ph ^ 1, g.limit_ns)))
                    break;
                const uint32_t at = stage0 + st * stage_bytes;
                mbar_expect_tx(&s.full[st], stage_bytes);
                load_operand<1, PMN, F8>(at, &pmap, p0, kPTile, kb, smem_u32(&s.full[st]));
                load_operand<1, QMN, F8>(at + kPBytes, &qmap, q0, g.bn, kb, smem_u32(&s.full[st]));
                if (++st == g.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (!ok) {
                set_status(g.status, ECC_ERR_TIMEOUT);
                for (uint32_t i = 0; i < g.stages; ++i) { // the copies in flight: a last wait each
                    if (st == 0) {
                        st = g.stages;
                        ph ^= 1;
                    }
                    --st;
                    (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && kb1 > kb0) {
            uint32_t st = 0, ph = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!(ok = mbar_wait(&s.full[st], ph, g.limit_ns))) {
                    (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                    break;
                }
                tmem_fence_after();
                const uint32_t at = stage0 + st * stage_bytes;
                multiply_block<1, PMN, QMN, F8>(tmem, at, at + kPBytes, g.idesc, kb == kb0);
                tensor_commit<1>(smem_u32(&s.empty[st]));
                if (++st == g.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            tensor_commit<1>(smem_u32(&s.tfull[0]));
            if (!ok)
                set_status(g.status, ECC_ERR_TIMEOUT);
        }
    } else {
        if (g.e.bias && col_ok)
            bias = load_any(g.e.bias, c, g.e.bias_type);
        auto wait = [&] {
            ok = __all_sync(~0u, mbar_wait(&s.tfull[0], 0, g.limit_ns));
            if (!ok && lane == 0)
                set_status(g.status, ECC_ERR_TIMEOUT);
            tmem_fence_after();
            return ok;
        };
        // once every product of this CTA is complete, the stages' memory holds its part
        float *part = reinterpret_cast<float *>(smem_raw + off);
        if (g.bn == 16)
            split_columns<16>(g, tmem, quad, lane, c, q0, col_ok, bias, g.split == 1, part, wait);
        else
            split_columns<32>(g, tmem, quad, lane, c, q0, col_ok, bias, g.split == 1, part, wait);
        tmem_fence_before();
    }
    __syncwarp();
    if (g.split > 1) {
        cluster_sync(); // all parts are written
        if (warp >= 2)
            join_parts(g, stage0 + (quad * 32 + lane) * 4, base, rank, q0, c);
        __syncwarp();
        cluster_sync(); // nobody reads this CTA's part any more
    } else {
        __syncthreads();
        __syncwarp();
    }
    tmem_fence_after();
    if (warp == 1)
        tmem_free<1>(tmem, tcols);
}

template <bool PMN, bool QMN, bool F8>
__global__ void __launch_bounds__(kSplitThreads, 2)
    gemm_split_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ GemmArgs g)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ GemmBars s;
    split_tile<PMN, QMN, F8>(pmap, qmap, g, blockIdx.x, smem_raw, s);
}

// A layer's two backward products in one launch: the first `n1` CTAs work on
// dx (w down its columns, t along its rows), the others on dw (both down
// their columns).  For layers whose products leave SMs idle: one after the
// other they took 22 us for 100 x 1000 x 1000, of which the kernels' starts and
// ends are most.
__global__ void __launch_bounds__(kSplitThreads, 2)
    gemm_both_kernel(const __grid_constant__ CUtensorMap p1, const __grid_constant__ CUtensorMap q1,
                     const __grid_constant__ GemmArgs g1, const __grid_constant__ CUtensorMap p2,
                     const __grid_constant__ CUtensorMap q2, const __grid_constant__ GemmArgs g2, uint32_t n1)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ GemmBars s;
    if (blockIdx.x < n1)
        split_tile<true, false, false>(p1, q1, g1, blockIdx.x, smem_raw, s);
    else
        split_tile<true, true, false>(p2, q2, g2, blockIdx.x - n1, smem_raw, s);
}

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

// map of an operand: boxes of 128 bytes x `box_rows`
bool make_map(CUtensorMap *map, const Operand &o, uint64_t rows, uint64_t K, uint32_t type, uint32_t box_rows)
{
    const uint32_t size = type_bytes(type);
    const uint64_t inner = o.mn ? rows : K, outer = o.mn ? K : rows;
    const cuuint64_t dims[2] = {inner, outer};
    // the stride of a single row is never used, but has to be a multiple of 16 bytes
    const cuuint64_t stride[1] = {outer > 1 ? o.ld * size : (inner * size + 15) / 16 * 16};
    const cuuint32_t box[2] = {kTileBytes / size, box_rows}, one[2] = {1, 1};
    const CUtensorMapDataType dt = type == ECC_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : type == ECC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return encode_tiled()(map, dt, 2, const_cast<void *>(o.p), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
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

// A product made ready: its maps, its arguments.
struct Plan {
    CUtensorMap pm{}, qm{};
    GemmArgs g{};
    bool pair = false;
    uint32_t stage_bytes = 0;
    uint32_t tiles() const { return g.ptiles * g.qtiles; }
};

Shape shape_of(const Product &x, uint32_t type, int sms)
{
    const uint32_t per = type == ECC_E4M3 ? 128 : 64;
    return choose_shape(x.rows, x.cols, x.K, (uint32_t)up(x.K, per), x.Q.mn, type == ECC_E4M3, sms);
}

ecc_status make_plan(Plan &plan, const Product &x, const Shape &shape, uint32_t type, uint32_t *status, bool clear_status)
{
    const uint64_t ptiles = up(x.cols, shape.pair ? 2 * kPTile : kPTile), qtiles = up(x.rows, shape.bn);
    if (ptiles * qtiles >= (1u << 27))
        return ECC_ERR_ARG;
    GemmArgs &g = plan.g;
    g.e = x.e;
    g.rows = x.rows;
    g.cols = x.cols;
    g.kblocks = (uint32_t)up(x.K, type == ECC_E4M3 ? 128 : 64);
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
    if (x.K && (!encode_tiled() || !make_map(&plan.pm, x.P, g.cols, x.K, type, x.P.mn ? 64 : kPTile) ||
                !make_map(&plan.qm, x.Q, g.rows, x.K, type, x.Q.mn ? 64 : qn)))
        return ECC_ERR_CUDA;
    return ECC_OK;
}

// stages and shared memory of a launch of `ctas` CTAs
size_t stage_memory(Plan &plan, uint32_t ctas, int sms)
{
    const bool alone = plan.pair || ctas <= (uint32_t)sms; // one CTA an SM
    const uint32_t budget = (alone ? kAloneSmem : kSharedSmem) - kSmemHead - (uint32_t)sizeof(GemmBars);
    plan.g.stages = std::min(kMaxStages, budget / plan.stage_bytes);
    return kSmemHead + (size_t)plan.g.stages * plan.stage_bytes;
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

template <bool PMN, bool QMN, bool F8> const void *kernel_of(bool pair)
{
    return pair ? (const void *)gemm_pair_kernel<PMN, QMN, F8> : (const void *)gemm_split_kernel<PMN, QMN, F8>;
}

} // namespace

bool tma_rows(const void *p, uint64_t ld, uint32_t type, uint64_t rows)
{
    const uint64_t bytes = ld * type_bytes(type);
    return ((uintptr_t)p & 15) == 0 && (rows <= 1 || ((bytes & 15) == 0 && bytes < (1ull << 40)));
}

ecc_status gemm(const Product &x, uint32_t type, uint32_t *status, bool clear_status, bool behind, cudaStream_t st)
{
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    Plan plan;
    const ecc_status rc = make_plan(plan, x, shape_of(x, type, sms), type, status, clear_status);
    if (rc != ECC_OK)
        return rc;
    const bool pair = plan.pair;
    const uint32_t ctas = pair ? 2 * std::min<uint32_t>(plan.tiles(), sms / 2) : plan.tiles() * plan.g.split;
    const size_t smem = stage_memory(plan, ctas, sms);
    const void *f = type == ECC_E4M3           ? kernel_of<false, false, true>(pair)
                    : x.P.mn && x.Q.mn         ? kernel_of<true, true, false>(pair)
                    : x.P.mn                   ? kernel_of<true, false, false>(pair)
                                               : kernel_of<false, false, false>(pair);
    void *args[] = {&plan.pm, &plan.qm, &plan.g};
    return launch_plan(f, pair ? kPairThreads : kSplitThreads, ctas, pair ? 2 : plan.g.split, smem, args, behind, st);
}

ecc_status gemm_backward(const Product &dx, const Product &dw, uint32_t type, uint32_t *status, bool clear_status, bool behind,
                         cudaStream_t st)
{
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    Shape s1 = shape_of(dx, type, sms), s2 = shape_of(dw, type, sms);
    // in one launch where neither fills the GPU by itself and both fit it, two CTAs an SM
    const uint64_t t1 = up(dx.cols, kPTile) * up(dx.rows, s1.bn), t2 = up(dw.cols, kPTile) * up(dw.rows, s2.bn);
    while (t1 * s1.split + t2 * s2.split > 2ull * sms && (s1.split > 1 || s2.split > 1)) {
        uint32_t &s = t1 * s1.split > t2 * s2.split ? (s1.split > 1 ? s1.split : s2.split) : (s2.split > 1 ? s2.split : s1.split);
        s /= 2;
    }
    if (s1.pair || s2.pair || !dx.K || !dw.K || t1 * s1.split + t2 * s2.split > 2ull * sms) {
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
    void *args[] = {&a.pm, &a.qm, &a.g, &b.pm, &b.qm, &b.g, &n1};
    return launch_plan((const void *)gemm_both_kernel, kSplitThreads, ctas, cluster, std::max(m1, m2), args, behind, st);
}

} // namespace ecc
