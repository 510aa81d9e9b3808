// ecc_head_gemm.cu -- the matrix products' kernels for logits that are never
// stored: their softmax statistics, and their gradient as an operand of the
// backward products.

#include "ecc_gemm.cuh"

namespace ecc {

// The softmax statistics of a few tokens: the head's rows are the lanes, the
// tokens (up to bn of them) the accumulator's columns, and the CTAs stream the
// head through a ring of 128-row blocks, a CTA an SM.  A warp joins its 32
// lanes' logits of 16 tokens by exchanging halves (16 shuffles for a sum over
// the lanes of 16 values each) and keeps the running statistics of two lanes'
// token over all of its tiles.  Bound by HBM: with tokens as the lanes, as for
// many, the products of 128 tokens whatever their number take as long as the
// loads (8 x 131072 x 4096: 330 us, and 259 in the clusters' kernel, which
// starts a CTA for each 128 rows).
// the sum or maximum over the lanes of 16 values: lane l gets that of value l / 2
template <int N, typename Op> __device__ __forceinline__ void halve(float (&v)[16], uint32_t lane, Op op)
{
    const bool high = lane & (2 * N);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float got = __shfl_xor_sync(~0u, high ? v[i] : v[i + N], 2 * N);
        v[i] = op(high ? v[i + N] : v[i], got);
    }
}
template <typename Op> __device__ __forceinline__ float over_lanes(float (&v)[16], uint32_t lane, Op op)
{
    halve<8>(v, lane, op);
    halve<4>(v, lane, op);
    halve<2>(v, lane, op);
    halve<1>(v, lane, op);
    return op(v[0], __shfl_xor_sync(~0u, v[0], 1));
}

template <bool F8>
__global__ void __launch_bounds__(kStreamThreads, 1)
    stats_stream_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ StreamArgs g)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ StreamBars s;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage0 = (smem_u32(smem_raw) + kSmemHead - 1) & ~(kSmemHead - 1);
    const uint32_t stage_bytes = kPBytes + g.bn * kTileBytes;
    const uint32_t per = (g.kblocks + g.segs - 1) / g.segs, used = (g.kblocks + per - 1) / per; // segments of the reduction
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < g.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 4);
        }
        fence_mbar_init();
        fence_proxy_async();
    }
    if (threadIdx.x == 32) {
        prefetch_map(&wmap);
        prefetch_map(&xmap);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), 512);
        tmem_fence_before();
    }
    wait_for_previous();
    let_next_start();
    if (threadIdx.x < 64) {
        const int64_t t = g.e.tokens && threadIdx.x < g.tokens ? g.e.tokens[threadIdx.x] : -1;
        s.token[threadIdx.x] = t >= 0 && t < (int64_t)g.vocab ? (int32_t)t : -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *(volatile uint32_t *)g.status = ECC_OK;
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&s.tmem;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t st = 0, ph = 0, issued = 0;
            bool ok = true;
            for (uint32_t t = blockIdx.x; t < g.tiles && ok; t += gridDim.x)
                for (uint32_t kb = 0; kb < g.kblocks; ++kb) {
                    if (!(ok = mbar_wait(&s.empty[st], ph ^ 1, g.limit_ns)))
                        break;
                    const uint32_t at = stage0 + st * stage_bytes, bar = smem_u32(&s.full[st]);
                    mbar_expect_tx(&s.full[st], stage_bytes);
                    load_operand<1, false, F8>(at, &wmap, (uint64_t)t * kPTile, kPTile, kb, false, bar);
                    load_operand<1, false, F8>(at + kPBytes, &xmap, 0, g.bn, kb, false, bar);
                    ++issued;
                    if (++st == g.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            if (!ok) { // the copies in flight: a last wait each
                set_status(g.status, ECC_ERR_TIMEOUT);
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
        if (lane == 0) {
            uint32_t st = 0, ph = 0, acc = 0, aph = 0;
            bool ok = true;
            for (uint32_t t = blockIdx.x; t < g.tiles && ok; t += gridDim.x) {
                if (!(ok = mbar_wait(&s.tempty[acc], aph ^ 1, g.limit_ns)))
                    break;
                tmem_fence_after();
                uint32_t k = 0, d = tmem + acc * 256;
                for (uint32_t kb = 0; kb < g.kblocks; ++kb) {
                    if (!(ok = mbar_wait(&s.full[st], ph, g.limit_ns))) {
                        (void)mbar_wait(&s.full[st], ph, g.limit_ns);
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t at = stage0 + st * stage_bytes;
                    multiply_block<1, false, false, F8>(d, at, at + kPBytes, g.idesc, k == 0);
                    tensor_commit<1>(smem_u32(&s.empty[st]));
                    if (++k == per) {
                        k = 0;
                        d += g.bn;
                    }
                    if (++st == g.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                tensor_commit<1>(smem_u32(&s.tfull[acc]));
                if (acc)
                    aph ^= 1;
                acc ^= 1;
            }
            if (!ok)
                set_status(g.status, ECC_ERR_TIMEOUT);
        }
    } else {
        const uint32_t quad = warp & 3;
        const float scale = g.e.scale * 1.44269504f;
        LogitsPart p[4]; // of token 16 i + lane / 2
        uint32_t acc = 0, aph = 0;
        for (uint32_t t = blockIdx.x; t < g.tiles; t += gridDim.x) {
            if (!__all_sync(~0u, mbar_wait(&s.tfull[acc], aph, g.limit_ns))) {
                if (lane == 0)
                    set_status(g.status, ECC_ERR_TIMEOUT);
                break;
            }
            tmem_fence_after();
            const uint64_t v = (uint64_t)t * kPTile + quad * 32 + lane;
            const bool ok = v < g.vocab;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                if (i * 16 >= g.bn)
                    continue;
                float y[16], m[16], x[16], d[16];
                const uint32_t at = tmem + (quad * 32 << 16) + acc * 256 + i * 16;
                tmem_load16(at, y);
                for (uint32_t k = 1; k < used; ++k) {
                    float more[16];
                    tmem_load16(at + k * g.bn, more);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        y[j] += more[j];
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    y[j] *= scale;
                    m[j] = ok ? y[j] : -INFINITY;
                    if (ok && s.token[i * 16 + j] == (int32_t)v)
                        g.e.token_logit[i * 16 + j] = y[j];
                }
                const float top = over_lanes(m, lane, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float r = y[j] - __shfl_sync(~0u, top, 2 * j);
                    x[j] = ok ? exp2_approx(r) : 0.f;
                    d[j] = ok ? x[j] * r : 0.f;
                }
                auto add = [](float a, float b) { return a + b; };
                const float sum = over_lanes(x, lane, add), ent = over_lanes(d, lane, add);
                if (sum != 0.f) { // (0: no row of the vocabulary among them)
                    const float most = fmaxf(p[i].m, top), old = p[i].s > 0.f ? p[i].m - most : 0.f, now = top - most;
                    const float ro = exp2_approx(old), rn = exp2_approx(now);
                    p[i].t = ro * fmaf(old, p[i].s, p[i].t) + rn * fmaf(now, sum, ent);
                    p[i].s = p[i].s * ro + sum * rn;
                    p[i].m = most;
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&s.tempty[acc])) : "memory");
            if (acc)
                aph ^= 1;
            acc ^= 1;
        }
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t c = i * 16 + lane / 2;
            if (!(lane & 1) && c < g.tokens && i * 16 < g.bn)
                g.e.part[((uint64_t)blockIdx.x * 4 + quad) * g.tokens + c] = make_float4(p[i].m, p[i].s, p[i].t, 0.f);
        }
    }
    __syncthreads();
    __syncwarp();
    tmem_fence_after();
    if (warp == 1)
        tmem_free<1>(tmem, 512);
}

const void *stats_stream(bool f8) { return f8 ? (const void *)stats_stream_kernel<true> : (const void *)stats_stream_kernel<false>; }

const void *stats_kernel(bool f8, bool pair)
{
    return f8 ? gemm_kernel<false, false, true, kStats>(pair) : gemm_kernel<false, false, false, kStats>(pair);
}
const void *slopes_kernel(bool pair) { return gemm_kernel<false, false, false, kSlopes>(pair); }

} // namespace ecc
