// ecc_gated.cu -- the gated feed-forward projections, out = act(g) * u with g =
// scale x w_gate^T + bias_gate and u = up_scale x w_up^T + bias_up, and their
// backward pass.
//
// Forward: one matrix product whose P rows are the two weights' in turns
// (ecc_gemm.cuh, kGated), so that x is read once for both and neither g nor u
// goes through memory unless it is wanted.  Backward: one elementwise kernel
// makes tg = dy u act'(g) and tu = dy act(g) side by side, [M, 2 N'] with N' = N
// rounded up to the products' block of 64 (float16: to 128, and twice, by powers
// of two that another kernel finds); dx is one product whose reduction runs over
// both weights (kDual), both weights' gradients are the rows of another one.
//
// 8192 x 16384 x 4096 bf16 with g and u kept takes 1.20 ms in a burst (1.83
// PFLOP/s, the tensor pipe 89% active), 1.37 ms under the power limit; one token
// of 16384 x 4096 44.8 us (6.0 TB/s); the backward pass of 8192 x 8192 x 4096 1.46
// ms, of which the elementwise kernel is 0.11 (HBM).

#include <cmath>

#include "ecc_linear.cuh"

namespace ecc {

// What tg and tu are rounded to.  bfloat16 has float32's exponents: both halves
// of one t, each times its scale's share of the larger scale, for all three
// products.  float16 has not: a product dy u may leave its range, or lose its
// bits below it, where dx and the weights' gradients are ordinary numbers.  So
// gated_range_kernel finds the largest |tg| and |tu| first, and a power of two
// brings the largest value of an operand to 2^14.  dx's operand (t) needs one
// power for both halves, since its reduction runs over them; the weights'
// gradients are different rows of theirs (tw), and each half has its own power
// there, so that the smaller one of very unequal halves keeps its bits too.
// (8192 x 8192 x 4096 float16 1.50 ms, 257 x 1000 x 771 31 us, both with cold caches;
// with one t in float16's own range 1.37 ms and 28 us.)
struct GatedSlopeParams {
    const void *dy, *gate, *up;
    void *t, *tw; // [M, 2 * np], for dx and (float16) for the weights' gradients; NULL: not wanted
    float *part;  // [parts][2 * N]; NULL: no sums
    uint64_t M, N, np, lddy, ldgate, ldup;
    float gate_factor, up_factor; // of t's two halves
    uint32_t act, parts;
    uint32_t *status;
    float2 *range; // float16: a block's largest |tg| and |tu|, of `ranges` blocks
    uint32_t ranges;
    float *factor; // float16: the inverse powers of two of t, of tw's gates and of its ups
};

// tg and tu of 2 H values, in place of g and u
template <int H>
__device__ __forceinline__ void gated_slopes(uint32_t by, const float2 (&v)[H], float2 (&g)[H], float2 (&u)[H])
{
    auto each = [&](auto act) {
        constexpr uint32_t ACT = decltype(act)::value;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 slope = act_slope2<ACT>(g[i]), value = act_value2<ACT>(g[i]);
            g[i] = mul2(mul2(v[i], u[i]), slope);
            u[i] = mul2(v[i], value);
        }
    };
    if (by == ECC_ACT_RELU)
        each(std::integral_constant<uint32_t, ECC_ACT_RELU>());
    else if (by == ECC_ACT_GELU)
        each(std::integral_constant<uint32_t, ECC_ACT_GELU>());
    else if (by == ECC_ACT_GELU_TANH)
        each(std::integral_constant<uint32_t, ECC_ACT_GELU_TANH>());
    else if (by == ECC_ACT_SILU)
        each(std::integral_constant<uint32_t, ECC_ACT_SILU>());
    else
        each(std::integral_constant<uint32_t, ECC_ACT_NONE>());
}

// the larger one of x and a finite |v|
__device__ __forceinline__ float finite_max(float x, float v) { return fabsf(v) < INFINITY ? fmaxf(x, fabsf(v)) : x; }
// the block's largest values, in every thread (called by all of them)
__device__ __forceinline__ float2 block_range(float2 top)
{
    __shared__ float2 s[kRowThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        top.x = fmaxf(top.x, __shfl_xor_sync(~0u, top.x, o));
        top.y = fmaxf(top.y, __shfl_xor_sync(~0u, top.y, o));
    }
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; ++i)
        top = make_float2(fmaxf(top.x, s[i].x), fmaxf(top.y, s[i].y));
    return top;
}

// The largest |tg| and |tu| that are finite, a pair for each block.  Pieces of
// 32 * V columns and 16 rows (two a warp) in turns, so that a small layer has
// blocks enough: 257 x 1000 takes 2.7 us (5.2 in pieces of 64 rows),
// 8192 x 8192 71 us, 5.6 TB/s.
constexpr uint32_t kRangeBlocks = 608, kRangeRows = 16; // four blocks an SM
template <typename T, typename PT, int V>
__global__ void __launch_bounds__(kRowThreads) gated_range_kernel(const __grid_constant__ GatedSlopeParams p)
{
    constexpr int H = (V + 1) / 2;
    let_next_start();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    // (32 bits count the pieces: each is 512 values or more)
    const uint32_t across = (uint32_t)((p.N + 32 * V - 1) / (32 * V)), pieces = across * (uint32_t)((p.M + kRangeRows - 1) / kRangeRows);
    float2 top = both(0.f);
    for (uint32_t i = blockIdx.x; i < pieces; i += gridDim.x) {
        const uint64_t c = (uint64_t)(i % across * 32 + tx) * V, r0 = (uint64_t)(i / across) * kRangeRows, r1 = min(p.M, r0 + kRangeRows);
        if (c >= p.N)
            continue;
#pragma unroll 2
        for (uint64_t r = r0 + ty; r < r1; r += 8) {
            float2 v[H], g[H], u[H];
            load_values<T, V>(p.dy, r * p.lddy + c, v);
            load_values<PT, V>(p.gate, r * p.ldgate + c, g);
            load_values<PT, V>(p.up, r * p.ldup + c, u);
            gated_slopes(p.act, v, g, u);
#pragma unroll
            for (int k = 0; k < H; ++k) {
                top.x = finite_max(finite_max(top.x, g[k].x), g[k].y);
                top.y = finite_max(finite_max(top.y, u[k].x), u[k].y);
            }
        }
    }
    top = block_range(top);
    if (threadIdx.x == 0)
        p.range[blockIdx.x] = top;
    // (launched behind the padding: whatever waits for this kernel waits for both)
    wait_for_previous();
}

// a block: 32 * V columns, one share of the rows, eight warps a row each
template <typename T, typename PT, int V>
__global__ void __launch_bounds__(kRowThreads) gated_slope_kernel(const __grid_constant__ GatedSlopeParams p)
{
    constexpr int H = (V + 1) / 2, W = V == 1 ? 1 : 2; // pairs; values used of a pair
    __shared__ float sums[8][2 * 32 * V + 1];
    let_next_start();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *p.status = ECC_OK;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const uint64_t c = ((uint64_t)blockIdx.x * 32 + tx) * V;
    const uint64_t per = (p.M + p.parts - 1) / p.parts, r0 = blockIdx.y * per, r1 = min(p.M, r0 + per);
    float gate_factor = p.gate_factor, up_factor = p.up_factor;
    float2 tw_factor = both(1.f);
    if constexpr (std::is_same_v<T, __half>) {
        if (p.range) {
            wait_for_previous();
            float2 top = both(0.f);
            for (uint32_t i = threadIdx.x; i < p.ranges; i += kRowThreads)
                top = make_float2(fmaxf(top.x, p.range[i].x), fmaxf(top.y, p.range[i].y));
            top = block_range(top);
            const int kt = half_power(fmaxf(fabsf(gate_factor) * top.x, fabsf(up_factor) * top.y));
            const int kg = half_power(top.x), ku = half_power(top.y);
            gate_factor *= ldexpf(1.f, kt);
            up_factor *= ldexpf(1.f, kt);
            tw_factor = make_float2(ldexpf(1.f, kg), ldexpf(1.f, ku));
            if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 3)
                p.factor[threadIdx.x] = ldexpf(1.f, threadIdx.x == 0 ? -kt : threadIdx.x == 1 ? -kg : -ku);
        }
    }
    float2 sg[H], su[H];
#pragma unroll
    for (int i = 0; i < H; ++i)
        sg[i] = su[i] = both(0.f);
    if (c < p.np)
#pragma unroll 2
        for (uint64_t r = r0 + ty; r < r1; r += 8) {
            float2 v[H], g[H], u[H];
            if (c < p.N) {
                load_values<T, V>(p.dy, r * p.lddy + c, v);
                load_values<PT, V>(p.gate, r * p.ldgate + c, g);
                load_values<PT, V>(p.up, r * p.ldup + c, u);
                gated_slopes(p.act, v, g, u);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    sg[i] = add2(sg[i], g[i]);
                    su[i] = add2(su[i], u[i]);
                }
            } else { // the halves' ends, which the products read
#pragma unroll
                for (int i = 0; i < H; ++i)
                    g[i] = u[i] = both(0.f);
            }
            auto store = [&](void *t, float fg, float fu) {
                float2 a[H], b[H];
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    a[i] = mul2(g[i], both(fg));
                    b[i] = mul2(u[i], both(fu));
                }
                T *o = static_cast<T *>(t) + r * 2 * p.np + c;
                if constexpr (V == 1) {
                    *o = from_f32<T>(a[0].x);
                    o[p.np] = from_f32<T>(b[0].x);
                } else {
                    *reinterpret_cast<uint4 *>(o) = pack2<T>(a);
                    *reinterpret_cast<uint4 *>(o + p.np) = pack2<T>(b);
                }
            };
            if (p.t)
                store(p.t, gate_factor, up_factor);
            if constexpr (std::is_same_v<T, __half>)
                if (p.tw)
                    store(p.tw, tw_factor.x, tw_factor.y);
        }
    // (launched behind the padding, which it does not read: whatever waits for this kernel waits for both)
    wait_for_previous();
    if (!p.part)
        return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sums[ty][tx + 32 * i] = i % W ? sg[i / 2].y : sg[i / W].x;
        sums[ty][32 * V + tx + 32 * i] = i % W ? su[i / 2].y : su[i / W].x;
    }
    __syncthreads();
    for (uint32_t k = threadIdx.x; k < 2 * 32 * V; k += kRowThreads) {
        const uint32_t half = k / (32 * V), i = k % (32 * V);
        const uint64_t at = (uint64_t)blockIdx.x * 32 * V + (i & 31) * V + (i >> 5);
        if (at < p.N) {
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 8; ++y)
                sum += sums[y][k];
            p.part[blockIdx.y * 2 * p.N + half * p.N + at] = sum;
        }
    }
}

namespace {

constexpr uint32_t kGatedParts = 64; // partial column sums at most

bool gated_ok(const ecc_gated_linear_job &j)
{
    if ((j.in_type != ECC_BF16 && j.in_type != ECC_F16 && j.in_type != ECC_E4M3) || j.act > ECC_ACT_SILU || j.reserved ||
        !(wide_type(j.out_type) || j.out_type == ECC_E4M3) || !std::isfinite(j.scale) || !std::isfinite(j.up_scale) ||
        !std::isfinite(j.out_scale) || (j.out_type != ECC_E4M3 && j.out_scale != 1.f) || j.M >= kMostDim || j.N >= kMostDim ||
        j.K >= kMostDim)
        return false;
    if (!j.M || !j.N)
        return true;
    if (!j.out || j.ldout < j.N || !aligned_to(j.out, j.out_type))
        return false;
    if (j.K && (!j.x || !j.w_gate || !j.w_up || j.ldx < j.K || j.ldgate < j.K || j.ldup < j.K || !aligned_to(j.x, j.in_type) ||
                !aligned_to(j.w_gate, j.in_type) || !aligned_to(j.w_up, j.in_type)))
        return false;
    if ((j.bias_gate || j.bias_up) &&
        (!wide_type(j.bias_type) || !aligned_to(j.bias_gate, j.bias_type) || !aligned_to(j.bias_up, j.bias_type)))
        return false;
    if (!j.pre_gate && !j.pre_up)
        return true;
    return j.pre_gate && j.pre_up && wide_type(j.pre_type) && j.ldpre_gate >= j.N && j.ldpre_up >= j.N &&
           aligned_to(j.pre_gate, j.pre_type) && aligned_to(j.pre_up, j.pre_type);
}

// few_rows_kernel in place of the tensor cores' kernels, by the rule of the
// linear layer over both weights together (16384 x 4096 bf16 one token 45.2 us,
// 8 by the tensor cores 46.0; e4m3 26.8 by the tensor cores)
bool gated_few_rows(const ecc_gated_linear_job &j)
{
    if (j.M > 4 || !j.K)
        return false;
    if (2 * j.N * j.K <= 1ull << 22)
        return true;
    return j.in_type != ECC_E4M3 && (j.M == 1 || (j.M == 2 && !(tma_rows(j.w_gate, j.ldgate, j.in_type, j.N) &&
                                                                tma_rows(j.w_up, j.ldup, j.in_type, j.N))));
}

bool gated_grad_ok(const ecc_gated_linear_grad_job &j)
{
    if ((j.in_type != ECC_BF16 && j.in_type != ECC_F16) || j.act > ECC_ACT_SILU || !std::isfinite(j.scale) ||
        !std::isfinite(j.up_scale) || j.M >= kMostDim || j.N >= kMostDim || j.K >= kMostDim || !j.dw_gate != !j.dw_up ||
        !j.dbias_gate != !j.dbias_up || (j.dw_gate && j.dw_type != j.in_type && j.dw_type != ECC_F32))
        return false;
    if (j.M && j.N &&
        (!j.dy || j.lddy < j.N || !aligned_to(j.dy, j.in_type) || !j.pre_gate || !j.pre_up || !wide_type(j.pre_type) ||
         j.ldpre_gate < j.N || j.ldpre_up < j.N || !aligned_to(j.pre_gate, j.pre_type) || !aligned_to(j.pre_up, j.pre_type)))
        return false;
    if (j.dx && j.M && j.K &&
        (j.lddx < j.K || !aligned_to(j.dx, j.in_type) ||
         (j.N && (!j.w_gate || !j.w_up || j.ldgate < j.K || j.ldup < j.K || !aligned_to(j.w_gate, j.in_type) ||
                  !aligned_to(j.w_up, j.in_type)))))
        return false;
    if (j.dw_gate && j.N && j.K &&
        (j.lddw_gate < j.K || j.lddw_up < j.K || !aligned_to(j.dw_gate, j.dw_type) || !aligned_to(j.dw_up, j.dw_type) ||
         (j.M && (!j.x || j.ldx < j.K || !aligned_to(j.x, j.in_type)))))
        return false;
    return aligned_to(j.dbias_gate, ECC_F32) && aligned_to(j.dbias_up, ECC_F32);
}

struct GatedGradPlan {
    uint64_t np; // columns of a half of t
    uint32_t parts;
    bool own_tw; // float16: the weights' gradients have an operand of their own
    size_t t_bytes, tw_bytes, range_bytes, part_bytes, bytes;
};
GatedGradPlan gated_grad_plan(const ecc_gated_linear_grad_job &j)
{
    GatedGradPlan g{};
    g.own_tw = j.in_type == ECC_F16;
    const uint64_t whole = g.own_tw ? 128 : 64; // the weights' gradients have a scale each: no half of a tile has rows of both
    g.np = (j.N + whole - 1) / whole * whole;
    const size_t t = pad256(j.M * 2 * g.np * type_bytes(j.in_type));
    g.t_bytes = j.dx || (j.dw_gate && !g.own_tw) ? t : 0;
    g.tw_bytes = j.dw_gate && g.own_tw ? t : 0;
    g.range_bytes = g.own_tw && g.t_bytes + g.tw_bytes ? 256 + pad256(kRangeBlocks * sizeof(float2)) : 0;
    // 64 rows a block, or down to 16 (two a warp) while there are fewer blocks than about two an SM: 257 x 1000
    // takes 11 us on 16 blocks
    const uint64_t across = (j.N + 255) / 256;
    g.parts = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>({kGatedParts, std::max(j.M / 64, 304 / std::max<uint64_t>(across, 1)), j.M / 16}));
    g.part_bytes = j.dbias_gate ? pad256(g.parts * 2 * j.N * sizeof(float)) : 0;
    g.bytes = g.t_bytes + g.tw_bytes + g.range_bytes + g.part_bytes;
    if (j.dx)
        g.bytes += copy_bytes(j.w_gate, j.ldgate, j.N, j.K, j.in_type) + copy_bytes(j.w_up, j.ldup, j.N, j.K, j.in_type);
    if (j.dw_gate)
        g.bytes += copy_bytes(j.x, j.ldx, j.M, j.K, j.in_type);
    return g;
}

template <typename T, typename PT> ecc_status gated_slope_launch(const GatedSlopeParams &p, bool behind, cudaStream_t st)
{
    const auto whole = [](const void *q, uint64_t ld, size_t size) { return ((uintptr_t)q & 15) == 0 && ld * size % 16 == 0; };
    // eight values a load where the rows allow it
    const bool v8 = p.N % 8 == 0 && whole(p.dy, p.lddy, sizeof(T)) && whole(p.gate, p.ldgate, sizeof(PT)) &&
                    whole(p.up, p.ldup, sizeof(PT));
    auto launch = [&](auto f, dim3 grid) {
        if (behind)
            return launch_status(launch_behind(f, grid, kRowThreads, 0, st, p));
        f<<<grid, kRowThreads, 0, st>>>(p);
        return launch_status(cudaGetLastError());
    };
    if constexpr (std::is_same_v<T, __half>) {
        if (p.range) {
            const ecc_status rc = launch(v8 ? gated_range_kernel<T, PT, 8> : gated_range_kernel<T, PT, 1>, dim3(p.ranges));
            if (rc != ECC_OK)
                return rc;
            behind = true;
        }
    }
    const uint64_t per = v8 ? 256 : 32;
    return launch(v8 ? gated_slope_kernel<T, PT, 8> : gated_slope_kernel<T, PT, 1>, dim3((unsigned)((p.np + per - 1) / per), p.parts));
}
template <typename T> ecc_status gated_slope_launch(const GatedSlopeParams &p, uint32_t pre_type, bool behind, cudaStream_t st)
{
    return pre_type == ECC_F32    ? gated_slope_launch<T, float>(p, behind, st)
           : pre_type == ECC_BF16 ? gated_slope_launch<T, bf16>(p, behind, st)
                                  : gated_slope_launch<T, __half>(p, behind, st);
}

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

size_t ecc_gated_linear_workspace_bytes(const ecc_gated_linear_job *job)
{
    if (!job || !job->M || !job->N || !job->K || gated_few_rows(*job))
        return 0;
    return copy_bytes(job->x, job->ldx, job->M, job->K, job->in_type) +
           copy_bytes(job->w_gate, job->ldgate, job->N, job->K, job->in_type) +
           copy_bytes(job->w_up, job->ldup, job->N, job->K, job->in_type);
}

ecc_status ecc_gated_linear(const ecc_gated_linear_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !gated_ok(*job))
        return ECC_ERR_ARG;
    const ecc_gated_linear_job &j = *job;
    cudaStream_t st = (cudaStream_t)stream;
    if (!j.M || !j.N)
        return launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    const size_t need = ecc_gated_linear_workspace_bytes(job);
    if (need && (!ws || !aligned16(ws) || ws_bytes < need))
        return ECC_ERR_ARG;
    Epilogue e{};
    e.bias = j.bias_gate;
    e.out = j.out;
    e.pre = j.pre_gate;
    e.ldout = j.ldout;
    e.ldpre = j.ldpre_gate;
    e.scale = j.scale;
    e.out_scale = j.out_scale;
    e.bias_type = j.bias_type;
    e.out_type = j.out_type;
    e.pre_type = j.pre_type;
    e.act = j.act;
    e.bias2 = j.bias_up;
    e.pre2 = j.pre_up;
    e.ldpre2 = j.ldpre_up;
    e.scale2 = j.up_scale;
    if (gated_few_rows(j)) {
        const int sms = sm_count();
        if (sms <= 0)
            return ECC_ERR_CUDA;
        const FewRows p{j.x, j.w_gate, j.ldx, j.ldgate, j.N, j.K, 1, e, status, j.w_up, j.ldup};
        if (j.in_type == ECC_BF16)
            few_rows_launch<bf16, true>(j.M, p, sms, st);
        else if (j.in_type == ECC_F16)
            few_rows_launch<__half, true>(j.M, p, sms, st);
        else
            few_rows_launch<e4m3, true>(j.M, p, sms, st);
        return launch_status(cudaGetLastError());
    }
    uint8_t *w = (uint8_t *)ws;
    Product p{};
    bool copied;
    const ecc_status rc = readable({{j.x, j.ldx, j.M, j.K, &p.Q}, {j.w_gate, j.ldgate, j.N, j.K, &p.P}, {j.w_up, j.ldup, j.N, j.K, &p.P2}},
                                   j.in_type, w, st, copied);
    if (rc != ECC_OK)
        return rc;
    p.rows = j.M;
    p.cols = j.N;
    p.K = j.K;
    p.e = e;
    p.mode = kGated;
    return gemm(p, j.in_type, status, true, copied, st);
}

size_t ecc_gated_linear_grad_workspace_bytes(const ecc_gated_linear_grad_job *job)
{
    return job ? gated_grad_plan(*job).bytes : 0;
}

ecc_status ecc_gated_linear_grad(const ecc_gated_linear_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !gated_grad_ok(*job))
        return ECC_ERR_ARG;
    const ecc_gated_linear_grad_job &j = *job;
    const GatedGradPlan g = gated_grad_plan(j);
    if (g.bytes && (!ws || !aligned16(ws) || ws_bytes < g.bytes))
        return ECC_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *w = (uint8_t *)ws;
    void *t = g.t_bytes ? w : nullptr;
    w += g.t_bytes;
    void *tw = g.tw_bytes ? w : nullptr;
    w += g.tw_bytes;
    float *factor = g.range_bytes && (t || tw) ? (float *)w : nullptr; // three, then the ranges
    float2 *range = factor ? (float2 *)(w + 256) : nullptr;
    w += g.range_bytes;
    float *part = j.dbias_gate ? (float *)w : nullptr;
    w += g.part_bytes;
    // read down their columns
    Product dx{}, dw{};
    bool own;
    ecc_status rc = readable({{j.x, j.ldx, j.dw_gate ? j.M : 0, j.K, &dw.P},
                              {j.w_gate, j.ldgate, j.dx ? j.N : 0, j.K, &dx.P},
                              {j.w_up, j.ldup, j.dx ? j.N : 0, j.K, &dx.P2}},
                             j.in_type, w, st, own);
    if (rc != ECC_OK)
        return rc;
    dw.P.mn = dx.P.mn = dx.P2.mn = true;
    // the products' common scale is the larger one; t's halves carry what is left
    const float scale = std::max(std::fabs(j.scale), std::fabs(j.up_scale)), inv = scale > 0.f ? 1.f : 0.f;
    const bool slope = j.N && (t || tw || part);
    if (slope) {
        // (a block of the range kernel for each of its pieces, or as many as there are places)
        const uint64_t pieces = (j.N + 31) / 32 * ((j.M + kRangeRows - 1) / kRangeRows);
        const GatedSlopeParams p{j.dy, j.pre_gate, j.pre_up, t, tw, part, j.M, j.N, g.np, j.lddy, j.ldpre_gate, j.ldpre_up,
                                 inv > 0.f ? j.scale / scale : 0.f, inv > 0.f ? j.up_scale / scale : 0.f, j.act, g.parts, status,
                                 range, (uint32_t)std::min<uint64_t>(pieces, kRangeBlocks), factor};
        rc = j.in_type == ECC_BF16 ? gated_slope_launch<bf16>(p, j.pre_type, own, st)
                                   : gated_slope_launch<__half>(p, j.pre_type, own, st);
        own = true;
    }
    bool clear = !slope; // status: cleared by t's kernel, or by a product, or by itself
    dx.Q = {t, 2 * g.np, false};
    dx.rows = j.M;
    dx.cols = j.K;
    dx.K = 2 * g.np;
    dx.mode = kDual;
    dx.kswitch = g.np;
    dx.kfirst = j.N;
    dx.e.out = j.dx;
    dx.e.ldout = j.lddx;
    dx.e.out_type = j.in_type;
    dw.Q = {g.own_tw ? tw : t, 2 * g.np, true};
    dw.rows = 2 * g.np;
    dw.cols = j.K;
    dw.K = j.M;
    dw.e.out = j.dw_gate;
    dw.e.ldout = j.lddw_gate;
    dw.e.out_type = j.dw_type;
    dw.e.out2 = j.dw_up;
    dw.e.ldout2 = j.lddw_up;
    dw.e.rswitch = g.np;
    dw.e.rows2 = j.N;
    dx.e.scale = scale;
    dw.e.scale = g.own_tw ? j.scale : scale;
    dw.e.scale2 = g.own_tw ? j.up_scale : scale;
    dx.e.factor = factor;
    dw.e.factor = factor ? factor + 1 : nullptr;
    dx.e.out_scale = dw.e.out_scale = 1.f;
    const bool want_dx = j.dx && j.M && j.K, want_dw = j.dw_gate && j.N && j.K;
    if (rc == ECC_OK && want_dx && want_dw)
        rc = gemm_backward(dx, dw, j.in_type, status, clear, own, st);
    else if (rc == ECC_OK && (want_dx || want_dw))
        rc = gemm(want_dx ? dx : dw, j.in_type, status, clear, own, st);
    if (want_dx || want_dw)
        clear = false;
    if (rc == ECC_OK && slope && part)
        rc = launch_status(launch_behind(sum_parts_kernel, dim3((unsigned)((2 * j.N + kRowThreads - 1) / kRowThreads)), kRowThreads, 0,
                                         st, (const float *)part, g.parts, 2 * j.N, j.dbias_gate, j.N, j.dbias_up));
    if (rc == ECC_OK && clear)
        rc = launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    return rc;
}

} // extern "C"
