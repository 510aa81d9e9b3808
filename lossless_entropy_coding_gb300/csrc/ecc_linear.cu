// ecc_linear.cu -- a layer's matrix product with its epilogue (scale, bias,
// activation, residual), and its backward pass: t = dy * act'(pre) with the
// bias gradient, then the two products (ecc_gemm.cu).
//
// The products read their operands by TMA, which wants rows on 16-byte
// boundaries: an operand with other rows is first copied to the workspace
// with padded rows.  Products of a few rows read theirs as they lie.

#include <algorithm>
#include <cmath>

#include "ecc_linear.cuh"

namespace ecc {

constexpr uint32_t kSlopeParts = 64; // partial column sums of t at most

// t = dy * act'(pre), rounded to the operand type (the tensor cores' input);
// the column sums of t before that rounding
struct SlopeParams {
    const void *dy, *pre;
    void *t;     // [M, ldt]; NULL: only the sums
    float *part; // [parts][N]; NULL: no sums
    uint64_t M, N, lddy, ldpre, ldt;
    uint32_t act, parts;
    uint32_t *status;
};

// a block: 32 * V columns, one share of the rows, eight warps a row each
template <typename T, typename PT, int V, uint32_t ACT>
__global__ void __launch_bounds__(kRowThreads) slope_kernel(SlopeParams p)
{
    constexpr int H = (V + 1) / 2, W = V == 1 ? 1 : 2; // pairs; values used of a pair
    __shared__ float sums[8][32 * V + 1];
    let_next_start();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *p.status = ECC_OK;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const uint64_t c = ((uint64_t)blockIdx.x * 32 + tx) * V;
    const uint64_t per = (p.M + p.parts - 1) / p.parts, r0 = blockIdx.y * per, r1 = min(p.M, r0 + per);
    float2 s[H];
#pragma unroll
    for (int i = 0; i < H; ++i)
        s[i] = both(0.f);
    if (c < p.N)
#pragma unroll 2
        for (uint64_t r = r0 + ty; r < r1; r += 8) {
            float2 v[H];
            load_values<T, V>(p.dy, r * p.lddy + c, v);
            if constexpr (ACT != ECC_ACT_NONE) {
                float2 a[H];
                load_values<PT, V>(p.pre, r * p.ldpre + c, a);
#pragma unroll
                for (int i = 0; i < H; ++i) { // (the sum fused, so that it is the same with and without t)
                    a[i] = act_slope2<ACT>(a[i]);
                    s[i] = fma2(v[i], a[i], s[i]);
                    v[i] = mul2(v[i], a[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i)
                    s[i] = add2(s[i], v[i]);
            }
            if (p.t) {
                T *o = static_cast<T *>(p.t) + r * p.ldt + c;
                if constexpr (V == 1)
                    *o = from_f32<T>(v[0].x);
                else
                    *reinterpret_cast<uint4 *>(o) = pack2<T>(v);
            }
        }
    // (launched behind the padding, which it does not read: whatever waits for this kernel waits for both)
    wait_for_previous();
    if (!p.part)
        return;
#pragma unroll
    for (int i = 0; i < V; ++i)
        sums[ty][tx + 32 * i] = i % W ? s[i / 2].y : s[i / W].x;
    __syncthreads();
    for (uint64_t k = threadIdx.x; k < 32 * V; k += kRowThreads) {
        const uint64_t at = (uint64_t)blockIdx.x * 32 * V + (k & 31) * V + (k >> 5);
        if (at < p.N) {
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 8; ++y)
                sum += sums[y][k];
            p.part[blockIdx.y * p.N + at] = sum;
        }
    }
}

namespace {

// Which products few_rows_kernel takes, in place of the tensor cores' kernels
// (with the padding copy they need off 16-byte boundaries), us on both sides:
// one token's with 16-bit weights, 1 x 16384 x 4096 25.5 and 27.0, 1 x 4096 x
// 4096 8.2 and 12.3, 1 x 4096 x 4097 14.3 and 20.5; two rows off boundaries,
// 2 x 4096 x 4097 22.5 and 28.7 (on them 2 x 4096 x 4096 14.4 and 12.3); up to
// four of a small layer, 4 x 2048 x 2048 8.2 and 12.3 (4 x 4096 x 4096 18.5
// and 12.3).  (8-bit weights convert slower: 1 x 16384 x 4096 22 and 16.5.)
bool few_rows(const ecc_linear_job &j)
{
    if (j.M > 4 || !j.K)
        return false;
    if (j.N * j.K <= 1ull << 22)
        return true;
    return j.in_type != ECC_E4M3 && (j.M == 1 || (j.M == 2 && !tma_rows(j.w, j.ldw, j.in_type, j.N)));
}
bool linear_ok(const ecc_linear_job &j)
{
    if ((j.in_type != ECC_BF16 && j.in_type != ECC_F16 && j.in_type != ECC_E4M3) || j.act > ECC_ACT_SILU ||
        !(wide_type(j.out_type) || j.out_type == ECC_E4M3) || !std::isfinite(j.scale) || !std::isfinite(j.out_scale) ||
        (j.out_type != ECC_E4M3 && j.out_scale != 1.f) || j.M >= kMostDim || j.N >= kMostDim || j.K >= kMostDim)
        return false;
    if (!j.M || !j.N)
        return true;
    if (!j.out || j.ldout < j.N || !aligned_to(j.out, j.out_type))
        return false;
    if (j.K && (!j.x || !j.w || j.ldx < j.K || j.ldw < j.K || !aligned_to(j.x, j.in_type) ||
                !aligned_to(j.w, j.in_type)))
        return false;
    if (j.bias && (!wide_type(j.bias_type) || !aligned_to(j.bias, j.bias_type)))
        return false;
    if (j.residual && (!wide_type(j.res_type) || j.ldres < j.N || !aligned_to(j.residual, j.res_type) ||
                       (j.residual == j.out && (j.res_type != j.out_type || j.ldres != j.ldout))))
        return false;
    return !j.pre || (wide_type(j.pre_type) && j.ldpre >= j.N && aligned_to(j.pre, j.pre_type));
}

bool grad_ok(const ecc_linear_grad_job &j)
{
    if ((j.in_type != ECC_BF16 && j.in_type != ECC_F16) || j.act > ECC_ACT_SILU || !std::isfinite(j.scale) ||
        j.M >= kMostDim || j.N >= kMostDim || j.K >= kMostDim ||
        (j.dw && j.dw_type != j.in_type && j.dw_type != ECC_F32))
        return false;
    if (j.M && j.N && (!j.dy || j.lddy < j.N || !aligned_to(j.dy, j.in_type)))
        return false;
    if (j.M && j.N && j.act != ECC_ACT_NONE &&
        (!j.pre || !wide_type(j.pre_type) || j.ldpre < j.N || !aligned_to(j.pre, j.pre_type)))
        return false;
    if (j.dx && j.M && j.K &&
        (j.lddx < j.K || !aligned_to(j.dx, j.in_type) || (j.N && (!j.w || j.ldw < j.K || !aligned_to(j.w, j.in_type)))))
        return false;
    if (j.dw && j.N && j.K &&
        (j.lddw < j.K || !aligned_to(j.dw, j.dw_type) || (j.M && (!j.x || j.ldx < j.K || !aligned_to(j.x, j.in_type)))))
        return false;
    return aligned_to(j.dbias, ECC_F32);
}

struct GradPlan {
    bool make_t;      // t does not lie readable in dy
    uint64_t ldt;
    uint32_t parts;
    size_t t_bytes, part_bytes, bytes;
};
GradPlan grad_plan(const ecc_linear_grad_job &j)
{
    GradPlan g{};
    const bool products = j.dx || j.dw;
    g.make_t = products && (j.act != ECC_ACT_NONE || !tma_rows(j.dy, j.lddy, j.in_type, j.M));
    g.ldt = g.make_t ? padded(j.N, j.in_type) : j.lddy;
    g.t_bytes = g.make_t ? pad256(j.M * g.ldt * type_bytes(j.in_type)) : 0;
    g.parts = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(kSlopeParts, j.M / 64));
    g.part_bytes = j.dbias ? pad256(g.parts * j.N * sizeof(float)) : 0;
    g.bytes = g.t_bytes + g.part_bytes;
    if (j.dx && j.N)
        g.bytes += copy_bytes(j.w, j.ldw, j.N, j.K, j.in_type);
    if (j.dw && j.M)
        g.bytes += copy_bytes(j.x, j.ldx, j.M, j.K, j.in_type);
    return g;
}

template <typename T, typename PT, int V> auto slope_of(uint32_t act)
{
    return act == ECC_ACT_NONE    ? slope_kernel<T, PT, V, ECC_ACT_NONE>
           : act == ECC_ACT_RELU  ? slope_kernel<T, PT, V, ECC_ACT_RELU>
           : act == ECC_ACT_GELU  ? slope_kernel<T, PT, V, ECC_ACT_GELU>
           : act == ECC_ACT_SILU  ? slope_kernel<T, PT, V, ECC_ACT_SILU>
                                  : slope_kernel<T, PT, V, ECC_ACT_GELU_TANH>;
}
template <typename T, typename PT> ecc_status slope_launch(const SlopeParams &p, bool behind, cudaStream_t st)
{
    const auto whole = [](const void *q, uint64_t ld, size_t size) { return ((uintptr_t)q & 15) == 0 && ld * size % 16 == 0; };
    // eight values a load where the rows allow it
    const bool v8 = p.N % 8 == 0 && whole(p.dy, p.lddy, sizeof(T)) && (!p.t || whole(p.t, p.ldt, sizeof(T))) &&
                    (p.act == ECC_ACT_NONE || whole(p.pre, p.ldpre, sizeof(PT)));
    const uint64_t per = v8 ? 256 : 32;
    const dim3 grid((unsigned)((p.N + per - 1) / per), p.parts);
    const auto f = v8 ? slope_of<T, PT, 8>(p.act) : slope_of<T, PT, 1>(p.act);
    if (behind)
        return launch_status(launch_behind(f, grid, kRowThreads, 0, st, p));
    f<<<grid, kRowThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}
template <typename T> ecc_status slope_launch(const SlopeParams &p, uint32_t pre_type, bool behind, cudaStream_t st)
{
    return pre_type == ECC_F32    ? slope_launch<T, float>(p, behind, st)
           : pre_type == ECC_BF16 ? slope_launch<T, bf16>(p, behind, st)
                                  : slope_launch<T, __half>(p, behind, st);
}

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

size_t ecc_linear_workspace_bytes(const ecc_linear_job *job)
{
    if (!job || !job->M || !job->N || !job->K || few_rows(*job))
        return 0;
    return copy_bytes(job->x, job->ldx, job->M, job->K, job->in_type) +
           copy_bytes(job->w, job->ldw, job->N, job->K, job->in_type);
}

ecc_status ecc_linear(const ecc_linear_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !linear_ok(*job))
        return ECC_ERR_ARG;
    const ecc_linear_job &j = *job;
    cudaStream_t st = (cudaStream_t)stream;
    if (!j.M || !j.N)
        return launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    const size_t need = ecc_linear_workspace_bytes(job);
    if (need && (!ws || !aligned16(ws) || ws_bytes < need))
        return ECC_ERR_ARG;
    const Epilogue e{j.bias,  j.residual,  j.out,       j.pre,      j.ldres,    j.ldout,    j.ldpre,
                     j.scale, j.out_scale, j.bias_type, j.res_type, j.out_type, j.pre_type, j.act};
    if (few_rows(j)) {
        const int sms = sm_count();
        if (sms <= 0)
            return ECC_ERR_CUDA;
        const FewRows p{j.x, j.w, j.ldx, j.ldw, j.N, j.K, 1, e, status, nullptr, 0};
        if (j.in_type == ECC_BF16)
            few_rows_launch<bf16, false>(j.M, p, sms, st);
        else if (j.in_type == ECC_F16)
            few_rows_launch<__half, false>(j.M, p, sms, st);
        else
            few_rows_launch<e4m3, false>(j.M, p, sms, st);
        return launch_status(cudaGetLastError());
    }
    uint8_t *w = (uint8_t *)ws;
    Operand x, wt;
    bool copied;
    const ecc_status rc = readable({{j.x, j.ldx, j.M, j.K, &x}, {j.w, j.ldw, j.N, j.K, &wt}}, j.in_type, w, st, copied);
    return rc != ECC_OK ? rc : gemm({wt, x, j.M, j.N, j.K, e}, j.in_type, status, true, copied, st);
}

size_t ecc_linear_grad_workspace_bytes(const ecc_linear_grad_job *job)
{
    return job ? grad_plan(*job).bytes : 0;
}

ecc_status ecc_linear_grad(const ecc_linear_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !grad_ok(*job))
        return ECC_ERR_ARG;
    const ecc_linear_grad_job &j = *job;
    const GradPlan g = grad_plan(j);
    if (g.bytes && (!ws || !aligned16(ws) || ws_bytes < g.bytes))
        return ECC_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *w = (uint8_t *)ws;
    void *t = g.make_t ? w : const_cast<void *>(j.dy);
    w += g.t_bytes;
    float *part = j.dbias ? (float *)w : nullptr;
    w += g.part_bytes;
    Operand x, wt; // read down their columns
    bool own;
    ecc_status rc = readable({{j.x, j.ldx, j.dw ? j.M : 0, j.K, &x}, {j.w, j.ldw, j.dx ? j.N : 0, j.K, &wt}}, j.in_type, w, st, own);
    if (rc != ECC_OK)
        return rc;
    x.mn = wt.mn = true;
    const bool slope = j.N && (j.M || j.dbias) && (g.make_t || j.dbias);
    if (slope) {
        const SlopeParams p{j.dy,  j.pre, g.make_t ? t : nullptr, part, j.M, j.N, j.lddy, j.ldpre, g.ldt, j.act,
                            g.parts, status};
        const uint32_t pre_type = j.act == ECC_ACT_NONE ? j.in_type : j.pre_type;
        rc = j.in_type == ECC_BF16 ? slope_launch<bf16>(p, pre_type, own, st) : slope_launch<__half>(p, pre_type, own, st);
        own = true;
    }
    // status: cleared by t's kernel, or by the first product, or by itself
    bool clear = !slope;
    Product dx{wt, {t, g.ldt, false}, j.M, j.K, j.N, {}}, dw{x, {t, g.ldt, true}, j.N, j.K, j.M, {}};
    dx.e.scale = dw.e.scale = j.scale;
    dx.e.out_scale = dw.e.out_scale = 1.f;
    dx.e.out = j.dx;
    dx.e.ldout = j.lddx;
    dx.e.out_type = j.in_type;
    dw.e.out = j.dw;
    dw.e.ldout = j.lddw;
    dw.e.out_type = j.dw_type;
    const bool want_dx = j.dx && j.M && j.K, want_dw = j.dw && j.N && j.K;
    if (rc == ECC_OK && want_dx && want_dw)
        rc = gemm_backward(dx, dw, j.in_type, status, clear, own, st);
    else if (rc == ECC_OK && (want_dx || want_dw))
        rc = gemm(want_dx ? dx : dw, j.in_type, status, clear, own, st);
    if (want_dx || want_dw)
        clear = false;
    if (rc == ECC_OK && slope && j.dbias)
        rc = launch_status(launch_behind(sum_parts_kernel, dim3((unsigned)((j.N + kRowThreads - 1) / kRowThreads)), kRowThreads, 0,
                                         st, (const float *)part, g.parts, j.N, j.dbias, j.N, (float *)nullptr));
    if (rc == ECC_OK && clear)
        rc = launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    return rc;
}

} // extern "C"
