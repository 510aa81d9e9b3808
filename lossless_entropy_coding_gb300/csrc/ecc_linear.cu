// ecc_linear.cu -- a layer's matrix product with its epilogue (scale, bias,
// activation, residual), and its backward pass: t = dy * act'(pre) with the
// bias gradient, then the two products (ecc_gemm.cu).
//
// The products read their operands by TMA, which wants rows on 16-byte
// boundaries: an operand with other rows is first copied to the workspace
// with padded rows.

#include <algorithm>
#include <cmath>

#include "ecc_gemm.h"
#include "ecc_lm.cuh"

namespace ecc {

constexpr int kRowThreads = 256;
constexpr uint32_t kSlopeParts = 64; // partial column sums of t at most

__device__ __forceinline__ float act_slope(uint32_t act, float a)
{
    switch (act) {
    case ECC_ACT_RELU:
        return a > 0.f ? 1.f : (a != a ? a : 0.f);
    case ECC_ACT_GELU: // Phi(a) + a phi(a)
        return 0.5f * (1.f + erff(a * 0.70710678f)) + a * 0.39894228f * __expf(-0.5f * a * a);
    case ECC_ACT_GELU_TANH: { // with h = (1 + tanh u) / 2 = 1 / (1 + e^-2u): h + 2 a h (1 - h) u'
        const float u2 = 1.59576912f * (a + 0.044715f * a * a * a), h = __fdividef(1.f, 1.f + __expf(-u2));
        return h + a * h * (1.f - h) * 1.59576912f * (1.f + 0.134145f * a * a);
    }
    case ECC_ACT_SILU: {
        const float h = __fdividef(1.f, 1.f + __expf(-a));
        return h * (1.f + a * (1.f - h));
    }
    default:
        return 1.f;
    }
}

// t = dy * act'(pre), rounded to the operand type (the tensor cores' input);
// the column sums of t before that rounding
struct SlopeParams {
    const void *dy, *pre;
    void *t;     // [M, ldt]; NULL: only the sums
    float *part; // [parts][N]; NULL: no sums
    uint64_t M, N, lddy, ldpre, ldt;
    uint32_t pre_type, act, parts;
    uint32_t *status;
};

// a block: 32 * V columns, one share of the rows, eight rows at a time
template <typename T, int V> __global__ void __launch_bounds__(kRowThreads) slope_kernel(SlopeParams p)
{
    __shared__ float sums[8][32 * V + 1];
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *p.status = ECC_OK;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const uint64_t c = ((uint64_t)blockIdx.x * 32 + tx) * V;
    const uint64_t per = (p.M + p.parts - 1) / p.parts, r0 = blockIdx.y * per, r1 = min(p.M, r0 + per);
    struct alignas(V * sizeof(T)) Vec {
        T v[V];
    };
    float s[V] = {};
    if (c < p.N)
        for (uint64_t r = r0 + ty; r < r1; r += 8) {
            const Vec d = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.dy) + r * p.lddy + c);
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = to_f32(d.v[i]);
            if (p.act != ECC_ACT_NONE) {
                float a[V];
                if (p.pre_type == TypeCode<T>::value) {
                    const Vec q = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.pre) + r * p.ldpre + c);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        a[i] = to_f32(q.v[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        a[i] = load_any(p.pre, r * p.ldpre + c + i, p.pre_type);
                }
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[i] *= act_slope(p.act, a[i]);
            }
            if (p.t) {
                Vec o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.v[i] = from_f32<T>(v[i]);
                *reinterpret_cast<Vec *>(static_cast<T *>(p.t) + r * p.ldt + c) = o;
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                s[i] += v[i];
        }
    if (!p.part)
        return;
#pragma unroll
    for (int i = 0; i < V; ++i)
        sums[ty][tx + 32 * i] = s[i];
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

__global__ void __launch_bounds__(kRowThreads) sum_parts_kernel(const float *part, uint32_t parts, uint64_t n, float *out)
{
    const uint64_t c = (uint64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (c >= n)
        return;
    float s = 0.f;
    for (uint32_t k = 0; k < parts; ++k)
        s += part[k * n + c];
    out[c] = s;
}

// rows of `cols` elements to rows of ldd elements on 16-byte boundaries
template <typename T>
__global__ void __launch_bounds__(kRowThreads) pad_rows_kernel(const T *src, uint64_t ld, uint64_t rows, uint64_t cols,
                                                               T *dst, uint64_t ldd)
{
    constexpr int V = 16 / sizeof(T);
    struct alignas(16) Vec {
        T v[V];
    };
    const uint64_t vecs = ldd / V, n = rows * vecs;
    for (uint64_t i = (uint64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += (uint64_t)gridDim.x * kRowThreads) {
        const uint64_t r = i / vecs, c = (i - r * vecs) * V;
        const T *s = src + r * ld + c;
        Vec o;
#pragma unroll
        for (int k = 0; k < V; ++k)
            o.v[k] = c + k < cols ? s[k] : T(0);
        *reinterpret_cast<Vec *>(dst + r * ldd + c) = o;
    }
}

namespace {

constexpr uint64_t kMostDim = 1ull << 31;

uint64_t padded(uint64_t cols, uint32_t type)
{
    const uint64_t v = 16 / type_bytes(type);
    return (cols + v - 1) / v * v;
}
size_t pad256(size_t b) { return (b + 255) / 256 * 256; }
size_t copy_bytes(const void *p, uint64_t ld, uint64_t rows, uint64_t cols, uint32_t type)
{
    return rows && cols && !tma_rows(p, ld, type, rows) ? pad256(rows * padded(cols, type) * type_bytes(type)) : 0;
}

// the operand itself, or its copy at ws (advanced past it)
Operand readable(const void *p, uint64_t ld, uint64_t rows, uint64_t cols, uint32_t type, uint8_t *&ws, cudaStream_t st)
{
    const size_t bytes = copy_bytes(p, ld, rows, cols, type);
    if (!bytes)
        return {p, ld, false};
    const uint64_t ldd = padded(cols, type), vecs = rows * ldd * type_bytes(type) / 16;
    const unsigned grid = (unsigned)std::min<uint64_t>((vecs + kRowThreads - 1) / kRowThreads, 1u << 16);
    if (type == ECC_E4M3)
        pad_rows_kernel<uint8_t><<<grid, kRowThreads, 0, st>>>((const uint8_t *)p, ld, rows, cols, ws, ldd);
    else
        pad_rows_kernel<uint16_t><<<grid, kRowThreads, 0, st>>>((const uint16_t *)p, ld, rows, cols, (uint16_t *)ws, ldd);
    const Operand o{ws, ldd, false};
    ws += bytes;
    return o;
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

template <typename T> ecc_status slope_launch(SlopeParams p, cudaStream_t st)
{
    const auto whole = [](const void *q, uint64_t ld) { return ((uintptr_t)q & 15) == 0 && ld % 8 == 0; };
    // eight values a load where the rows allow it (1: 16-bit rows anywhere)
    const bool v8 = p.N % 8 == 0 && whole(p.dy, p.lddy) && (!p.t || whole(p.t, p.ldt)) &&
                    (p.act == ECC_ACT_NONE || p.pre_type != TypeCode<T>::value || whole(p.pre, p.ldpre));
    const uint64_t per = v8 ? 256 : 32;
    const dim3 grid((unsigned)((p.N + per - 1) / per), p.parts);
    if (v8)
        slope_kernel<T, 8><<<grid, kRowThreads, 0, st>>>(p);
    else
        slope_kernel<T, 1><<<grid, kRowThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

size_t ecc_linear_workspace_bytes(const ecc_linear_job *job)
{
    if (!job || !job->M || !job->N || !job->K)
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
    uint8_t *w = (uint8_t *)ws;
    const Operand x = readable(j.x, j.ldx, j.M, j.K, j.in_type, w, st);
    const Operand wt = readable(j.w, j.ldw, j.N, j.K, j.in_type, w, st);
    const Epilogue e{j.bias,  j.residual,  j.out,       j.pre,      j.ldres,    j.ldout,    j.ldpre,
                     j.scale, j.out_scale, j.bias_type, j.res_type, j.out_type, j.pre_type, j.act};
    return gemm(wt, x, j.M, j.N, j.K, j.in_type, e, status, true, st);
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
    ecc_status rc = ECC_OK;
    const bool slope = j.N && (j.M || j.dbias) && (g.make_t || j.dbias);
    if (slope) {
        const SlopeParams p{j.dy,  j.pre,  g.make_t ? t : nullptr, part, j.M, j.N, j.lddy, j.ldpre, g.ldt,
                            j.pre_type, j.act, g.parts, status};
        rc = j.in_type == ECC_BF16 ? slope_launch<bf16>(p, st) : slope_launch<__half>(p, st);
        if (rc == ECC_OK && j.dbias) {
            sum_parts_kernel<<<(unsigned)((j.N + kRowThreads - 1) / kRowThreads), kRowThreads, 0, st>>>(part, g.parts, j.N,
                                                                                                    j.dbias);
            rc = launch_status(cudaGetLastError());
        }
    } else if (cudaMemsetAsync(status, 0, sizeof(uint32_t), st) != cudaSuccess) {
        rc = launch_status(cudaErrorUnknown);
    }
    Epilogue e{};
    e.scale = j.scale;
    e.out_scale = 1.f;
    if (rc == ECC_OK && j.dx && j.M && j.K) { // rows M, columns K, reduction N: w is read down its columns
        Operand wt = readable(j.w, j.ldw, j.N, j.K, j.in_type, w, st);
        wt.mn = true;
        e.out = j.dx;
        e.ldout = j.lddx;
        e.out_type = j.in_type;
        rc = gemm(wt, {t, g.ldt, false}, j.M, j.K, j.N, j.in_type, e, status, false, st);
    }
    if (rc == ECC_OK && j.dw && j.N && j.K) { // rows N, columns K, reduction M: t and x are read down their columns
        Operand x = readable(j.x, j.ldx, j.M, j.K, j.in_type, w, st);
        x.mn = true;
        e.out = j.dw;
        e.ldout = j.lddw;
        e.out_type = j.dw_type;
        rc = gemm(x, {t, g.ldt, true}, j.N, j.K, j.M, j.in_type, e, status, false, st);
    }
    return rc;
}

} // extern "C"
