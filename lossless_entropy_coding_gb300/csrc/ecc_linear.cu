// ecc_linear.cu -- a layer's matrix product with its epilogue (scale, bias,
// activation, residual), and its backward products.

#include <algorithm>
#include <cmath>

#include "ecc_lm.cuh"

namespace ecc {

constexpr int kTile = 64, kTileK = 16, kGemmThreads = 256;

// C[i, j] = sum over k of A[i, k] B[j, k], each operand read through a row and
// a reduction stride, then the epilogue
struct GemmParams {
    const void *a, *b;
    uint64_t M, N, K;
    uint64_t a_row, a_red, b_row, b_red; // strides in elements
    const void *bias, *residual;
    void *out, *pre;
    uint64_t ldres, ldout, ldpre;
    float scale, out_scale;
    uint32_t bias_type, res_type, out_type, pre_type, act;
    uint32_t *status;
};

__device__ __forceinline__ float act_value(uint32_t act, float a)
{
    switch (act) {
    case ECC_ACT_RELU:
        return a > 0.f ? a : (a != a ? a : 0.f);
    case ECC_ACT_GELU:
        return 0.5f * a * (1.f + erff(a * 0.70710678f));
    case ECC_ACT_GELU_TANH:
        return 0.5f * a * (1.f + tanhf(0.79788456f * (a + 0.044715f * a * a * a)));
    case ECC_ACT_SILU:
        return a / (1.f + expf(-a));
    default:
        return a;
    }
}

__device__ __forceinline__ float act_slope(uint32_t act, float a)
{
    switch (act) {
    case ECC_ACT_RELU:
        return a > 0.f ? 1.f : (a != a ? a : 0.f);
    case ECC_ACT_GELU: // Phi(a) + a phi(a)
        return 0.5f * (1.f + erff(a * 0.70710678f)) + a * 0.39894228f * expf(-0.5f * a * a);
    case ECC_ACT_GELU_TANH: {
        const float t = tanhf(0.79788456f * (a + 0.044715f * a * a * a));
        return 0.5f * (1.f + t) + 0.5f * a * (1.f - t * t) * 0.79788456f * (1.f + 0.134145f * a * a);
    }
    case ECC_ACT_SILU: {
        const float s = 1.f / (1.f + expf(-a));
        return s * (1.f + a * (1.f - s));
    }
    default:
        return 1.f;
    }
}

template <typename T> __global__ void __launch_bounds__(kGemmThreads) gemm_tile_kernel(GemmParams p)
{
    __shared__ float sa[kTileK][kTile + 1], sb[kTileK][kTile + 1];
    const T *A = static_cast<const T *>(p.a), *B = static_cast<const T *>(p.b);
    const uint64_t i0 = (uint64_t)blockIdx.y * kTile, j0 = (uint64_t)blockIdx.x * kTile;
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    if (p.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *p.status = ECC_OK;
    float acc[4][4] = {};
    for (uint64_t k0 = 0; k0 < p.K; k0 += kTileK) {
        for (int e = threadIdx.x; e < kTile * kTileK; e += kGemmThreads) {
            const int i = e / kTileK, k = e % kTileK;
            sa[k][i] = i0 + i < p.M && k0 + k < p.K ? to_f32(A[(i0 + i) * p.a_row + (k0 + k) * p.a_red]) : 0.f;
            sb[k][i] = j0 + i < p.N && k0 + k < p.K ? to_f32(B[(j0 + i) * p.b_row + (k0 + k) * p.b_red]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTileK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] += sa[k][ti * 4 + i] * sb[k][tj + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const uint64_t r = i0 + ti * 4 + i, c = j0 + tj + 16 * j;
            if (r >= p.M || c >= p.N)
                continue;
            float a = acc[i][j] * p.scale;
            if (p.bias)
                a += load_any(p.bias, c, p.bias_type);
            if (p.pre)
                store_any(p.pre, r * p.ldpre + c, p.pre_type, a);
            a = act_value(p.act, a);
            if (p.residual)
                a += load_any(p.residual, r * p.ldres + c, p.res_type);
            store_any(p.out, r * p.ldout + c, p.out_type, p.out_type == ECC_E4M3 ? a * p.out_scale : a);
        }
}

// t = dy * act'(pre), rounded to the operand type
struct SlopeParams {
    const void *dy, *pre;
    void *t;
    float *dbias;
    uint64_t M, N, lddy, ldpre, ldt;
    uint32_t type, pre_type, act;
};

// a block: 32 columns, 8 rows at a time
__global__ void __launch_bounds__(256) slope_kernel(SlopeParams p, uint32_t *status)
{
    __shared__ float part[8][33];
    if (status && blockIdx.x == 0 && threadIdx.x == 0)
        *status = ECC_OK;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const uint64_t c = (uint64_t)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < p.N)
        for (uint64_t r = ty; r < p.M; r += 8) {
            float v = load_any(p.dy, r * p.lddy + c, p.type);
            if (p.act != ECC_ACT_NONE) {
                v *= act_slope(p.act, load_any(p.pre, r * p.ldpre + c, p.pre_type));
                store_any(p.t, r * p.ldt + c, p.type, v);
            }
            s += v;
        }
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < p.N && p.dbias) {
        for (int k = 1; k < 8; ++k)
            s += part[k][tx];
        p.dbias[c] = s;
    }
}

namespace {

ecc_status gemm(const GemmParams &p, uint32_t type, cudaStream_t st)
{
    if (!p.M || !p.N)
        return ECC_OK;
    const dim3 grid((unsigned)((p.N + kTile - 1) / kTile), (unsigned)((p.M + kTile - 1) / kTile));
    if (grid.y > 65535)
        return ECC_ERR_ARG;
    if (type == ECC_BF16)
        gemm_tile_kernel<bf16><<<grid, kGemmThreads, 0, st>>>(p);
    else if (type == ECC_F16)
        gemm_tile_kernel<__half><<<grid, kGemmThreads, 0, st>>>(p);
    else
        gemm_tile_kernel<e4m3><<<grid, kGemmThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

constexpr uint64_t kMostDim = 1ull << 31;

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

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

size_t ecc_linear_workspace_bytes(const ecc_linear_job *)
{
    return 0;
}

ecc_status ecc_linear(const ecc_linear_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !linear_ok(*job))
        return ECC_ERR_ARG;
    const ecc_linear_job &j = *job;
    cudaStream_t st = (cudaStream_t)stream;
    if (!j.M || !j.N)
        return launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    GemmParams p{j.x,     j.w,     j.M,      j.N,     j.K,          j.ldx,       1,          j.ldw,      1,     j.bias, j.residual, j.out, j.pre,
                 j.ldres, j.ldout, j.ldpre, j.scale, j.out_scale, j.bias_type, j.res_type, j.out_type, j.pre_type, j.act, status};
    return gemm(p, j.in_type, st);
}

size_t ecc_linear_grad_workspace_bytes(const ecc_linear_grad_job *job)
{
    if (!job || job->act == ECC_ACT_NONE)
        return 0;
    return (size_t)job->M * job->N * 2;
}

ecc_status ecc_linear_grad(const ecc_linear_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream)
{
    if (!job || !status || !aligned_to(status, ECC_F32) || !grad_ok(*job))
        return ECC_ERR_ARG;
    const ecc_linear_grad_job &j = *job;
    if (ecc_linear_grad_workspace_bytes(job) && (!ws || !aligned16(ws) || ws_bytes < ecc_linear_grad_workspace_bytes(job)))
        return ECC_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const bool slope = j.act != ECC_ACT_NONE;
    SlopeParams s{j.dy, j.pre, ws, j.dbias, j.M, j.N, j.lddy, j.ldpre, j.N, j.in_type, j.pre_type, j.act};
    if (j.N)
        slope_kernel<<<(unsigned)((j.N + 31) / 32), 256, 0, st>>>(s, status);
    else if (cudaMemsetAsync(status, 0, sizeof(uint32_t), st) != cudaSuccess)
        return launch_status(cudaErrorUnknown);
    const void *t = slope ? ws : j.dy;
    const uint64_t ldt = slope ? j.N : j.lddy;
    ecc_status rc = launch_status(cudaGetLastError());
    if (rc == ECC_OK && j.dx) {
        GemmParams p{t, j.w, j.M, j.K, j.N, ldt, 1, 1, j.ldw, nullptr, nullptr, j.dx, nullptr, 0, j.lddx, 0, j.scale, 1.f, 0, 0, j.in_type, 0, 0, nullptr};
        rc = gemm(p, j.in_type, st);
    }
    if (rc == ECC_OK && j.dw) {
        GemmParams p{t, j.x, j.N, j.K, j.M, 1, ldt, 1, j.ldx, nullptr, nullptr, j.dw, nullptr, 0, j.lddw, 0, j.scale, 1.f, 0, 0, j.dw_type, 0, 0, nullptr};
        rc = gemm(p, j.in_type, st);
    }
    return rc;
}

} // extern "C"
