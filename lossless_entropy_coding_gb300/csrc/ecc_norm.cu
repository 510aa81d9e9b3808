// ecc_norm.cu -- layer norm of rows and its backward pass.
//
// y = (x - mean) * rstd * weight + bias, the variance as the mean square
// deviation from the mean (two passes: a single pass of squares loses digits
// when the mean is large).  Backward, with xh = (x - mean) * rstd and
// g = dy * weight: dx = rstd * (g - avg(g) - xh * avg(g * xh)), dweight and
// dbias the column sums of dy * xh and dy, added up in a fixed order.

#include <algorithm>
#include <cmath>

#include "ecc_lm.cuh"

namespace ecc {

constexpr int kNormThreads = 256;
constexpr uint32_t kNormParts = 304; // partial column sums at most (rows of the workspace)

struct NormParams {
    const void *x, *weight, *bias;
    void *y;
    float *mean, *rstd;
    uint64_t ldx, ldy, rows, cols;
    uint32_t p_type;
    float eps, y_scale;
};

struct NormGradParams {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void *dx;
    float *dweight, *dbias, *part; // part: [2][parts][cols]
    uint64_t lddy, ldx, lddx, rows, cols;
    uint32_t p_type, parts;
};

// sum of a and b over a block of kNormThreads
__device__ __forceinline__ float2 block_sum2(float a, float b)
{
    __shared__ float2 part[kNormThreads / 32];
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads(); // the previous call's reads are done
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) {
        s.x += part[i].x;
        s.y += part[i].y;
    }
    return s;
}

// rows of any length: a block a row, the row read once per pass
template <typename T, typename TO> __global__ void __launch_bounds__(kNormThreads) norm_rows_kernel(NormParams p)
{
    const float inv = 1.f / (float)p.cols;
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        TO *y = static_cast<TO *>(p.y) + r * p.ldy;
        float s = 0.f;
        for (uint64_t i = threadIdx.x; i < p.cols; i += kNormThreads)
            s += to_f32(x[i]);
        const float mean = block_sum2(s, 0.f).x * inv;
        s = 0.f;
        for (uint64_t i = threadIdx.x; i < p.cols; i += kNormThreads) {
            const float d = to_f32(x[i]) - mean;
            s += d * d;
        }
        const float rstd = 1.f / sqrtf(block_sum2(s, 0.f).x * inv + p.eps);
        for (uint64_t i = threadIdx.x; i < p.cols; i += kNormThreads) {
            float v = (to_f32(x[i]) - mean) * rstd;
            if (p.weight)
                v *= load_any(p.weight, i, p.p_type);
            if (p.bias)
                v += load_any(p.bias, i, p.p_type);
            y[i] = from_f32<TO>(v * p.y_scale);
        }
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[r] = mean;
            if (p.rstd)
                p.rstd[r] = rstd;
        }
    }
}

template <typename T> __global__ void __launch_bounds__(kNormThreads) norm_dx_rows_kernel(NormGradParams p)
{
    const float inv = 1.f / (float)p.cols;
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        const T *dy = static_cast<const T *>(p.dy) + r * p.lddy;
        T *dx = static_cast<T *>(p.dx) + r * p.lddx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s = 0.f, q = 0.f;
        for (uint64_t i = threadIdx.x; i < p.cols; i += kNormThreads) {
            float g = to_f32(dy[i]);
            if (p.weight)
                g *= load_any(p.weight, i, p.p_type);
            s += g;
            q += g * ((to_f32(x[i]) - mean) * rstd);
        }
        const float2 c = block_sum2(s, q);
        const float c1 = c.x * inv, c2 = c.y * inv;
        for (uint64_t i = threadIdx.x; i < p.cols; i += kNormThreads) {
            float g = to_f32(dy[i]);
            if (p.weight)
                g *= load_any(p.weight, i, p.p_type);
            dx[i] = from_f32<T>(rstd * (g - c1 - (to_f32(x[i]) - mean) * rstd * c2));
        }
    }
}

// partial column sums: block (c, k) sums 256 columns over the k-th share of the rows
template <typename T> __global__ void __launch_bounds__(kNormThreads) norm_dw_rows_kernel(NormGradParams p)
{
    const uint64_t c = (uint64_t)blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= p.cols)
        return;
    const uint64_t per = (p.rows + p.parts - 1) / p.parts;
    const uint64_t r0 = blockIdx.y * per, r1 = min(p.rows, r0 + per);
    float w = 0.f, b = 0.f;
    for (uint64_t r = r0; r < r1; ++r) {
        const float d = to_f32(static_cast<const T *>(p.dy)[r * p.lddy + c]);
        const float xh = (to_f32(static_cast<const T *>(p.x)[r * p.ldx + c]) - p.mean[r]) * p.rstd[r];
        w += d * xh;
        b += d;
    }
    p.part[blockIdx.y * p.cols + c] = w;
    p.part[(p.parts + blockIdx.y) * p.cols + c] = b;
}

__global__ void __launch_bounds__(kNormThreads) norm_parts_kernel(const float *part, uint32_t parts, uint64_t cols,
                                                                  float *dweight, float *dbias)
{
    const uint64_t c = (uint64_t)blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= cols)
        return;
    float *out = blockIdx.y ? dbias : dweight;
    if (!out)
        return;
    part += (uint64_t)blockIdx.y * parts * cols;
    float s = 0.f;
    for (uint32_t k = 0; k < parts; ++k)
        s += part[k * cols + c];
    out[c] = s;
}

namespace {

unsigned row_grid(uint64_t rows) { return (unsigned)std::min<uint64_t>(rows, 1u << 20); }

template <typename T> ecc_status norm_launch(const NormParams &p, uint32_t y_type, cudaStream_t st)
{
    if (y_type == ECC_E4M3)
        norm_rows_kernel<T, e4m3><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    else
        norm_rows_kernel<T, T><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

template <typename T> ecc_status norm_grad_launch(NormGradParams p, cudaStream_t st)
{
    const unsigned cb = (unsigned)((p.cols + kNormThreads - 1) / kNormThreads);
    if (p.dweight || p.dbias) {
        p.parts = (uint32_t)std::min<uint64_t>(kNormParts, p.rows);
        if (p.rows) // before dx, which may overwrite dy or x
            norm_dw_rows_kernel<T><<<dim3(cb, p.parts), kNormThreads, 0, st>>>(p);
        norm_parts_kernel<<<dim3(cb, 2), kNormThreads, 0, st>>>(p.part, p.parts, p.cols, p.dweight, p.dbias);
    }
    if (p.dx && p.rows)
        norm_dx_rows_kernel<T><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

bool p_type_ok(uint32_t p_type, uint32_t type) { return p_type == type || p_type == ECC_F32; }

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

ecc_status ecc_layer_norm(const void *x, uint64_t ldx, uint32_t x_type, const void *weight, const void *bias,
                          uint32_t p_type, uint64_t rows, uint64_t cols, float eps, void *y, uint64_t ldy,
                          uint32_t y_type, float y_scale, float *mean, float *rstd, void *stream)
{
    if (!wide_type(x_type) || (y_type != x_type && y_type != ECC_E4M3) || !p_type_ok(p_type, x_type) || !cols ||
        cols >= (1u << 31) || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(y_scale) ||
        (y_type != ECC_E4M3 && y_scale != 1.f))
        return ECC_ERR_ARG;
    if (!rows)
        return ECC_OK;
    if (!x || !y || ldx < cols || ldy < cols || !aligned_to(x, x_type) || !aligned_to(y, y_type) ||
        !aligned_to(weight, p_type) || !aligned_to(bias, p_type) || !aligned_to(mean, ECC_F32) ||
        !aligned_to(rstd, ECC_F32) || (x == y && (x_type != y_type || ldx != ldy)))
        return ECC_ERR_ARG;
    NormParams p{x, weight, bias, y, mean, rstd, ldx, ldy, rows, cols, p_type, eps, y_scale};
    cudaStream_t st = (cudaStream_t)stream;
    return x_type == ECC_F32    ? norm_launch<float>(p, y_type, st)
           : x_type == ECC_BF16 ? norm_launch<bf16>(p, y_type, st)
                                : norm_launch<__half>(p, y_type, st);
}

size_t ecc_layer_norm_grad_workspace_bytes(uint64_t rows, uint64_t cols)
{
    return (size_t)std::min<uint64_t>(rows, kNormParts) * cols * 2 * sizeof(float);
}

ecc_status ecc_layer_norm_grad(const void *dy, uint64_t lddy, const void *x, uint64_t ldx, uint32_t type,
                               const void *weight, uint32_t p_type, const float *mean, const float *rstd,
                               uint64_t rows, uint64_t cols, void *dx, uint64_t lddx, float *dweight, float *dbias,
                               void *ws, size_t ws_bytes, void *stream)
{
    if (!wide_type(type) || !p_type_ok(p_type, type) || !cols || cols >= (1u << 31))
        return ECC_ERR_ARG;
    if (rows && (!dy || !x || !mean || !rstd || lddy < cols || ldx < cols || (dx && lddx < cols)))
        return ECC_ERR_ARG;
    if (!aligned_to(dy, type) || !aligned_to(x, type) || !aligned_to(dx, type) || !aligned_to(weight, p_type) ||
        !aligned_to(mean, ECC_F32) || !aligned_to(rstd, ECC_F32) || !aligned_to(dweight, ECC_F32) ||
        !aligned_to(dbias, ECC_F32) || (dx && dx == dy && lddx != lddy) || (dx && dx == x && lddx != ldx))
        return ECC_ERR_ARG;
    if ((dweight || dbias) && rows &&
        (!ws || !aligned16(ws) || ws_bytes < ecc_layer_norm_grad_workspace_bytes(rows, cols)))
        return ECC_ERR_ARG;
    if (!rows && !dweight && !dbias)
        return ECC_OK;
    NormGradParams p{dy,  x,    weight, mean, rstd, dx, dweight, dbias, (float *)ws, lddy, ldx, lddx, rows, cols,
                     p_type, 0};
    cudaStream_t st = (cudaStream_t)stream;
    return type == ECC_F32    ? norm_grad_launch<float>(p, st)
           : type == ECC_BF16 ? norm_grad_launch<bf16>(p, st)
                              : norm_grad_launch<__half>(p, st);
}

} // extern "C"
