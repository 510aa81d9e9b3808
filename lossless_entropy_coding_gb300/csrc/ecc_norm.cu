// ecc_norm.cu -- layer norm of rows and its backward pass.
//
// y = (x - mean) * rstd * weight + bias, the variance as the mean square
// deviation from the mean (two passes: a single pass of squares loses digits
// when the mean is large).  Backward, with xh = (x - mean) * rstd and
// g = dy * weight: dx = rstd * (g - avg(g) - xh * avg(g * xh)), dweight and
// dbias the column sums of dy * xh and dy, added up in a fixed order.

#include <algorithm>
#include <cmath>

#include "ecc_device.cuh"
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

// rows of any length: a block a row, the row read in each of three passes
// (rows that do not fit a block's registers)
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

// A block: 32 columns, the parts in 16 shares, a thread's loads all under way
// at once (in eight shares, four at a time, and with a single group's sums
// through shared memory, 16384 x 4096 took 4 us more).
__global__ void __launch_bounds__(512) norm_parts_kernel(const float *part, uint32_t parts, uint64_t cols, float *dweight,
                                                         float *dbias)
{
    constexpr uint32_t AHEAD = 10; // (of 16 shares of 152 parts)
    __shared__ float sums[16][33];
    wait_for_previous();
    const uint32_t tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const uint64_t c = (uint64_t)blockIdx.x * 32 + tx;
    float *out = blockIdx.y ? dbias : dweight;
    if (!out)
        return;
    part += (uint64_t)blockIdx.y * parts * cols;
    float s = 0.f;
    if (c < cols)
        for (uint32_t k0 = ty; k0 < parts; k0 += 16 * AHEAD) {
            float v[AHEAD];
#pragma unroll
            for (uint32_t k = 0; k < AHEAD; ++k)
                v[k] = k0 + 16 * k < parts ? part[(uint64_t)(k0 + 16 * k) * cols + c] : 0.f;
#pragma unroll
            for (uint32_t k = 0; k < AHEAD; ++k)
                s += v[k];
        }
    sums[ty][tx] = s;
    __syncthreads();
    if (ty || c >= cols)
        return;
    for (int k = 1; k < 16; ++k)
        s += sums[k][tx];
    out[c] = s;
}

// ---------------------------------------------------------------- rows in registers
// A thread holds E values of a row, in pairs: E / V accesses of V values
// (V = 16 / sizeof(T), rows on 16-byte boundaries; V = 1, rows anywhere),
// access k at columns (t + k * width) V; values past the row's end are 0.
// (Loads are not through the read-only path: the output may be the input.)
template <typename T, int V, int E>
__device__ __forceinline__ void load_row(const T *row, uint32_t t, uint32_t width, uint32_t n, float2 (&f)[E / 2])
{
    if constexpr (V == 1) {
        T q[E];
#pragma unroll
        for (int k = 0; k < E; ++k)
            q[k] = t + k * width < n ? row[t + k * width] : T(0.f);
#pragma unroll
        for (int k = 0; k < E; k += 2)
            f[k / 2] = make_float2(to_f32(q[k]), to_f32(q[k + 1]));
    } else {
        uint4 q[E / V];
#pragma unroll
        for (int k = 0; k < E / V; ++k)
            q[k] = t + k * width < n ? *reinterpret_cast<const uint4 *>(row + (uint64_t)(t + k * width) * V)
                                     : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < E / V; ++k)
            unpack2<T>(q[k], f + k * V / 2);
    }
}
// access k of a parameter vector (of the rows' type, or float32)
template <typename T, int V>
__device__ __forceinline__ void load_params(const void *p, uint32_t at, uint32_t type, float2 (&f)[V / 2])
{
    if (type == TypeCode<T>::value) {
        unpack2<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + (uint64_t)at * V), f);
    } else {
        const float *q = static_cast<const float *>(p) + (uint64_t)at * V;
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            f[i] = make_float2(q[2 * i], q[2 * i + 1]);
    }
}
// a thread's single parameters (`none` where there is no such vector)
template <typename T, int E>
__device__ __forceinline__ void load_singles(const void *p, uint32_t type, uint32_t t, uint32_t width, uint32_t n,
                                             float none, float (&f)[E])
{
#pragma unroll
    for (int k = 0; k < E; ++k)
        f[k] = none;
    if (!p)
        return;
    if (type == TypeCode<T>::value) {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (t + k * width < n)
                f[k] = to_f32(static_cast<const T *>(p)[t + k * width]);
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (t + k * width < n)
                f[k] = static_cast<const float *>(p)[t + k * width];
    }
}
template <typename T, int V> __device__ __forceinline__ void store_values(T *p, const float2 *f)
{
    if constexpr (sizeof(T) == 1) {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(f[2 * i], __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(f[2 * i + 1], __NV_SATFINITE, __NV_E4M3) << 16;
        if constexpr (V == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    } else {
        *reinterpret_cast<uint4 *>(p) = pack2<T>(f);
    }
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 load_shared16(uint32_t at)
{
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}
__device__ __forceinline__ void store_shared16(uint32_t at, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <typename T> __device__ __forceinline__ void store_shared(uint32_t at, T v) // of 2 or 4 bytes
{
    if constexpr (sizeof(T) == 2)
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<uint16_t *>(&v)) : "memory");
    else
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(*reinterpret_cast<uint32_t *>(&v)) : "memory");
}
template <typename T> __device__ __forceinline__ T load_shared(uint32_t at)
{
    T v;
    if constexpr (sizeof(T) == 2)
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(*reinterpret_cast<uint16_t *>(&v)) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(*reinterpret_cast<uint32_t *>(&v)) : "r"(at) : "memory");
    return v;
}

// ROWS rows by `warps` warps: they are read once and both passes over them
// (the mean, the squared deviations) run on registers.  Blocks of one warp a
// row hold four warps.  Two rows at a time share the parameters (read for each
// row they cost twice the row's own L1 traffic), the barriers and the
// shuffles' latency.  16384 x 4096: bf16 to e4m3 48 us, 4.2 TB/s, to bf16 51,
// 5.2 TB/s; float32 84, 6.4 TB/s.  HBM bounds float32; with the 16-bit types the
// latency from a block's loads to its stores, 20 warps an SM (96 registers a
// thread).  Slower, all of 16384 x 4096 to e4m3: persistent blocks behind a
// ring as in the gradient 66 to 80 us (two joins a row one after the other),
// both sums joined in one go from the threads' means 51, rows kept as read for
// 6 blocks an SM instead of 5 57.
template <typename T, typename TO, int V, int E, int ROWS>
__global__ void __launch_bounds__(ROWS > 1 ? 128 : 1024, ROWS > 1 ? 5 : 1) norm_kernel(NormParams p, uint32_t warps)
{
    __shared__ float part[2][ROWS][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = warps * 32;
    const uint64_t r = (warps == 1 ? (uint64_t)blockIdx.x * (blockDim.x / 32) + warp : blockIdx.x) * ROWS;
    if (r >= p.rows)
        return; // (whole warps of a block of one warp a row)
    const uint32_t t = warps == 1 ? lane : threadIdx.x, n = (uint32_t)(p.cols / V);
    float2 f[ROWS][E / 2];
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
        load_row<T, V, E>(static_cast<const T *>(p.x) + (r + j) * p.ldx, t, width, r + j < p.rows ? n : 0, f[j]);
    auto total = [&](float (&s)[ROWS], int which) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            s[j] = warp_sum(s[j]);
        if (warps == 1)
            return;
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                part[which][j][warp] = s[j];
        }
        __syncthreads();
        if (warps <= 4) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                s[j] = part[which][j][0];
                for (uint32_t i = 1; i < warps; ++i)
                    s[j] += part[which][j][i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                s[j] = warp_sum(lane < warps ? part[which][j][lane] : 0.f);
        }
    };
    const float inv = 1.f / (float)p.cols;
    float mean[ROWS], rstd[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            s = add2(s, f[j][i]);
        mean[j] = s.x + s.y;
    }
    total(mean, 0);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        mean[j] *= inv;
        const float2 minus = both(-mean[j]);
        float2 s = both(0.f);
        if (n == width * (E / V)) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                f[j][i] = add2(f[j][i], minus);
                s = fma2(f[j][i], f[j][i], s);
            }
        } else { // past the end: no deviation
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                f[j][i] = add2(f[j][i], minus);
                f[j][i].x = t + (2 * i / V) * width < n ? f[j][i].x : 0.f;
                f[j][i].y = t + ((2 * i + 1) / V) * width < n ? f[j][i].y : 0.f;
                s = fma2(f[j][i], f[j][i], s);
            }
        }
        rstd[j] = s.x + s.y;
    }
    total(rstd, 1);
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
        rstd[j] = 1.f / sqrtf(rstd[j] * inv + p.eps);
    TO *y = static_cast<TO *>(p.y) + r * p.ldy;
    if constexpr (V == 1) {
#pragma unroll
        for (int k0 = 0; k0 < E; k0 += 4) {
            const uint32_t t0 = t + k0 * width;
            float w[4], b[4];
            load_singles<T, 4>(p.weight, p.p_type, t0, width, n, 1.f, w);
            load_singles<T, 4>(p.bias, p.p_type, t0, width, n, 0.f, b);
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (t0 + k * width < n && r + j < p.rows) {
                        const float2 q = f[j][(k0 + k) / 2];
                        float v = fmaf((k & 1 ? q.y : q.x) * rstd[j], w[k], b[k]);
                        if constexpr (sizeof(TO) == 1)
                            v *= p.y_scale;
                        y[j * p.ldy + t0 + k * width] = from_f32<TO>(v);
                    }
        }
    } else {
        const float2 scale = both(p.y_scale);
#pragma unroll
        for (int k = 0; k < E / V; ++k)
            if (t + k * width < n) {
                float2 w[V / 2], b[V / 2];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    w[i] = both(1.f);
                    b[i] = both(0.f);
                }
                if (p.weight)
                    load_params<T, V>(p.weight, t + k * width, p.p_type, w);
                if (p.bias)
                    load_params<T, V>(p.bias, t + k * width, p.p_type, b);
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    float2 *v = f[j] + k * V / 2;
                    const float2 r2 = both(rstd[j]);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        v[i] = fma2(mul2(v[i], r2), w[i], b[i]);
                        if constexpr (sizeof(TO) == 1)
                            v[i] = mul2(v[i], scale);
                    }
                    if (r + j < p.rows)
                        store_values<TO, V>(y + j * p.ldy + (uint64_t)(t + k * width) * V, v);
                }
            }
    }
    if (t == 0) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            if (r + j < p.rows) {
                if (p.mean)
                    p.mean[r + j] = mean[j];
                if (p.rstd)
                    p.rstd[r + j] = rstd[j];
            }
    }
}

// Rows on any boundary: as above, but a row's vectors begin where those of the
// output's row do; the row and the parameters are read across boundaries, and
// the at most 2 (V - 1) values at the row's ends are a thread's each.  (With a
// value an access, the load and store units' instructions were the bound:
// 16384 x 4097 bf16 took 178 us instead of 102.)
template <typename T, typename TO, int E>
__global__ void __launch_bounds__(512) norm_shifted_kernel(NormParams p, uint32_t warps)
{
    __shared__ float part[2][32];
    constexpr int V = 16 / sizeof(T), PER = E / V;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = warps * 32;
    const uint64_t r = warps == 1 ? (uint64_t)blockIdx.x * (blockDim.x / 32) + warp : blockIdx.x;
    if (r >= p.rows)
        return; // (whole warps of a block of one warp a row)
    const uint32_t t = warps == 1 ? lane : threadIdx.x, cols = (uint32_t)p.cols;
    const T *x = static_cast<const T *>(p.x), *row = x + r * p.ldx;
    TO *y = static_cast<TO *>(p.y) + r * p.ldy;
    const void *end = x + (p.rows - 1) * p.ldx + p.cols;
    constexpr uint32_t A = V * sizeof(TO); // bytes of an output vector
    const uint32_t head = min(((A - ((uint32_t)(uintptr_t)y & (A - 1))) & (A - 1)) / (uint32_t)sizeof(TO), cols);
    const uint32_t n = (cols - head) / V, tail = head + n * V;
    const uint32_t at = t < head ? t : min(tail + (t - head), cols); // this thread's single column (cols: none)
    float2 f[E / 2];
#pragma unroll
    for (int k = 0; k < PER; ++k)
        unpack2<T>(t + k * width < n ? load_anywhere(row + head + (uint64_t)(t + k * width) * V, p.x, end)
                                     : make_uint4(0, 0, 0, 0),
                   f + k * V / 2);
    float single = at < cols ? to_f32(row[at]) : 0.f;
    auto total = [&](float s, int which) {
        s = warp_sum(s);
        if (warps == 1)
            return s;
        if (lane == 0)
            part[which][warp] = s;
        __syncthreads();
        return warp_sum(lane < warps ? part[which][lane] : 0.f);
    };
    const float inv = 1.f / (float)cols;
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        s = add2(s, f[i]);
    const float mean = total(s.x + s.y + single, 0) * inv;
    const float2 minus = both(-mean);
    s = both(0.f);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const bool in = t + k * width < n;
#pragma unroll
        for (int i = k * V / 2; i < (k + 1) * V / 2; ++i) {
            f[i] = add2(f[i], minus);
            f[i].x = in ? f[i].x : 0.f;
            f[i].y = in ? f[i].y : 0.f;
            s = fma2(f[i], f[i], s);
        }
    }
    single = at < cols ? single - mean : 0.f;
    const float rstd = 1.f / sqrtf(total(s.x + s.y + single * single, 1) * inv + p.eps);
    const float2 scale = both(p.y_scale), r2 = both(rstd);
    auto params = [&](const void *q, uint32_t c, float2 (&v)[V / 2]) {
        if (p.p_type == TypeCode<T>::value) {
            const T *v0 = static_cast<const T *>(q);
            unpack2<T>(load_anywhere(v0 + c, v0, v0 + cols), v);
        } else {
            const float *v0 = static_cast<const float *>(q);
#pragma unroll
            for (int i = 0; i < V / 2; i += 2)
                unpack2<float>(load_anywhere(v0 + c + 2 * i, v0, v0 + cols), v + i);
        }
    };
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (t + k * width < n) {
            const uint32_t c = head + (t + k * width) * V;
            float2 *v = f + k * V / 2, w[V / 2], b[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                w[i] = both(1.f);
                b[i] = both(0.f);
            }
            if (p.weight)
                params(p.weight, c, w);
            if (p.bias)
                params(p.bias, c, b);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                v[i] = fma2(mul2(v[i], r2), w[i], b[i]);
                if constexpr (sizeof(TO) == 1)
                    v[i] = mul2(v[i], scale);
            }
            store_values<TO, V>(y + c, v);
        }
    if (at < cols) {
        const float v = fmaf(single * rstd, p.weight ? load_any(p.weight, at, p.p_type) : 1.f,
                             p.bias ? load_any(p.bias, at, p.p_type) : 0.f);
        y[at] = from_f32<TO>(sizeof(TO) == 1 ? v * p.y_scale : v);
    }
    if (t == 0) {
        if (p.mean)
            p.mean[r] = mean;
        if (p.rstd)
            p.rstd[r] = rstd;
    }
}

// ---------------------------------------------------------------- backward, rows in registers
__device__ __forceinline__ void group_barrier(uint32_t id, uint32_t threads) // id below 15
{
    __syncwarp(); // (a lane wrote for its warp: the warp arrives as a whole)
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
}
// The sums over a group's threads of 2 ROWS values each, known to all of them
// on return: within a warp the values are halved over the lanes (each lane
// ends with one value), the warps' sums go through shared memory.
template <int ROWS>
__device__ __forceinline__ void group_sums(float (&v)[2 * ROWS], float (*part)[2 * ROWS], uint32_t group, uint32_t width,
                                           uint32_t warp0)
{
    constexpr int NV = 2 * ROWS, SPAN = 32 / NV; // lanes that hold one value's parts in the end
    const uint32_t lane = threadIdx.x & 31, warps = width / 32;
    int n = NV;
#pragma unroll
    for (int o = 16; o >= SPAN; o >>= 1) {
        n /= 2;
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(~0u, send, o);
        }
    }
    float s = v[0]; // value lane / SPAN
#pragma unroll
    for (int o = SPAN / 2; o; o >>= 1)
        s += __shfl_xor_sync(~0u, s, o);
    if (warps > 1) {
        if (lane % SPAN == 0)
            part[threadIdx.x >> 5][lane / SPAN] = s;
        group_barrier(group, width);
        s = 0.f;
        for (uint32_t w = lane % SPAN; w < warps; w += SPAN)
            s += part[warp0 + w][lane / SPAN];
#pragma unroll
        for (int o = SPAN / 2; o; o >>= 1)
            s += __shfl_xor_sync(~0u, s, o);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        v[i] = __shfl_sync(~0u, s, i * SPAN);
}

// The compiler takes v as new: what it computed from v before is not kept, but computed again.
__device__ __forceinline__ void forget(uint4 &v)
{
    asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
}
// A row at any boundary of an element into a slot of 16-byte pieces: piece v
// holds the v-th aligned 16 bytes from the one with the row's first value on.
// A thread copies the pieces t + k width for k < PER, the first thread one
// more.  (Those of a row at the array's ends may stick out of it: they are
// copied by element.)
template <typename T, int PER>
__device__ __forceinline__ void fetch_row(uint32_t slot, uint32_t t, uint32_t width, const T *row, uint32_t cols,
                                          const T *begin, const T *end)
{
    const uintptr_t low = (uintptr_t)row & ~(uintptr_t)15;
    const uint32_t bytes = ((uint32_t)(uintptr_t)row & 15) + cols * (uint32_t)sizeof(T);
    const bool inside = low >= (uintptr_t)begin && low + ((bytes + 15) & ~15u) <= (uintptr_t)end;
#pragma unroll
    for (int k = 0; k <= PER; ++k) {
        const uint32_t v = t + k * width;
        if (v * 16 >= bytes || (k == PER && t))
            return;
        if (inside) {
            copy_async16(slot + v * 16, reinterpret_cast<const void *>(low + v * 16));
            continue;
        }
        const T *q = reinterpret_cast<const T *>(low + v * 16);
        for (uint32_t i = 0; i < 16 / sizeof(T); ++i)
            if (q + i >= begin && q + i < end)
                store_shared(slot + v * 16 + i * (uint32_t)sizeof(T), q[i]);
    }
}
// the row's v-th vector, 0 past its end
template <typename T>
__device__ __forceinline__ uint4 read_piece(uint32_t slot, uint32_t v, uint32_t off, uint32_t cols)
{
    constexpr uint32_t V = 16 / sizeof(T);
    uint4 a = load_shared16(slot + v * 16);
    if (off)
        a = shift16<false>(a, load_shared16(slot + v * 16 + 16), off);
    if (v * V + V > cols) {
        const uint32_t left = cols > v * V ? (cols - v * V) * (uint32_t)sizeof(T) : 0; // bytes
        uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            w[i] &= left >= 4 * i + 4 ? ~0u : left > 4 * i ? 0xffffu : 0u; // (two bytes of a word, or all)
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return a;
}
// A warp's 32 V values (vectors v, v + 1, ...) to their place at any boundary:
// through its pieces of the slot, then vectors on the boundaries of the place
// and, for the at most 2 (V - 1) values around them, a lane each.
template <typename T, int V>
__device__ __forceinline__ void write_pieces(uint32_t slot, uint32_t v, T *row, uint32_t cols, const float2 *f)
{
    const uint32_t lane = threadIdx.x & 31, first = (v - lane) * V, from = slot + (v - lane) * 16;
    const uint32_t count = cols > first ? min(cols - first, 32u * V) : 0;
    store_shared16(slot + v * 16, pack2<T>(f));
    __syncwarp();
    T *o = row + first;
    const uint32_t head = min(((16 - ((uint32_t)(uintptr_t)o & 15)) & 15) / (uint32_t)sizeof(T), count);
    const uint32_t full = (count - head) / V, tail = head + full * V;
    if (lane < full) {
        uint4 a = load_shared16(from + lane * 16);
        if (head)
            a = shift16<false>(a, load_shared16(from + lane * 16 + 16), head * (uint32_t)sizeof(T));
        *reinterpret_cast<uint4 *>(o + head + lane * V) = a;
    }
    const uint32_t i = lane < head ? lane : tail + (lane - head);
    if (i < count)
        o[i] = load_shared<T>(from + i * (uint32_t)sizeof(T));
}

// Persistent, a block an SM: groups of `width` of its NT threads walk their
// rows ROWS at a time; each thread keeps its columns' sums of dy * xh and dy
// in registers, so x and dy are read once for all three gradients.  A ring in
// shared memory holds the next steps' rows.  On 16-byte boundaries a thread
// copies what it will read itself, RING - 1 steps ahead, without a barrier.
// SHIFT, rows on any boundary: the rows' aligned pieces, which neighbours read
// too, are copied RING - 2 steps ahead, and the barrier that joins a step's
// sums also publishes the next step's pieces; dx leaves through the pieces of
// x just read.  (A value an access, 16384 x 4097 bf16 took 312 us, now 194:
// the shifts' instructions; the aligned 16384 x 4096 71 us, 16384 x 8192 132,
// 5.6 and 6.1 TB/s.)  The groups' column sums are added in shared memory and
// the blocks' in norm_parts_kernel, both in a fixed order.  Bound by HBM.
template <typename T, int NT, int E, int RING, int ROWS, bool SHIFT>
__global__ void __launch_bounds__(NT, 1) norm_grad_kernel(NormGradParams p, uint32_t width)
{
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ float part[2][NT / 32][2 * ROWS];
    constexpr int V = 16 / sizeof(T), PER = E / V;
    let_next_start();
    const uint32_t tid = threadIdx.x, group = tid / width, t = tid - group * width;
    const uint32_t groups = NT / width, warp0 = group * (width / 32), cols = (uint32_t)p.cols;
    const uint32_t n = (cols + V - 1) / V;
    const uint64_t step = (uint64_t)gridDim.x * groups * ROWS;
    const float inv = 1.f / (float)p.cols;
    float2 w[E / 2], aw[E / 2], ab[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        w[i] = both(1.f);
        aw[i] = ab[i] = both(0.f);
    }
    const bool works = group < groups; // threads past the last whole group only join the barriers of the end
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    T *dx = static_cast<T *>(p.dx);
    if (works) {
        if (p.weight) {
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (t + k * width < n) {
                    float2 *q = w + k * V / 2;
                    const uint32_t c = (t + k * width) * V;
                    if constexpr (SHIFT) {
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            q[i].x = c + 2 * i < cols ? load_any(p.weight, c + 2 * i, p.p_type) : 0.f;
                            q[i].y = c + 2 * i + 1 < cols ? load_any(p.weight, c + 2 * i + 1, p.p_type) : 0.f;
                        }
                    } else {
                        float2 u[V / 2];
                        load_params<T, V>(p.weight, t + k * width, p.p_type, u);
#pragma unroll
                        for (int i = 0; i < V / 2; ++i)
                            q[i] = u[i];
                    }
                }
        }
        const uint64_t r0 = ((uint64_t)blockIdx.x * groups + group) * ROWS;
        // SHIFT: a row's slot holds one piece more than the group's threads read
        const uint32_t row_bytes = SHIFT ? (PER * width + 1) * 16 : PER * width * 16;
        const uint32_t ring0 = smem_u32(raw) + group * (2 * ROWS * RING) * row_bytes;
        auto slot = [&](uint32_t at, int j) { return ring0 + (at * ROWS + j) * 2 * row_bytes; }; // x's row, then dy's
        const T *x_end = x + (p.rows - 1) * p.ldx + p.cols, *dy_end = dy + (p.rows - 1) * p.lddy + p.cols;
        auto fetch = [&](uint64_t r, uint32_t at) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (r + j < p.rows) {
                    const uint32_t to = slot(at, j);
                    const T *xr = x + (r + j) * p.ldx, *dyr = dy + (r + j) * p.lddy;
                    if constexpr (SHIFT) {
                        fetch_row<T, PER>(to, t, width, xr, cols, x, x_end);
                        fetch_row<T, PER>(to + row_bytes, t, width, dyr, cols, dy, dy_end);
                    } else {
#pragma unroll
                        for (int k = 0; k < PER; ++k)
                            if (t + k * width < n) {
                                const uint32_t v = t + k * width;
                                copy_async16(to + v * 16, xr + (uint64_t)v * V);
                                copy_async16(to + row_bytes + v * 16, dyr + (uint64_t)v * V);
                            }
                    }
                }
            copy_async_commit();
        };
        auto publish = [&] { // the pieces copied so far to the group
            if (width == 32)
                __syncwarp();
            else
                group_barrier(group, width);
        };
#pragma unroll
        for (int k = 0; k + 1 < RING; ++k)
            fetch(r0 + k * step, k);
        if constexpr (SHIFT) {
            copy_async_wait<RING - 2>();
            publish();
        }
        uint32_t at = 0, flip = 0;
        float mean[ROWS], rstd[ROWS];
        auto stats = [&](uint64_t r) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                mean[j] = r + j < p.rows ? p.mean[r + j] : 0.f;
                rstd[j] = r + j < p.rows ? p.rstd[r + j] : 0.f;
            }
        };
        stats(r0);
        for (uint64_t r = r0; r < p.rows; r += step) {
            fetch(r + (RING - 1) * step, at ? at - 1 : RING - 1);
            if constexpr (!SHIFT)
                copy_async_wait<RING - 1>();
            // the pieces stay as read: as float32 values they would take twice
            // the registers, and half the rows in flight
            uint4 rx[ROWS][PER], rd[ROWS][PER];
            float2 minus[ROWS], r2[ROWS];
            float v[2 * ROWS];
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                minus[j] = both(-mean[j]);
                r2[j] = both(rstd[j]);
                float2 s = both(0.f), q = both(0.f);
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const uint32_t s0 = slot(at, j), u = t + k * width;
                    if constexpr (SHIFT) {
                        const uint32_t m = r + j < p.rows ? cols : 0;
                        rx[j][k] = read_piece<T>(s0, u, (uint32_t)(uintptr_t)(x + (r + j) * p.ldx) & 15, m);
                        rd[j][k] = read_piece<T>(s0 + row_bytes, u, (uint32_t)(uintptr_t)(dy + (r + j) * p.lddy) & 15, m);
                    } else {
                        const bool in = r + j < p.rows && u < n;
                        const uint4 zero = make_uint4(0, 0, 0, 0);
                        rx[j][k] = in ? load_shared16(s0 + u * 16) : zero;
                        rd[j][k] = in ? load_shared16(s0 + row_bytes + u * 16) : zero;
                    }
                    float2 xh[V / 2], d[V / 2];
                    unpack2<T>(rx[j][k], xh);
                    unpack2<T>(rd[j][k], d);
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const int c = k * V / 2 + i;
                        xh[i] = mul2(add2(xh[i], minus[j]), r2[j]);
                        const float2 g = mul2(d[i], w[c]);
                        s = add2(s, g);
                        q = fma2(g, xh[i], q);
                        aw[c] = fma2(d[i], xh[i], aw[c]);
                        ab[c] = add2(ab[c], d[i]);
                    }
                }
                v[2 * j] = s.x + s.y;
                v[2 * j + 1] = q.x + q.y;
            }
            stats(r + step); // a step ahead: they would be waited for
            if constexpr (SHIFT) {
                copy_async_wait<RING - 2>();
                if (!p.dx || width == 32)
                    publish(); // (else the sums' barrier does it)
            }
            if (p.dx) {
                group_sums<ROWS>(v, part[flip], group, width, warp0);
                flip ^= 1;
#pragma unroll
                for (int j = 0; j < ROWS; ++j)
                    if (r + j < p.rows) {
                        const float2 s = both(-v[2 * j] * inv), q = both(-v[2 * j + 1] * inv);
                        T *o = dx + (r + j) * p.lddx;
#pragma unroll
                        for (int k = 0; k < PER; ++k) {
                            const uint32_t u = t + k * width;
                            float2 xh[V / 2], g[V / 2];
                            forget(rx[j][k]);
                            forget(rd[j][k]);
                            unpack2<T>(rx[j][k], xh);
                            unpack2<T>(rd[j][k], g);
#pragma unroll
                            for (int i = 0; i < V / 2; ++i) {
                                xh[i] = mul2(add2(xh[i], minus[j]), r2[j]);
                                g[i] = mul2(fma2(xh[i], q, add2(mul2(g[i], w[k * V / 2 + i]), s)), r2[j]);
                            }
                            if (SHIFT && (cols % V || ((uintptr_t)o & 15)))
                                write_pieces<T, V>(slot(at, j), u, o, cols, g);
                            else if (u < n)
                                store_values<T, V>(o + (uint64_t)u * V, g);
                        }
                    }
                if constexpr (SHIFT)
                    __syncwarp(); // before the pieces are filled again
            }
            at = at + 1 == RING ? 0 : at + 1;
        }
        copy_async_wait<0>();
    }
    if (!p.part)
        return;
    // the groups' sums, then their sum in the groups' order; a single group's go straight out
    float *sums = reinterpret_cast<float *>(raw); // [groups][2][cols]
    float *out_w = p.part + (uint64_t)blockIdx.x * p.cols, *out_b = p.part + (uint64_t)(p.parts + blockIdx.x) * p.cols;
    __syncthreads();
    if (works) {
        float *to_w = groups == 1 ? out_w : sums + (uint64_t)group * 2 * p.cols, *to_b = groups == 1 ? out_b : to_w + p.cols;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (t + k * width < n) {
                const uint32_t c = (t + k * width) * V;
                const float2 *pw = aw + k * V / 2, *pb = ab + k * V / 2;
                if constexpr (SHIFT) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < cols) {
                            to_w[c + i] = i & 1 ? pw[i / 2].y : pw[i / 2].x;
                            to_b[c + i] = i & 1 ? pb[i / 2].y : pb[i / 2].x;
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < V / 2; i += 2) {
                        *reinterpret_cast<float4 *>(to_w + c + 2 * i) = make_float4(pw[i].x, pw[i].y, pw[i + 1].x, pw[i + 1].y);
                        *reinterpret_cast<float4 *>(to_b + c + 2 * i) = make_float4(pb[i].x, pb[i].y, pb[i + 1].x, pb[i + 1].y);
                    }
                }
            }
    }
    if (groups == 1)
        return;
    __syncthreads();
    for (uint32_t c = tid; c < 2 * p.cols; c += NT) {
        float s = 0.f;
        for (uint32_t k = 0; k < groups; ++k)
            s += sums[k * 2 * p.cols + c];
        (c < p.cols ? out_w + c : out_b + (c - p.cols))[0] = s;
    }
}

namespace {

bool whole(const void *p, uint64_t ld, uint32_t size) { return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0; }

unsigned row_grid(uint64_t rows) { return (unsigned)std::min<uint64_t>(rows, 1u << 20); }

template <typename T, typename TO, int V> bool norm_registers(const NormParams &p, int sms, cudaStream_t st)
{
    // Accesses a thread.  Few rows: 8 values, a row over as many warps as it
    // takes (its latency counts); many: four accesses of aligned rows or 16
    // values, fewer warps to join.
    const uint64_t n = p.cols / V;
    constexpr uint64_t few = 8 / V, many = V == 1 ? 16 : 4;
    const bool plenty = p.rows >= 16ull * sms;
    const uint64_t per = (p.rows < 4ull * sms && n <= 1024 * few) || (plenty && n <= 32 * few) ? few : many;
    if (n > 1024 * many)
        return false;
    const uint64_t warps = (n + 32 * per - 1) / (32 * per);
    // several rows a team where blocks of four warps hold them and there are plenty
    const uint64_t rows = !plenty || warps > 4 ? 1 : per == few ? 4 : 2;
    const uint64_t teams = (p.rows + rows - 1) / rows, blocks = warps == 1 ? (teams + 3) / 4 : teams;
    if (blocks >= (1ull << 31))
        return false;
    const unsigned threads = warps == 1 ? 128 : (unsigned)warps * 32;
    const auto f = per == few  ? (rows == 1 ? norm_kernel<T, TO, V, few * V, 1> : norm_kernel<T, TO, V, few * V, 4>)
                   : rows == 1 ? norm_kernel<T, TO, V, many * V, 1>
                               : norm_kernel<T, TO, V, many * V, 2>;
    f<<<(unsigned)blocks, threads, 0, st>>>(p, (uint32_t)warps);
    return true;
}

template <typename T, typename TO> bool norm_shifted(const NormParams &p, int sms, cudaStream_t st)
{
    constexpr uint64_t V = 16 / sizeof(T), per = 4;
    const uint64_t n = (p.cols + V - 1) / V, warps = (n + 32 * per - 1) / (32 * per);
    // (a value an access is as fast on short rows and for few)
    if (warps > 16 || p.cols < 512 || p.rows * p.cols < (1ull << 20))
        return false;
    const uint64_t blocks = warps == 1 ? (p.rows + 3) / 4 : p.rows;
    if (blocks >= (1ull << 31))
        return false;
    const auto f = norm_shifted_kernel<T, TO, per * V>;
    f<<<(unsigned)blocks, warps == 1 ? 128 : (unsigned)warps * 32, 0, st>>>(p, (uint32_t)warps);
    return true;
}

template <typename T, typename TO> ecc_status norm_launch_to(const NormParams &p, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    // 16-byte accesses where every row, the output (8 or 4 bytes for e4m3)
    // and the parameters allow them
    const bool vec = p.cols % V == 0 && whole(p.x, p.ldx, sizeof(T)) && ((uintptr_t)p.y & (V * sizeof(TO) - 1)) == 0 &&
                     p.ldy % V == 0 && (p.p_type != TypeCode<T>::value || (whole(p.weight, 0, 1) && whole(p.bias, 0, 1)));
    if (!(vec ? norm_registers<T, TO, V>(p, sms, st) : norm_shifted<T, TO>(p, sms, st) || norm_registers<T, TO, 1>(p, sms, st)))
        norm_rows_kernel<T, TO><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

template <typename T> ecc_status norm_launch(const NormParams &p, uint32_t y_type, cudaStream_t st)
{
    return y_type == ECC_E4M3 ? norm_launch_to<T, e4m3>(p, st) : norm_launch_to<T, T>(p, st);
}

template <typename T, int NT, int E, int RING, int ROWS, bool SHIFT>
bool norm_grad_registers(NormGradParams &p, cudaStream_t st)
{
    constexpr uint64_t V = 16 / sizeof(T);
    const uint64_t width = (p.cols + E * 32 - 1) / (E * 32) * 32;
    if (width > NT)
        return false;
    const uint64_t steps = (p.rows + ROWS - 1) / ROWS, groups = NT / width;
    const size_t row = (width * (E / V) + SHIFT) * 16;
    const size_t smem = std::max<size_t>(groups * RING * ROWS * 2 * row, p.part && groups > 1 ? groups * p.cols * 8 : 0);
    const void *f = (const void *)norm_grad_kernel<T, NT, E, RING, ROWS, SHIFT>;
    if (smem > kMaxDynSmem - 2048 || occupancy(f, NT, smem) <= 0)
        return false;
    p.parts = (uint32_t)std::min<uint64_t>((steps + groups - 1) / groups, p.parts);
    norm_grad_kernel<T, NT, E, RING, ROWS, SHIFT><<<p.parts, NT, smem, st>>>(p, (uint32_t)width);
    return true;
}

// Values a thread.  float32: the fewest that let a block of 512 threads hold a
// row (its threads' sums take 128 registers).  16-bit types, rows of up to
// 4096: 8 values and 4 rows a step or 16 and 2, whichever leaves fewer threads
// without columns (16384 x 2049: 113 us with 8, 82 with 16; 20000 x 514: 39
// and 45); else 8 for few rows (2400 x 4096: 20.5 and 22.5 us; 16384 x 4096:
// 73.6 and 71.4).  Longer ones: at last 1024 threads.
template <typename T, bool SHIFT> bool norm_grad_any(NormGradParams &p, int sms, cudaStream_t st)
{
    if constexpr (sizeof(T) == 4)
        return norm_grad_registers<T, 512, 8, 3, 2, SHIFT>(p, st) || norm_grad_registers<T, 512, 16, 3, 1, SHIFT>(p, st);
    else {
        auto groups = [&](uint64_t e) { return 512 / ((p.cols + e * 32 - 1) / (e * 32) * 32); };
        const uint64_t g8 = 2 * groups(8), g16 = groups(16); // (in halves: a group of 16 values a thread covers twice the columns)
        if ((g8 > g16 || (g8 == g16 && p.rows < 64ull * sms)) && norm_grad_registers<T, 512, 8, 3, 4, SHIFT>(p, st))
            return true;
        return norm_grad_registers<T, 512, 16, 3, 2, SHIFT>(p, st) || norm_grad_registers<T, 1024, 16, 3, 1, SHIFT>(p, st);
    }
}

template <typename T> ecc_status norm_grad_launch(NormGradParams p, cudaStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    const bool sums = p.dweight || p.dbias;
    const unsigned cb = (unsigned)((p.cols + kNormThreads - 1) / kNormThreads);
    p.parts = (uint32_t)std::min<uint64_t>({kNormParts, p.rows, (uint64_t)sms});
    if (!sums)
        p.part = nullptr;
    bool done = !p.rows;
    if (p.rows) {
        const bool vec = p.cols % V == 0 && whole(p.x, p.ldx, sizeof(T)) && whole(p.dy, p.lddy, sizeof(T)) &&
                         (!p.dx || whole(p.dx, p.lddx, sizeof(T))) &&
                         (p.p_type != TypeCode<T>::value || whole(p.weight, 0, 1));
        done = vec ? norm_grad_any<T, false>(p, sms, st) : norm_grad_any<T, true>(p, sms, st);
    }
    if (!done) { // longer rows
        if (sums) // before dx, which may overwrite dy or x
            norm_dw_rows_kernel<T><<<dim3(cb, p.parts), kNormThreads, 0, st>>>(p);
        if (p.dx)
            norm_dx_rows_kernel<T><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    }
    const ecc_status rc = launch_status(cudaGetLastError());
    if (rc != ECC_OK || !sums)
        return rc;
    const dim3 grid((unsigned)((p.cols + 31) / 32), 2);
    if (p.rows && done) // lets it start early
        return launch_status(launch_behind(norm_parts_kernel, grid, 512, 0, st, (const float *)p.part, p.parts, p.cols,
                                           p.dweight, p.dbias));
    norm_parts_kernel<<<grid, 512, 0, st>>>(p.part, p.parts, p.cols, p.dweight, p.dbias);
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
