// ecc_linear.cuh -- what the operators around a matrix product share: operands
// made readable for the products, products of a few rows, column sums in a
// fixed order.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "ecc_act.cuh"
#include "ecc_gemm.h"

namespace ecc {

constexpr int kRowThreads = 256;

// V values from element i of an array, in pairs (V = 1: the second is 0)
template <typename T, int V> __device__ __forceinline__ void load_values(const void *p, uint64_t i, float2 (&f)[(V + 1) / 2])
{
    const T *q = static_cast<const T *>(p) + i;
    if constexpr (V == 1) {
        f[0] = make_float2(to_f32(*q), 0.f);
    } else {
        constexpr int E = 16 / sizeof(T);
#pragma unroll
        for (int k = 0; k < V; k += E)
            unpack2<T>(*reinterpret_cast<const uint4 *>(q + k), f + k / 2);
    }
}

// column sums of `parts` rows of n; from column n1 on they go to out2
static __global__ void __launch_bounds__(kRowThreads) sum_parts_kernel(const float *part, uint32_t parts, uint64_t n, float *out,
                                                                                uint64_t n1, float *out2)
{
    wait_for_previous();
    const uint64_t c = (uint64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (c >= n)
        return;
    float s = 0.f;
#pragma unroll 8
    for (uint32_t k = 0; k < parts; ++k)
        s += part[k * n + c];
    *(c < n1 ? out + c : out2 + (c - n1)) = s;
}

// k such that 2^k brings the largest of a float16 operand's magnitudes, `top`,
// to at least 2^14 and below 2^15 (as far as 2^k and 2^-k are ordinary numbers)
__device__ __forceinline__ int half_power(float top) { return top > 0.f ? max(-113, min(112, 14 - ilogbf(top))) : 0; }

// Rows of `cols` elements to rows of ldd elements on 16-byte boundaries, for
// up to three operands in one launch (blockIdx.y): the two vectors around each
// 16 bytes, shifted, at the rate of a copy (820 MB read and written in 118 us;
// five words around them 134).
struct PadJob {
    const void *src;
    void *dst;
    uint64_t ld, rows, cols, ldd;
};
struct PadJobs {
    PadJob j[3];
};
template <typename T> __global__ void __launch_bounds__(kRowThreads) pad_rows_kernel(const __grid_constant__ PadJobs jobs)
{
    constexpr int V = 16 / sizeof(T);
    let_next_start();
    const PadJob &j = jobs.j[blockIdx.y];
    const uint32_t vecs = (uint32_t)(j.ldd / V);
    const uint64_t n = j.rows * vecs;
    const T *src = static_cast<const T *>(j.src), *end = src + (j.rows - 1) * j.ld + j.cols;
    T *dst = static_cast<T *>(j.dst);
#pragma unroll 2
    for (uint64_t i = (uint64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += (uint64_t)gridDim.x * kRowThreads) {
        const uint64_t r = n >> 32 ? i / vecs : (uint32_t)i / vecs;
        const uint32_t at = (uint32_t)(i - r * vecs) * V;
        const T *s = src + r * j.ld + at;
        uint4 q;
        const uintptr_t low = (uintptr_t)s & ~(uintptr_t)15;
        if (at + V <= j.cols && low >= (uintptr_t)src && low + 32 <= (uintptr_t)end) { // the two vectors around the 16 bytes
            q = shift16<false>(*reinterpret_cast<const uint4 *>(low), *reinterpret_cast<const uint4 *>(low + 16),
                               (uint32_t)((uintptr_t)s - low));
        } else { // a row's last ones, the array's first and last
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (at + k < j.cols)
                    w[k * sizeof(T) / 4] |= (uint32_t)s[k] << k * sizeof(T) % 4 * 8;
            q = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4 *>(dst + i * V) = q;
    }
}

// ---------------------------------------------------------------- few rows
constexpr int kFewColumns = 4;
struct FewRows {
    const void *x, *w;
    uint64_t ldx, ldw, N, K;
    uint32_t warps; // that share kFewColumns rows of the weights
    Epilogue e;
    uint32_t *status;
    const void *w2; // the ups' weights (w: the gates'), for gated products
    uint64_t ldw2;
};
template <typename T> __device__ __forceinline__ void unpack_all(const uint4 &q, float2 (&f)[8 / sizeof(T)])
{
    if constexpr (sizeof(T) == 2) {
        unpack2<T>(q, f);
    } else {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i / 2] >> (i & 1) * 16), __NV_E4M3);
            f[i] = __half22float2(__half2(h));
        }
    }
}
// M rows of x by the rows of w, on any boundaries: the weights are read once,
// as vectors shifted from the aligned ones around them, and multiplied as they
// come.  A warp (or p.warps of them) takes four columns of the output, so that
// they share the conversion of x; its lanes' sums are joined in a fixed order.
// Bound by HBM for one token, 1 x 16384 x 4096 bf16 25.5 us, 5.3 TB/s, 1 x
// 12616 x 14088 63 us, 5.6 TB/s (at 1 x 16384 x 4096, two columns a warp 29.5,
// two vectors of four columns at a time 30.1, the next vectors loaded ahead
// 30.7); off 16-byte boundaries by the shifts, the second 129 us; with more
// rows by the multiplications, M of them a weight.
// Gated: the four are two columns' gates and ups.
template <typename T, int M, bool GATED>
__global__ void __launch_bounds__(kRowThreads) few_rows_kernel(const __grid_constant__ FewRows p)
{
    constexpr int R = kFewColumns, C = GATED ? R / 2 : R, V = 16 / sizeof(T), H = V / 2, OUT = R * M;
    __shared__ float sums[8][OUT];
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.status = ECC_OK;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / p.warps, part = warp % p.warps;
    const uint64_t n0 = ((uint64_t)blockIdx.x * (8 / p.warps) + group) * C;
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    const T *x_end = x + (M - 1) * p.ldx + p.K, *w_end = w + (p.N - 1) * p.ldw + p.K;
    const T *w2 = GATED ? static_cast<const T *>(p.w2) : w, *w2_end = GATED ? w2 + (p.N - 1) * p.ldw2 + p.K : w_end;
    const T *wr[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        wr[r] = r < C ? w + min(n0 + r, p.N - 1) * p.ldw : w2 + min(n0 + r - C, p.N - 1) * p.ldw2;
    float2 acc[R][M];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m)
            acc[r][m] = both(0.f);
    const uint64_t vecs = p.K / V, step = (uint64_t)p.warps * 32;
    for (uint64_t v = part * 32 + lane; v < vecs; v += step) {
        float2 f[R][H];
        uint4 q[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            q[r] = load_anywhere(wr[r] + v * V, r < C ? w : w2, r < C ? w_end : w2_end);
#pragma unroll
        for (int r = 0; r < R; ++r)
            unpack_all<T>(q[r], f[r]);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float2 g[H];
            unpack_all<T>(load_anywhere(x + m * p.ldx + v * V, x, x_end), g);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < H; ++i)
                    acc[r][m] = fma2(f[r][i], g[i], acc[r][m]);
        }
    }
    if (part == 0)
        for (uint64_t k = vecs * V + lane; k < p.K; k += 32)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int m = 0; m < M; ++m)
                    acc[r][m].x = fmaf(to_f32(wr[r][k]), to_f32(x[m * p.ldx + k]), acc[r][m].x);
    float a = 0.f; // lane r M + m keeps column r's sum of row m
#pragma unroll
    for (int i = 0; i < OUT; ++i) {
        const float t = warp_sum(acc[i / M][i % M].x + acc[i / M][i % M].y);
        if (lane == i)
            a = t;
    }
    if (p.warps > 1) {
        if (lane < OUT)
            sums[warp][lane] = a;
        __syncthreads();
        if (part)
            return;
        if (lane < OUT)
            for (uint32_t i = 1; i < p.warps; ++i)
                a += sums[warp + i][lane];
    }
    const bool up = GATED && lane >= C * M;
    const uint64_t c = n0 + lane / M - (up ? C : 0), r = lane % M;
    const Epilogue &e = p.e;
    const bool ok = lane < OUT && c < p.N;
    if (!GATED && !ok)
        return;
    const void *bias = up ? e.bias2 : e.bias;
    a = a * (up ? e.scale2 : e.scale) + (bias && ok ? load_any(bias, c, e.bias_type) : 0.f);
    if (e.pre && ok)
        store_any(up ? e.pre2 : e.pre, r * (up ? e.ldpre2 : e.ldpre) + c, e.pre_type, a);
    float other = 1.f;
    if constexpr (GATED) {
        other = __shfl_down_sync(~0u, a, C * M);
        if (up || !ok)
            return;
    }
    if (e.act == ECC_ACT_RELU)
        a = act_value2<ECC_ACT_RELU>(both(a)).x;
    else if (e.act == ECC_ACT_GELU)
        a = act_value2<ECC_ACT_GELU>(both(a)).x;
    else if (e.act == ECC_ACT_GELU_TANH)
        a = act_value2<ECC_ACT_GELU_TANH>(both(a)).x;
    else if (e.act == ECC_ACT_SILU)
        a = act_value2<ECC_ACT_SILU>(both(a)).x;
    if constexpr (GATED)
        a *= other;
    if (e.residual)
        a += load_any(e.residual, r * e.ldres + c, e.res_type);
    store_any(e.out, r * e.ldout + c, e.out_type, e.out_type == ECC_E4M3 ? a * e.out_scale : a);
}

constexpr uint64_t kMostDim = 1ull << 31;

inline uint64_t padded(uint64_t cols, uint32_t type)
{
    const uint64_t v = 16 / type_bytes(type);
    return (cols + v - 1) / v * v;
}
inline size_t pad256(size_t b) { return (b + 255) / 256 * 256; }
inline size_t copy_bytes(const void *p, uint64_t ld, uint64_t rows, uint64_t cols, uint32_t type)
{
    return rows && cols && !tma_rows(p, ld, type, rows) ? pad256(rows * padded(cols, type) * type_bytes(type)) : 0;
}

// The operands (arrays of `type`), each itself or its copy at ws (advanced
// past it); rows = 0: not wanted.  `launched`: whether something was.
struct Array {
    const void *p;
    uint64_t ld, rows, cols;
    Operand *o;
};
inline ecc_status readable(std::initializer_list<Array> arrays, uint32_t type, uint8_t *&ws, cudaStream_t st, bool &launched)
{
    launched = false;
    PadJobs jobs{};
    int n = 0;
    uint64_t most = 0;
    for (const Array &x : arrays) {
        *x.o = {x.p, x.ld, false};
        const size_t bytes = copy_bytes(x.p, x.ld, x.rows, x.cols, type);
        if (bytes) {
            *x.o = {ws, padded(x.cols, type), false};
            jobs.j[n++] = {x.p, ws, x.ld, x.rows, x.cols, x.o->ld};
            most = std::max<uint64_t>(most, bytes / 16);
            ws += bytes;
        }
    }
    if (!n)
        return ECC_OK;
    const dim3 grid((unsigned)std::min<uint64_t>((most + kRowThreads - 1) / kRowThreads, 1u << 15), n);
    if (type == ECC_E4M3)
        pad_rows_kernel<uint8_t><<<grid, kRowThreads, 0, st>>>(jobs);
    else
        pad_rows_kernel<uint16_t><<<grid, kRowThreads, 0, st>>>(jobs);
    launched = true;
    return launch_status(cudaGetLastError());
}

template <typename T, bool GATED> void few_rows_launch(uint64_t M, FewRows p, int sms, cudaStream_t st)
{
    // more warps to four columns while 16 an SM are not reached, each with two vectors a lane at least (32 an SM: 1 x
    // 4096 x 4096 9.3 us instead of 8.2, 1 x 12616 x 14088 66 instead of 63)
    constexpr int C = GATED ? kFewColumns / 2 : kFewColumns;
    const uint64_t teams = (p.N + C - 1) / C;
    p.warps = 1;
    while (p.warps < 8 && teams * p.warps < 16ull * sms && p.K * sizeof(T) >= 2048ull * p.warps)
        p.warps *= 2;
    const unsigned blocks = (unsigned)((teams * p.warps + 7) / 8);
    const auto f = M == 1   ? few_rows_kernel<T, 1, GATED>
                   : M == 2 ? few_rows_kernel<T, 2, GATED>
                   : M == 3 ? few_rows_kernel<T, 3, GATED>
                            : few_rows_kernel<T, 4, GATED>;
    f<<<blocks, kRowThreads, 0, st>>>(p);
}

} // namespace ecc
