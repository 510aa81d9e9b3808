// ecc_linear.cu -- a layer's matrix product with its epilogue (scale, bias,
// activation, residual), and its backward pass: t = dy * act'(pre) with the
// bias gradient, then the two products (ecc_gemm.cu).
//
// The products read their operands by TMA, which wants rows on 16-byte
// boundaries: an operand with other rows is first copied to the workspace
// with padded rows.  Products of a few rows read theirs as they lie.

#include <algorithm>
#include <cmath>

#include "ecc_act.cuh"
#include "ecc_gemm.h"

namespace ecc {

constexpr int kRowThreads = 256;
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

__global__ void __launch_bounds__(kRowThreads) sum_parts_kernel(const float *part, uint32_t parts, uint64_t n, float *out)
{
    wait_for_previous();
    const uint64_t c = (uint64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (c >= n)
        return;
    float s = 0.f;
#pragma unroll 8
    for (uint32_t k = 0; k < parts; ++k)
        s += part[k * n + c];
    out[c] = s;
}

// Rows of `cols` elements to rows of ldd elements on 16-byte boundaries, for
// up to two operands in one launch (blockIdx.y).
struct PadJob {
    const void *src;
    void *dst;
    uint64_t ld, rows, cols, ldd;
};
template <typename T> __global__ void __launch_bounds__(kRowThreads) pad_rows_kernel(PadJob a, PadJob b)
{
    constexpr int V = 16 / sizeof(T);
    let_next_start();
    const PadJob &j = blockIdx.y ? b : a;
    const uint32_t vecs = (uint32_t)(j.ldd / V);
    const uint64_t n = j.rows * vecs;
    for (uint64_t i = (uint64_t)blockIdx.x * kRowThreads + threadIdx.x; i < n; i += (uint64_t)gridDim.x * kRowThreads) {
        const uint64_t r = n >> 32 ? i / vecs : (uint32_t)i / vecs;
        const uint32_t c = (uint32_t)(i - r * vecs) * V;
        const T *s = static_cast<const T *>(j.src) + r * j.ld + c;
        uint32_t o[4];
        const uint32_t off = (uint32_t)(uintptr_t)s & 3;
        if (c + V + 4 / sizeof(T) <= j.cols && c) { // five words around the 16 bytes, all inside the row
            const uint32_t *w = reinterpret_cast<const uint32_t *>((uintptr_t)s & ~(uintptr_t)3);
            uint32_t q[5];
#pragma unroll
            for (int k = 0; k < 5; ++k)
                q[k] = w[k];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = __funnelshift_r(q[k], q[k + 1], off * 8);
        } else { // a row's first and last ones
            struct alignas(16) {
                T v[V];
            } t;
#pragma unroll
            for (int k = 0; k < V; ++k)
                t.v[k] = c + k < j.cols ? s[k] : T(0);
            const uint4 q = *reinterpret_cast<const uint4 *>(&t);
            o[0] = q.x;
            o[1] = q.y;
            o[2] = q.z;
            o[3] = q.w;
        }
        *reinterpret_cast<uint4 *>(static_cast<T *>(j.dst) + r * j.ldd + c) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---------------------------------------------------------------- few rows
constexpr int kFewColumns = 4;
struct FewRows {
    const void *x, *w;
    uint64_t ldx, ldw, N, K;
    uint32_t warps; // that share kFewColumns columns of the output
    Epilogue e;
    uint32_t *status;
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
template <typename T, int M>
__global__ void __launch_bounds__(kRowThreads) few_rows_kernel(const __grid_constant__ FewRows p)
{
    constexpr int R = kFewColumns, V = 16 / sizeof(T), H = V / 2, OUT = R * M;
    __shared__ float sums[8][OUT];
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *p.status = ECC_OK;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / p.warps, part = warp % p.warps;
    const uint64_t n0 = ((uint64_t)blockIdx.x * (8 / p.warps) + group) * R;
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    const T *x_end = x + (M - 1) * p.ldx + p.K, *w_end = w + (p.N - 1) * p.ldw + p.K;
    const T *wr[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        wr[r] = w + min(n0 + r, p.N - 1) * p.ldw;
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
            q[r] = load_anywhere(wr[r] + v * V, w, w_end);
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
    const uint64_t c = n0 + lane / M, r = lane % M;
    if (lane >= OUT || c >= p.N)
        return;
    const Epilogue &e = p.e;
    a = a * e.scale + (e.bias ? load_any(e.bias, c, e.bias_type) : 0.f);
    if (e.pre)
        store_any(e.pre, r * e.ldpre + c, e.pre_type, a);
    if (e.act == ECC_ACT_RELU)
        a = act_value2<ECC_ACT_RELU>(both(a)).x;
    else if (e.act == ECC_ACT_GELU)
        a = act_value2<ECC_ACT_GELU>(both(a)).x;
    else if (e.act == ECC_ACT_GELU_TANH)
        a = act_value2<ECC_ACT_GELU_TANH>(both(a)).x;
    else if (e.act == ECC_ACT_SILU)
        a = act_value2<ECC_ACT_SILU>(both(a)).x;
    if (e.residual)
        a += load_any(e.residual, r * e.ldres + c, e.res_type);
    store_any(e.out, r * e.ldout + c, e.out_type, e.out_type == ECC_E4M3 ? a * e.out_scale : a);
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

// The operands (arrays a and b of `type`), each itself or its copy at ws
// (advanced past it); rows = 0: not wanted.  Whether something was launched.
struct Array {
    const void *p;
    uint64_t ld, rows, cols;
};
bool readable(const Array &a, const Array &b, uint32_t type, uint8_t *&ws, cudaStream_t st, Operand &oa, Operand &ob)
{
    PadJob jobs[2];
    int n = 0;
    uint64_t most = 0;
    auto one = [&](const Array &x, Operand &o) {
        o = {x.p, x.ld, false};
        const size_t bytes = copy_bytes(x.p, x.ld, x.rows, x.cols, type);
        if (bytes) {
            o = {ws, padded(x.cols, type), false};
            jobs[n++] = {x.p, ws, x.ld, x.rows, x.cols, o.ld};
            most = std::max<uint64_t>(most, bytes / 16);
            ws += bytes;
        }
    };
    one(a, oa);
    one(b, ob);
    if (!n)
        return false;
    const dim3 grid((unsigned)std::min<uint64_t>((most + kRowThreads - 1) / kRowThreads, 1u << 15), n);
    if (type == ECC_E4M3)
        pad_rows_kernel<uint8_t><<<grid, kRowThreads, 0, st>>>(jobs[0], jobs[n - 1]);
    else
        pad_rows_kernel<uint16_t><<<grid, kRowThreads, 0, st>>>(jobs[0], jobs[n - 1]);
    return true;
}

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
template <typename T> void few_rows_launch(const ecc_linear_job &j, FewRows p, int sms, cudaStream_t st)
{
    // more warps to four columns while 16 an SM are not reached, each with two vectors a lane at least (32 an SM: 1 x
    // 4096 x 4096 9.3 us instead of 8.2, 1 x 12616 x 14088 66 instead of 63)
    const uint64_t teams = (j.N + kFewColumns - 1) / kFewColumns;
    p.warps = 1;
    while (p.warps < 8 && teams * p.warps < 16ull * sms && j.K * sizeof(T) >= 2048ull * p.warps)
        p.warps *= 2;
    const unsigned blocks = (unsigned)((teams * p.warps + 7) / 8);
    const auto f = j.M == 1 ? few_rows_kernel<T, 1> : j.M == 2 ? few_rows_kernel<T, 2> : j.M == 3 ? few_rows_kernel<T, 3>
                                                                                                : few_rows_kernel<T, 4>;
    f<<<blocks, kRowThreads, 0, st>>>(p);
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
        const FewRows p{j.x, j.w, j.ldx, j.ldw, j.N, j.K, 1, e, status};
        if (j.in_type == ECC_BF16)
            few_rows_launch<bf16>(j, p, sms, st);
        else if (j.in_type == ECC_F16)
            few_rows_launch<__half>(j, p, sms, st);
        else
            few_rows_launch<e4m3>(j, p, sms, st);
        return launch_status(cudaGetLastError());
    }
    uint8_t *w = (uint8_t *)ws;
    Operand x, wt;
    const bool copied = readable({j.x, j.ldx, j.M, j.K}, {j.w, j.ldw, j.N, j.K}, j.in_type, w, st, x, wt);
    return gemm({wt, x, j.M, j.N, j.K, e}, j.in_type, status, true, copied, st);
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
    Operand x, wt; // read down their columns
    bool own = readable({j.x, j.ldx, j.dw ? j.M : 0, j.K}, {j.w, j.ldw, j.dx ? j.N : 0, j.K}, j.in_type, w, st, x, wt);
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
                                         st, (const float *)part, g.parts, j.N, j.dbias));
    if (rc == ECC_OK && clear)
        rc = launch_status(cudaMemsetAsync(status, 0, sizeof(uint32_t), st));
    return rc;
}

} // extern "C"
