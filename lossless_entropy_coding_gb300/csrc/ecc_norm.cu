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

// a block: 32 columns, the parts in eight shares
__global__ void __launch_bounds__(kNormThreads) norm_parts_kernel(const float *part, uint32_t parts, uint64_t cols,
                                                                  float *dweight, float *dbias)
{
    __shared__ float sums[8][33];
    const uint32_t tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const uint64_t c = (uint64_t)blockIdx.x * 32 + tx;
    float *out = blockIdx.y ? dbias : dweight;
    if (!out)
        return;
    part += (uint64_t)blockIdx.y * parts * cols;
    float s = 0.f;
    if (c < cols)
        for (uint32_t k = ty; k < parts; k += 8)
            s += part[k * cols + c];
    sums[ty][tx] = s;
    __syncthreads();
    if (ty || c >= cols)
        return;
    for (int k = 1; k < 8; ++k)
        s += sums[k][tx];
    out[c] = s;
}

// ---------------------------------------------------------------- rows in registers
// V consecutive elements as one memory access
template <typename T, int V> struct alignas(V * sizeof(T)) Pack {
    T v[V];
};
// not through the read-only path: the output may be the input
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T *p)
{
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T *p, const float (&f)[V])
{
    Pack<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i)
        o.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = o;
}
template <int V> __device__ __forceinline__ void store_pack(e4m3 *p, const float (&f)[V])
{
    if constexpr (V % 2 == 0) {
        Pack<uint16_t, V / 2> o;
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            o.v[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<Pack<uint16_t, V / 2> *>(p) = o;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            p[i] = from_f32<e4m3>(f[i]);
    }
}
// V parameters from column c: of the rows' type in one access, or float32
template <typename T, int V> __device__ __forceinline__ void load_params(const void *p, uint64_t c, uint32_t type, float (&f)[V])
{
    if (type == TypeCode<T>::value) {
        const Pack<T, V> q = load_pack<T, V>(static_cast<const T *>(p) + c);
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = to_f32(q.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = static_cast<const float *>(p)[c + i];
    }
}

// A row by `warps` warps, PER accesses of V elements a thread: the row is
// read once and both passes over it (the mean, the squared deviations) run
// on registers.  Blocks of one warp a row hold four rows.  Bound by HBM: the
// row read, the output written.
template <typename T, typename TO, int V, int PER>
__global__ void __launch_bounds__(1024) norm_kernel(NormParams p, uint32_t warps)
{
    __shared__ float part[2][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = warps * 32;
    const uint64_t r = warps == 1 ? (uint64_t)blockIdx.x * (blockDim.x / 32) + warp : blockIdx.x;
    if (r >= p.rows)
        return; // (whole warps of a block of one warp a row)
    const uint32_t t = warps == 1 ? lane : threadIdx.x, n = (uint32_t)(p.cols / V);
    const T *x = static_cast<const T *>(p.x) + r * p.ldx;
    Pack<T, V> q[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (t + k * width < n)
            q[k] = load_pack<T, V>(x + (uint64_t)(t + k * width) * V);
    auto total = [&](float s, int which) {
        s = warp_sum(s);
        if (warps == 1)
            return s;
        if (lane == 0)
            part[which][warp] = s;
        __syncthreads();
        s = lane < warps ? part[which][lane] : 0.f;
        return warp_sum(s);
    };
    const float inv = 1.f / (float)p.cols;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (t + k * width < n) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                s += to_f32(q[k].v[i]);
        }
    const float mean = total(s, 0) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (t + k * width < n) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(q[k].v[i]) - mean;
                s += d * d;
            }
        }
    const float rstd = 1.f / sqrtf(total(s, 1) * inv + p.eps);
    TO *y = static_cast<TO *>(p.y) + r * p.ldy;
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (t + k * width < n) {
            const uint64_t c = (uint64_t)(t + k * width) * V;
            float f[V], w[V], b[V];
            if (p.weight)
                load_params<T, V>(p.weight, c, p.p_type, w);
            if (p.bias)
                load_params<T, V>(p.bias, c, p.p_type, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[i] = (to_f32(q[k].v[i]) - mean) * rstd;
                if (p.weight)
                    f[i] *= w[i];
                if (p.bias)
                    f[i] += b[i];
                f[i] *= p.y_scale;
            }
            if constexpr (sizeof(TO) == 1)
                store_pack<V>(y + c, f);
            else
                store_pack<TO, V>(y + c, f);
        }
    if (t == 0) {
        if (p.mean)
            p.mean[r] = mean;
        if (p.rstd)
            p.rstd[r] = rstd;
    }
}

// ---------------------------------------------------------------- backward, rows in registers
constexpr int kGradThreads = 1024; // a block an SM; groups of `width` threads take a row each
constexpr int kGradWarps = kGradThreads / 32;

// groups of a block; each of several warps has a barrier of its own (1 to 15)
__host__ __device__ inline uint32_t grad_groups(uint32_t width)
{
    const uint32_t g = kGradThreads / width;
    return width > 32 && g > 15 ? 15 : g;
}

__device__ __forceinline__ void group_barrier(uint32_t id, uint32_t threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Persistent: a group of `width` threads walks the rows g, g + groups, ...;
// each thread keeps its columns' sums of dy * xh and dy in registers, so x
// and dy are read once for all three gradients.  With RING > 0 a thread
// copies its 16-byte pieces of the next RING - 1 rows ahead into its own
// part of shared memory (nobody else reads it: no barrier); otherwise
// (elements on other boundaries) it loads as it goes.  One barrier a row joins the
// warps' sums.  The groups' column sums are added in shared memory and the
// blocks' in norm_parts_kernel, both in a fixed order.  Bound by HBM.
template <typename T, int V, int PER, int RING>
__global__ void __launch_bounds__(kGradThreads, 1) norm_grad_kernel(NormGradParams p, uint32_t width)
{
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ float2 part[2][kGradWarps];
    const uint32_t tid = threadIdx.x, lane = tid & 31, group = tid / width, t = tid - group * width;
    const uint32_t groups = grad_groups(width), warps = width / 32, warp0 = group * warps, warp = tid >> 5;
    const uint32_t n = (uint32_t)(p.cols / V);
    const uint64_t step = (uint64_t)gridDim.x * groups;
    const float inv = 1.f / (float)p.cols;
    float w[PER][V], aw[PER][V], ab[PER][V];
#pragma unroll
    for (int k = 0; k < PER; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = 1.f;
            aw[k][i] = ab[k][i] = 0.f;
        }
    const bool works = group < groups; // threads past the last whole group only join the barriers of the end
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    T *dx = static_cast<T *>(p.dx);
    if (works) {
        if (p.weight)
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (t + k * width < n)
                    load_params<T, V>(p.weight, (uint64_t)(t + k * width) * V, p.p_type, w[k]);
        const uint64_t r0 = (uint64_t)blockIdx.x * groups + group;
        const uint32_t slots = smem_u32(raw) + tid * 16; // piece s of a row's 2 PER at s * kGradThreads * 16
        auto fetch = [&](uint64_t r, uint32_t at) {
            if constexpr (RING > 0) {
                if (r < p.rows)
#pragma unroll
                    for (int k = 0; k < PER; ++k)
                        if (t + k * width < n) {
                            const uint64_t c = (uint64_t)(t + k * width) * V;
                            copy_async16(slots + (at * 2 * PER + 2 * k) * kGradThreads * 16, x + r * p.ldx + c);
                            copy_async16(slots + (at * 2 * PER + 2 * k + 1) * kGradThreads * 16, dy + r * p.lddy + c);
                        }
                copy_async_commit();
            }
        };
#pragma unroll
        for (int k = 0; k + 1 < RING; ++k)
            fetch(r0 + k * step, k);
        uint32_t at = 0, flip = 0;
        for (uint64_t r = r0; r < p.rows; r += step) {
            Pack<T, V> xq[PER], dq[PER];
            const float mean = p.mean[r], rstd = p.rstd[r];
            if constexpr (RING > 0) {
                fetch(r + (RING - 1) * step, at ? at - 1 : RING - 1);
                copy_async_wait<RING - 1>();
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    xq[k] = *reinterpret_cast<const Pack<T, V> *>(raw + ((at * 2 * PER + 2 * k) * kGradThreads + tid) * 16);
                    dq[k] = *reinterpret_cast<const Pack<T, V> *>(raw + ((at * 2 * PER + 2 * k + 1) * kGradThreads + tid) * 16);
                }
                at = at + 1 == RING ? 0 : at + 1;
            } else {
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if (t + k * width < n) {
                        xq[k] = load_pack<T, V>(x + r * p.ldx + (uint64_t)(t + k * width) * V);
                        dq[k] = load_pack<T, V>(dy + r * p.lddy + (uint64_t)(t + k * width) * V);
                    }
            }
            float s = 0.f, q = 0.f;
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (t + k * width < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = to_f32(dq[k].v[i]), xh = (to_f32(xq[k].v[i]) - mean) * rstd, g = d * w[k][i];
                        s += g;
                        q += g * xh;
                        aw[k][i] += d * xh;
                        ab[k][i] += d;
                    }
                }
            if (!p.dx)
                continue;
            s = warp_sum(s);
            q = warp_sum(q);
            if (warps > 1) {
                if (lane == 0)
                    part[flip][warp] = make_float2(s, q);
                group_barrier(group, width);
                const float2 o = lane < warps ? part[flip][warp0 + lane] : make_float2(0.f, 0.f);
                s = warp_sum(o.x);
                q = warp_sum(o.y);
                flip ^= 1;
            }
            s *= inv;
            q *= inv;
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (t + k * width < n) {
                    float f[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float xh = (to_f32(xq[k].v[i]) - mean) * rstd;
                        f[i] = rstd * (to_f32(dq[k].v[i]) * w[k][i] - s - xh * q);
                    }
                    store_pack<T, V>(dx + r * p.lddx + (uint64_t)(t + k * width) * V, f);
                }
        }
        if constexpr (RING > 0)
            copy_async_wait<0>();
    }
    if (!p.part)
        return;
    // the groups' sums, one group after the other
    float *sums = reinterpret_cast<float *>(raw); // [2][cols]
    for (uint32_t g = 0; g < groups; ++g) {
        __syncthreads();
        if (works && group == g)
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (t + k * width < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t c = (t + k * width) * V + i;
                        const float a = aw[k][i], b = ab[k][i];
                        sums[c] = g ? sums[c] + a : a;
                        sums[p.cols + c] = g ? sums[p.cols + c] + b : b;
                    }
                }
    }
    __syncthreads();
    for (uint32_t c = tid; c < p.cols; c += kGradThreads) {
        p.part[(uint64_t)blockIdx.x * p.cols + c] = sums[c];
        p.part[(uint64_t)(p.parts + blockIdx.x) * p.cols + c] = sums[p.cols + c];
    }
}

namespace {

bool whole(const void *p, uint64_t ld, uint32_t size) { return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0; }

unsigned row_grid(uint64_t rows) { return (unsigned)std::min<uint64_t>(rows, 1u << 20); }

template <typename T, typename TO, int V> bool norm_registers(const NormParams &p, int sms, cudaStream_t st)
{
    // few rows: spread a row over more warps (its latency counts); many: a
    // warp a row while 16 accesses a thread hold it (no barriers)
    const uint64_t n = p.cols / V;
    const uint64_t per = p.rows < 4ull * sms ? 1 : n <= 32 * 4 ? 4 : 16;
    uint64_t warps = 1;
    while (warps < 32 && warps * 32 * per < n)
        warps *= 2;
    const uint64_t need = (n + warps * 32 - 1) / (warps * 32);
    if (need > 16)
        return false;
    const uint64_t blocks = warps == 1 ? (p.rows + 3) / 4 : p.rows;
    if (blocks >= (1ull << 31))
        return false;
    const unsigned threads = warps == 1 ? 128 : (unsigned)warps * 32;
    if (need == 1)
        norm_kernel<T, TO, V, 1><<<(unsigned)blocks, threads, 0, st>>>(p, (uint32_t)warps);
    else if (need <= 4)
        norm_kernel<T, TO, V, 4><<<(unsigned)blocks, threads, 0, st>>>(p, (uint32_t)warps);
    else
        norm_kernel<T, TO, V, 16><<<(unsigned)blocks, threads, 0, st>>>(p, (uint32_t)warps);
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
    if (!(vec ? norm_registers<T, TO, V>(p, sms, st) : norm_registers<T, TO, 1>(p, sms, st)))
        norm_rows_kernel<T, TO><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

template <typename T> ecc_status norm_launch(const NormParams &p, uint32_t y_type, cudaStream_t st)
{
    return y_type == ECC_E4M3 ? norm_launch_to<T, e4m3>(p, st) : norm_launch_to<T, T>(p, st);
}

template <typename T, int V, int PER, int RING>
bool norm_grad_registers(const NormGradParams &p, unsigned grid, uint32_t width, cudaStream_t st)
{
    const size_t smem = std::max<size_t>((size_t)RING * 2 * PER * kGradThreads * 16, p.part ? p.cols * 8 : 0);
    const void *f = (const void *)norm_grad_kernel<T, V, PER, RING>;
    if (smem > kMaxDynSmem - 1024 || occupancy(f, kGradThreads, smem) <= 0)
        return false;
    norm_grad_kernel<T, V, PER, RING><<<grid, kGradThreads, smem, st>>>(p, width);
    return true;
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
        const uint64_t n = vec ? p.cols / V : p.cols;
        const uint64_t per = vec ? (n > kGradThreads ? 2 : 1) : 8; // accesses a thread
        const uint64_t width = (n + per * 32 - 1) / (per * 32) * 32;
        if (width <= kGradThreads) {
            const uint32_t w = (uint32_t)width, g = grad_groups(w);
            p.parts = (uint32_t)std::min<uint64_t>((p.rows + g - 1) / g, p.parts);
            done = !vec       ? norm_grad_registers<T, 1, 8, 0>(p, p.parts, w, st)
                   : per == 1 ? norm_grad_registers<T, V, 1, 4>(p, p.parts, w, st)
                              : norm_grad_registers<T, V, 2, 3>(p, p.parts, w, st);
        }
    }
    if (!done) { // longer rows
        if (sums) // before dx, which may overwrite dy or x
            norm_dw_rows_kernel<T><<<dim3(cb, p.parts), kNormThreads, 0, st>>>(p);
        if (p.dx)
            norm_dx_rows_kernel<T><<<row_grid(p.rows), kNormThreads, 0, st>>>(p);
    }
    if (sums)
        norm_parts_kernel<<<dim3((unsigned)((p.cols + 31) / 32), 2), kNormThreads, 0, st>>>(p.part, p.parts, p.cols, p.dweight,
                                                                                           p.dbias);
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
