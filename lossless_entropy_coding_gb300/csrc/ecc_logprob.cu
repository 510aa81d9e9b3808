// ecc_logprob.cu -- log probabilities of given tokens with the entropy and
// the most probable alternatives, and the gradient with respect to the
// logits.
//
// z = scale * x.  With m the row's maximum, s = sum e^(z - m) and
// t = sum e^(z - m) (z - m): lse = m + log s, log p[v] = z[v] - m - log s,
// H = log s - t / s.  (z[v] - lse would lose log s where |m| is large, as in
// a row of nothing but the type's lowest value, whose tokens are equally
// probable.)

#include <algorithm>
#include <cmath>

#include "ecc_lm.cuh"

namespace ecc {

constexpr int kLpThreads = 256;

struct LogprobParams {
    const void *logits;
    const int64_t *tokens;
    uint64_t ld, rows, vocab;
    float scale;
    uint32_t top;
    float *logprob, *entropy, *lse, *top_logprob;
    int32_t *top_index;
};

struct LogprobGradParams {
    const void *logits;
    const int64_t *tokens;
    uint64_t ld, ldd, rows, vocab;
    float scale;
    const float *lse, *entropy, *dlogprob, *dentropy;
    void *dlogits;
};

// Order of the alternatives as one unsigned number: larger logits first (NaN
// before +infinity, -0 = +0), equal ones by the lower index.
__device__ __forceinline__ uint32_t order_bits(float x)
{
    if (x != x)
        return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.f); // -0 + 0 = +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(float x, uint32_t index)
{
    return (uint64_t)order_bits(x) << 32 | (0xFFFFFFFFu - index);
}

// a row's results from its largest logit m and its sums
struct RowResult {
    float m, scale, logs, lse, entropy;
    __device__ __forceinline__ RowResult(float m_, float s, float t, float scale_)
        : m(m_), scale(scale_), logs(logf(s))
    {
        if (m == -INFINITY && s == 0.f) { // no token has a probability
            lse = -INFINITY;
            entropy = 0.f;
        } else if (m == INFINITY && s == s) {
            lse = INFINITY;
            entropy = NAN;
        } else {
            lse = m * scale + logs;
            entropy = logs - t / s;
        }
    }
    __device__ __forceinline__ float logprob(float x) const
    {
        return lse == -INFINITY ? -INFINITY : lse == INFINITY ? x - m : (x - m) * scale - logs;
    }
};

// log p in the gradient: from lse, unless lse is so large that rounding it
// to float32 (2^-24 |lse|) would show; the row's maximum and log sum are then
// found again.
constexpr float kLseMost = 256.f;

template <typename Op> __device__ __forceinline__ float block_reduce(float v, Op op)
{
    __shared__ float part[kLpThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = op(v, __shfl_xor_sync(~0u, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < kLpThreads / 32; ++i)
        v = op(v, part[i]);
    return v;
}

template <typename T> __global__ void __launch_bounds__(kLpThreads) logprob_rows_kernel(LogprobParams p)
{
    __shared__ unsigned long long best;
    auto add = [](float a, float b) { return a + b; };
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.logits) + r * p.ld;
        float m = -INFINITY, nan = 0.f;
        for (uint64_t i = threadIdx.x; i < p.vocab; i += kLpThreads) {
            const float v = to_f32(x[i]);
            m = fmaxf(m, v);
            nan += v != v;
        }
        m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); });
        nan = block_reduce(nan, add);
        float s = 0.f, t = 0.f;
        if (fabsf(m) < INFINITY)
            for (uint64_t i = threadIdx.x; i < p.vocab; i += kLpThreads) {
                const float d = (to_f32(x[i]) - m) * p.scale, e = expf(d);
                s += e;
                t += e > 0.f ? e * d : 0.f;
            }
        s = block_reduce(s, add);
        t = block_reduce(t, add);
        if (nan > 0.f)
            s = t = NAN;
        const RowResult res(m, s, t, p.scale);
        if (threadIdx.x == 0) {
            if (p.lse)
                p.lse[r] = res.lse;
            if (p.entropy)
                p.entropy[r] = res.entropy;
            if (p.logprob && p.tokens) {
                const int64_t tok = p.tokens[r];
                p.logprob[r] = tok < 0                   ? 0.f
                               : tok >= (int64_t)p.vocab ? NAN
                                                         : res.logprob(to_f32(x[tok]));
            }
        }
        uint64_t last = ~0ull; // one alternative a pass: the largest key below the last one
        for (uint32_t k = 0; k < p.top; ++k) {
            if (threadIdx.x == 0)
                best = 0;
            __syncthreads();
            uint64_t mine = 0;
            for (uint64_t i = threadIdx.x; i < p.vocab; i += kLpThreads) {
                const uint64_t key = order_key(to_f32(x[i]), (uint32_t)i);
                if (key > mine && key < last)
                    mine = key;
            }
            atomicMax(&best, (unsigned long long)mine);
            __syncthreads();
            last = best;
            if (threadIdx.x == 0) {
                const uint32_t i = 0xFFFFFFFFu - (uint32_t)last;
                p.top_index[r * p.top + k] = (int32_t)i;
                p.top_logprob[r * p.top + k] = res.logprob(to_f32(x[i]));
            }
            __syncthreads();
        }
    }
}

template <typename T> __global__ void __launch_bounds__(kLpThreads) logprob_grad_rows_kernel(LogprobGradParams p)
{
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.logits) + r * p.ld;
        T *d = static_cast<T *>(p.dlogits) + r * p.ldd;
        const int64_t tok = p.tokens ? p.tokens[r] : -1;
        const float lse = p.lse[r];
        const float dlp = p.dlogprob && tok >= 0 && tok < (int64_t)p.vocab ? p.dlogprob[r] : 0.f;
        const float dent = p.dentropy ? p.dentropy[r] : 0.f, ent = p.dentropy ? p.entropy[r] : 0.f;
        float m = 0.f, l = lse; // log p = (x - m) scale - l
        if (fabsf(lse) > kLseMost && fabsf(lse) < INFINITY) {
            m = -INFINITY;
            for (uint64_t i = threadIdx.x; i < p.vocab; i += kLpThreads)
                m = fmaxf(m, to_f32(x[i]));
            m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); });
            l = 0.f;
            for (uint64_t i = threadIdx.x; i < p.vocab; i += kLpThreads)
                l += expf((to_f32(x[i]) - m) * p.scale);
            l = logf(block_reduce(l, [](float a, float b) { return a + b; }));
        }
        for (uint64_t i = threadIdx.x; i < p.vocab; i += kLpThreads) {
            float v = 0.f;
            if (lse != -INFINITY) {
                const float logp = (to_f32(x[i]) - m) * p.scale - l, q = expf(logp);
                const float tail = q != 0.f ? q * (logp + ent) : 0.f;
                v = -q * dlp - dent * tail;
                if ((int64_t)i == tok) { // 1 - q and the two terms may cancel: the row's one value in 64 bits
                    d[i] = from_f32<T>((float)(((double)dlp * (1.0 - q) - (double)dent * tail) * p.scale));
                    continue;
                }
            }
            d[i] = from_f32<T>(v * p.scale);
        }
    }
}

namespace {
unsigned row_grid(uint64_t rows) { return (unsigned)std::min<uint64_t>(rows, 1u << 20); }
} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

ecc_status ecc_token_logprob(const void *logits, uint64_t ld, uint32_t type, const int64_t *tokens, uint64_t rows,
                             uint64_t vocab, float scale, uint32_t top, float *logprob, float *entropy, float *lse,
                             float *top_logprob, int32_t *top_index, void *stream)
{
    if (!wide_type(type) || !vocab || vocab >= (1ull << 31) || !(scale > 0.f) || !std::isfinite(scale) ||
        top > ECC_MAX_TOP || top > vocab)
        return ECC_ERR_ARG;
    if (!rows)
        return ECC_OK;
    if (!logits || ld < vocab || !aligned_to(logits, type) || (top && (!top_logprob || !top_index)) ||
        ((uintptr_t)tokens & 7) || !aligned_to(logprob, ECC_F32) || !aligned_to(entropy, ECC_F32) ||
        !aligned_to(lse, ECC_F32) || !aligned_to(top_logprob, ECC_F32) || !aligned_to(top_index, ECC_F32))
        return ECC_ERR_ARG;
    LogprobParams p{logits, tokens, ld, rows, vocab, scale, top, logprob, entropy, lse, top_logprob, top_index};
    cudaStream_t st = (cudaStream_t)stream;
    if (type == ECC_F32)
        logprob_rows_kernel<float><<<row_grid(rows), kLpThreads, 0, st>>>(p);
    else if (type == ECC_BF16)
        logprob_rows_kernel<bf16><<<row_grid(rows), kLpThreads, 0, st>>>(p);
    else
        logprob_rows_kernel<__half><<<row_grid(rows), kLpThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

ecc_status ecc_token_logprob_grad(const void *logits, uint64_t ld, uint32_t type, const int64_t *tokens,
                                  uint64_t rows, uint64_t vocab, float scale, const float *lse,
                                  const float *entropy, const float *dlogprob, const float *dentropy, void *dlogits,
                                  uint64_t ldd, void *stream)
{
    if (!wide_type(type) || !vocab || vocab >= (1ull << 31) || !(scale > 0.f) || !std::isfinite(scale))
        return ECC_ERR_ARG;
    if (!rows)
        return ECC_OK;
    if (!logits || !dlogits || !lse || ld < vocab || ldd < vocab || (dlogprob && !tokens) ||
        (dentropy && !entropy) || !aligned_to(logits, type) || !aligned_to(dlogits, type) ||
        ((uintptr_t)tokens & 7) || !aligned_to(lse, ECC_F32) || !aligned_to(entropy, ECC_F32) ||
        !aligned_to(dlogprob, ECC_F32) || !aligned_to(dentropy, ECC_F32) || (logits == dlogits && ld != ldd))
        return ECC_ERR_ARG;
    LogprobGradParams p{logits, tokens, ld, ldd, rows, vocab, scale, lse, entropy, dlogprob, dentropy, dlogits};
    cudaStream_t st = (cudaStream_t)stream;
    if (type == ECC_F32)
        logprob_grad_rows_kernel<float><<<row_grid(rows), kLpThreads, 0, st>>>(p);
    else if (type == ECC_BF16)
        logprob_grad_rows_kernel<bf16><<<row_grid(rows), kLpThreads, 0, st>>>(p);
    else
        logprob_grad_rows_kernel<__half><<<row_grid(rows), kLpThreads, 0, st>>>(p);
    return launch_status(cudaGetLastError());
}

} // extern "C"
