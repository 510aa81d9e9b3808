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
#include "ecc_tensor.cuh"

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

// ---------------------------------------------------------------- rows in vectors
// A row of logits as `head` single values, `vecs` 16-byte aligned vectors and
// `tail` single values.
template <typename T> struct RowView {
    static constexpr uint32_t V = 16 / sizeof(T);
    const T *x;
    uint32_t head, tail;
    uint64_t vecs;
    __device__ __forceinline__ RowView(const T *row, uint64_t n) : x(row)
    {
        const uint64_t h = ((16 - ((uintptr_t)row & 15)) & 15) / sizeof(T);
        head = (uint32_t)min(h, n);
        vecs = (n - head) / V;
        tail = (uint32_t)((n - head) % V);
    }
    __device__ __forceinline__ const uint4 *vec(uint64_t i) const { return reinterpret_cast<const uint4 *>(x + head) + i; }
    // the k-th of the head and tail values (k < head + tail): its index
    __device__ __forceinline__ uint64_t single(uint32_t k) const { return k < head ? k : vecs * V + k; }
};

template <typename T> __device__ __forceinline__ void unpack(const uint4 &v, float *f);
template <> __device__ __forceinline__ void unpack<float>(const uint4 &v, float *f)
{
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
template <> __device__ __forceinline__ void unpack<bf16>(const uint4 &v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <> __device__ __forceinline__ void unpack<__half>(const uint4 &v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = g.x;
        f[2 * i + 1] = g.y;
    }
}

__device__ __forceinline__ float max_nan(float a, float b) // NaN if either is
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Running maximum m of the logits x, s = sum 2^d and t = sum 2^d d with
// d = (x - m) c, c = scale * log2(e).  d is cut at -200 (2^-200 is 0 in
// float32), so that -infinity adds nothing; a NaN shows in m alone.
struct Softmax {
    float m = -INFINITY, s = 0.f, t = 0.f;
    __device__ __forceinline__ void raise(float to, float c) // to a larger (or NaN) maximum
    {
        const float d = fmaxf((m - to) * c, -200.f), f = exp2_fast(d);
        t = f * fmaf(s, d, t);
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void add(float x, float c)
    {
        const float d = fmaxf((x - m) * c, -200.f), e = exp2_fast(d);
        s += e;
        t = fmaf(e, d, t);
    }
    __device__ __forceinline__ void join(float om, float os, float ot, float c)
    {
        Softmax o;
        o.m = om;
        o.s = os;
        o.t = ot;
        const float to = max_nan(m, om);
        if (m != to)
            raise(to, c);
        if (om != to)
            o.raise(to, c);
        s += o.s;
        t += o.t;
    }
};

constexpr int kLpWarps = kLpThreads / 32;
constexpr uint32_t kUnroll = 4;    // vectors a thread loads at a time: a group
constexpr uint32_t kGroupMax = 16; // group maxima kept for each thread
constexpr uint32_t kCandidates = 1024;

struct LogprobShared {
    float gmax[kGroupMax][kLpThreads]; // largest logit of the groups of a slot
    unsigned long long key[kCandidates];
    uint32_t pair[kLpThreads * kGroupMax];
    unsigned long long best[ECC_MAX_TOP]; // the CTA's alternatives, in order
    unsigned long long largest;
    float m[kLpWarps], s[kLpWarps], t[kLpWarps];
    uint32_t low[kLpWarps];
    float cta[3];
    uint32_t n_key, n_pair;
};

// The `top` largest keys of key[0, n) in order (a key's rank is the number
// of larger ones; keys differ); missing ones are 0.
__device__ __forceinline__ void rank_keys(LogprobShared &sh, uint32_t n, uint32_t top)
{
    for (uint32_t i = threadIdx.x; i < n; i += kLpThreads) {
        const unsigned long long k = sh.key[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; ++j)
            rank += sh.key[j] > k;
        if (rank < top)
            sh.best[rank] = k;
    }
    for (uint32_t i = n + threadIdx.x; i < top; i += kLpThreads)
        sh.best[i] = 0;
}

// A row by a cluster of `split` CTAs, each a share of its vectors (the first
// also the single values at the ends): one pass over the row that keeps the
// softmax sums, and for the alternatives the largest logit of each group of
// vectors.  At least `top` threads' largest logits reach the bound
// min over warps (r-th largest of the warp's threads), r = top / warps, so
// every alternative does; only the groups that reach it are read again (a few
// dozen, a lane a value, from L2), and the values that do are ranked.  Bound
// by HBM: one read of the logits.
template <typename T> __global__ void __launch_bounds__(kLpThreads, 4) logprob_kernel(LogprobParams p, uint32_t split)
{
    extern __shared__ __align__(16) uint8_t raw[];
    LogprobShared &sh = *reinterpret_cast<LogprobShared *>(raw);
    constexpr uint32_t V = RowView<T>::V;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = split > 1 ? cluster_rank() : 0;
    const uint64_t r = blockIdx.x / split;
    const T *x = static_cast<const T *>(p.logits) + r * p.ld;
    const RowView<T> row(x, p.vocab);
    const uint64_t v0 = row.vecs * rank / split, v1 = row.vecs * (rank + 1) / split;
    const uint32_t singles = rank == 0 ? row.head + row.tail : 0;
    const float c = p.scale * 1.44269504f;
    const int64_t tok = p.tokens && tid == 0 && rank == 0 ? p.tokens[r] : -1;
    const float xtok = tok >= 0 && tok < (int64_t)p.vocab ? to_f32(x[tok]) : 0.f;

    const uint64_t groups = (v1 - v0 + kUnroll * kLpThreads - 1) / (kUnroll * kLpThreads);
    const uint32_t per_slot = (uint32_t)((groups + kGroupMax - 1) / kGroupMax);
    Softmax sm;
    float own = -INFINITY, slot_max = -INFINITY; // largest logit of this thread's vectors, of the slot's
    uint32_t slot = 0, in_slot = 0;
    for (uint64_t g = 0; g < groups; ++g) {
        const uint64_t i0 = v0 + g * kUnroll * kLpThreads + tid;
        uint4 q[kUnroll];
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u)
            if (i0 + u * kLpThreads < v1)
                q[u] = ld_stream16(row.vec(i0 + u * kLpThreads));
        float f[kUnroll][V], big = -INFINITY;
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u) {
            if (i0 + u * kLpThreads < v1) {
                unpack<T>(q[u], f[u]);
            } else {
#pragma unroll
                for (uint32_t k = 0; k < V; ++k)
                    f[u][k] = -INFINITY;
            }
#pragma unroll
            for (uint32_t k = 0; k < V; ++k)
                big = max_nan(big, f[u][k]);
        }
        if (!(big <= sm.m))
            sm.raise(max_nan(sm.m, big), c);
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u)
#pragma unroll
            for (uint32_t k = 0; k < V; ++k)
                sm.add(f[u][k], c);
        if (p.top) {
            slot_max = max_nan(slot_max, big);
            if (++in_slot == per_slot || g + 1 == groups) {
                sh.gmax[slot][tid] = slot_max;
                own = max_nan(own, slot_max);
                slot_max = -INFINITY;
                ++slot;
                in_slot = 0;
            }
        }
    }
    for (uint32_t k = tid; k < singles; k += kLpThreads) {
        const float v = to_f32(x[row.single(k)]);
        if (!(v <= sm.m))
            sm.raise(max_nan(sm.m, v), c);
        sm.add(v, c);
    }
    // join lanes, warps (thread 0)
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sm.join(__shfl_xor_sync(~0u, sm.m, o), __shfl_xor_sync(~0u, sm.s, o), __shfl_xor_sync(~0u, sm.t, o), c);
    if (lane == 0) {
        sh.m[warp] = sm.m;
        sh.s[warp] = sm.s;
        sh.t[warp] = sm.t;
    }
    if (p.top) {
        // warps whose threads all have a vector; with none, every finite value is ranked
        const uint32_t full = (uint32_t)min((uint64_t)kLpWarps, (v1 - v0) / 32);
        const uint32_t take = full ? (p.top + full - 1) / full : 0;
        uint32_t mine = order_bits(own), low = 0;
        for (uint32_t i = 0; i < min(take, 32u); ++i) {
            low = __reduce_max_sync(~0u, mine);
            const uint32_t at = __ffs(__ballot_sync(~0u, mine == low)) - 1;
            if (lane == at)
                mine = 0;
        }
        if (lane == 0)
            sh.low[warp] = low;
        if (tid == 0)
            sh.n_key = sh.n_pair = 0;
        __syncthreads();
        uint32_t bound = order_bits(-INFINITY) + 1; // -infinity is no candidate
        if (full) {
            uint32_t b = 0xFFFFFFFFu;
            for (uint32_t w = 0; w < full; ++w)
                b = min(b, sh.low[w]);
            bound = max(bound, b);
        }
        for (uint32_t k = 0; k < slot; ++k)
            if (order_bits(sh.gmax[k][tid]) >= bound)
                sh.pair[atomicAdd(&sh.n_pair, 1u)] = k << 16 | tid;
        for (uint32_t k = tid; k < singles; k += kLpThreads) {
            const uint64_t i = row.single(k);
            const float v = to_f32(x[i]);
            if (order_bits(v) >= bound)
                sh.key[atomicAdd(&sh.n_key, 1u)] = order_key(v, (uint32_t)i); // at most 14
        }
        __syncthreads();
        const uint32_t pairs = sh.n_pair;
        for (uint32_t i = warp; i < pairs; i += kLpWarps) {
            const uint32_t k = sh.pair[i] >> 16, t = sh.pair[i] & 0xFFFFu;
            const uint64_t g0 = (uint64_t)k * per_slot, g1 = min(groups, g0 + per_slot);
            for (uint64_t e = lane; e < (g1 - g0) * kUnroll * V; e += 32) {
                const uint64_t v = v0 + (g0 * kUnroll + e / V) * kLpThreads + t;
                if (v < v1) {
                    const uint64_t at = row.head + v * V + e % V;
                    const float f = to_f32(x[at]);
                    if (order_bits(f) >= bound) {
                        const uint32_t n = atomicAdd(&sh.n_key, 1u);
                        if (n < kCandidates)
                            sh.key[n] = order_key(f, (uint32_t)at);
                    }
                }
            }
        }
        __syncthreads();
        const uint32_t n = sh.n_key;
        if (n <= kCandidates) {
            rank_keys(sh, n, p.top);
            __syncthreads();
            if (n < p.top && warp == 0) { // fewer values than asked for: tokens without probability, lowest index first
                uint32_t have = n;
                // this CTA's values in index order: heads, vectors, tails
                const uint64_t first = rank == 0 ? 0 : row.head + v0 * V;
                const uint64_t last = row.head + v1 * V;
                for (uint64_t i0 = first; have < p.top; i0 += 32) {
                    // the vectors' range, then (first CTA) the tail
                    uint64_t i = i0 + lane;
                    bool in = i < last;
                    if (!in && rank == 0) {
                        i = row.head + row.vecs * V + (i - last);
                        in = i < p.vocab;
                    }
                    const bool hit = in && order_bits(to_f32(x[in ? i : 0])) < bound;
                    const uint32_t hits = __ballot_sync(~0u, hit), at = have + __popc(hits & ((1u << lane) - 1));
                    if (hit && at < p.top)
                        sh.best[at] = order_key(-INFINITY, (uint32_t)i);
                    have += __popc(hits);
                    if (!__any_sync(~0u, in))
                        break;
                }
            }
        } else { // many equal values: one alternative a pass, the largest key below the last one
            unsigned long long before = ~0ull;
            for (uint32_t k = 0; k < p.top; ++k) {
                if (tid == 0)
                    sh.largest = 0;
                __syncthreads();
                unsigned long long big = 0;
                auto look = [&](uint64_t i) {
                    const unsigned long long key = order_key(to_f32(x[i]), (uint32_t)i);
                    if (key < before && key > big)
                        big = key;
                };
                for (uint64_t i = row.head + v0 * V + tid; i < row.head + v1 * V; i += kLpThreads)
                    look(i);
                for (uint32_t i = tid; i < singles; i += kLpThreads)
                    look(row.single(i));
                atomicMax(&sh.largest, big);
                __syncthreads();
                before = sh.largest;
                if (tid == 0)
                    sh.best[k] = before;
                __syncthreads();
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        sm.m = sh.m[0];
        sm.s = sh.s[0];
        sm.t = sh.t[0];
        for (int w = 1; w < kLpWarps; ++w)
            sm.join(sh.m[w], sh.s[w], sh.t[w], c);
        sh.cta[0] = sm.m;
        sh.cta[1] = sm.s;
        sh.cta[2] = sm.t;
    }
    __syncthreads();
    if (split > 1) {
        cluster_sync();
        if (rank == 0) {
            if (tid == 0) {
                for (uint32_t q = 1; q < split; ++q) {
                    const uint32_t a = cluster_addr(smem_u32(sh.cta), q);
                    sm.join(cluster_load(a), cluster_load(a + 4), cluster_load(a + 8), c);
                }
                sh.cta[0] = sm.m;
                sh.cta[1] = sm.s;
                sh.cta[2] = sm.t;
            }
            const uint32_t n = split * p.top; // at most 256 keys; those of short shares are 0
            if (tid == 0)
                sh.n_key = 0;
            __syncthreads();
            for (uint32_t i = tid; i < n; i += kLpThreads) {
                const uint32_t q = i / p.top, a = cluster_addr(smem_u32(sh.best + i % p.top), q);
                const uint32_t lo = __float_as_uint(cluster_load(a)), hi = __float_as_uint(cluster_load(a + 4));
                if (hi)
                    sh.key[atomicAdd(&sh.n_key, 1u)] = (unsigned long long)hi << 32 | lo;
            }
            __syncthreads();
            if (p.top)
                rank_keys(sh, sh.n_key, p.top);
            __syncthreads();
        }
        __syncwarp();
        cluster_sync(); // the first CTA has read the others' results
        if (rank)
            return;
    }
    // t and log2 s are in units of log2(e)
    const RowResult res(sh.cta[0], sh.cta[1], sh.cta[2] * 0.69314718f, p.scale);
    if (tid == 0) {
        if (p.lse)
            p.lse[r] = res.lse;
        if (p.entropy)
            p.entropy[r] = res.entropy;
        if (p.logprob && p.tokens)
            p.logprob[r] = tok < 0 ? 0.f : tok >= (int64_t)p.vocab ? NAN : res.logprob(xtok);
    }
    if (tid < p.top) {
        const unsigned long long k = sh.best[tid];
        const uint32_t bits = (uint32_t)(k >> 32);
        const float v = bits == 0xFFFFFFFFu ? NAN : __uint_as_float(bits & 0x80000000u ? bits & 0x7FFFFFFFu : ~bits);
        p.top_index[r * p.top + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)k);
        p.top_logprob[r * p.top + tid] = res.logprob(v);
    }
}

// ---------------------------------------------------------------- gradient
// With g = log2 p = (x - m) c - l (m = 0 and l = lse log2(e), unless lse is
// too large for that): the gradient is 2^g (A + B g), A = -scale (dlogprob +
// dentropy H), B = -scale dentropy ln 2, and the token's own value in 64
// bits, where dlogprob (1 - p) and the other term may cancel.  g is cut at
// -200, where 2^g is 0.  Bound by HBM: the logits read, the gradient written.
// a vector that this thread may write over later (so not through the read-only path)
__device__ __forceinline__ uint4 load_once(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

struct GradRow {
    float m, c, l, A, B, dlp, dent, ent, scale;
    int64_t tok;
    __device__ __forceinline__ float value(float x) const
    {
        const float g = fmaxf(fmaf(x - m, c, -l), -200.f);
        return exp2_fast(g) * fmaf(B, g, A);
    }
    __device__ __forceinline__ float token_value(float x) const
    {
        const float g = fmaxf(fmaf(x - m, c, -l), -200.f);
        const double q = exp2_fast(g), tail = q * ((double)g * 0.6931471805599453 + ent);
        return (float)(((double)dlp * (1.0 - q) - (double)dent * tail) * scale);
    }
};

template <typename Op> __device__ __forceinline__ float block_reduce(float v, Op op)
{
    __shared__ float part[kLpWarps];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = op(v, __shfl_xor_sync(~0u, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < kLpWarps; ++i)
        v = op(v, part[i]);
    return v;
}

template <typename T> __device__ __forceinline__ uint4 pack(const float *f);
template <> __device__ __forceinline__ uint4 pack<float>(const float *f)
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 pack<bf16>(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 pack<__half>(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row by a cluster of `split` CTAs, each a share of it.
template <typename T> __global__ void __launch_bounds__(kLpThreads) logprob_grad_kernel(LogprobGradParams p, uint32_t split)
{
    constexpr uint32_t V = RowView<T>::V;
    const uint32_t tid = threadIdx.x, part = blockIdx.x % split;
    const uint64_t r = blockIdx.x / split;
    const T *x = static_cast<const T *>(p.logits) + r * p.ld;
    T *d = static_cast<T *>(p.dlogits) + r * p.ldd;
    GradRow row;
    const float lse = p.lse[r];
    row.tok = p.tokens ? p.tokens[r] : -1;
    if (row.tok >= (int64_t)p.vocab || !p.dlogprob)
        row.tok = -1;
    row.dlp = row.tok >= 0 ? p.dlogprob[r] : 0.f;
    row.dent = p.dentropy ? p.dentropy[r] : 0.f;
    row.ent = p.dentropy ? p.entropy[r] : 0.f;
    row.scale = p.scale;
    row.c = p.scale * 1.44269504f;
    row.m = 0.f;
    row.l = lse * 1.44269504f;
    if (fabsf(lse) > kLseMost && fabsf(lse) < INFINITY) {
        float m = -INFINITY, s = 0.f;
        for (uint64_t i = tid; i < p.vocab; i += kLpThreads)
            m = fmaxf(m, to_f32(x[i]));
        row.m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); });
        for (uint64_t i = tid; i < p.vocab; i += kLpThreads)
            s += exp2_fast(fmaxf((to_f32(x[i]) - row.m) * row.c, -200.f));
        row.l = log2f(block_reduce(s, [](float a, float b) { return a + b; }));
        if (split > 1) { // the row's other CTAs may write over what they read here (dlogits = logits)
            __syncwarp();
            cluster_sync();
        }
    }
    row.A = -p.scale * fmaf(row.dent, row.ent, row.dlp);
    row.B = -p.scale * row.dent * 0.69314718f;
    if (lse == -INFINITY) { // no token has a probability
        row.A = row.B = row.m = row.l = 0.f;
        row.tok = -1;
    } else if (!(lse < INFINITY)) {
        row.A = NAN;
    }
    const RowView<T> view(x, p.vocab);
    if ((((uintptr_t)x ^ (uintptr_t)d) & 15) == 0) { // both rows' vectors start at the same value
        const uint64_t v0 = view.vecs * part / split, v1 = view.vecs * (part + 1) / split;
        uint4 *out = reinterpret_cast<uint4 *>(d + view.head);
        for (uint64_t i0 = v0 + tid; i0 < v1; i0 += kUnroll * kLpThreads) {
            uint4 q[kUnroll];
#pragma unroll
            for (uint32_t u = 0; u < kUnroll; ++u)
                if (i0 + u * kLpThreads < v1)
                    q[u] = load_once(view.vec(i0 + u * kLpThreads));
#pragma unroll
            for (uint32_t u = 0; u < kUnroll; ++u) {
                const uint64_t i = i0 + u * kLpThreads;
                if (i < v1) {
                    float f[V];
                    unpack<T>(q[u], f);
                    const uint64_t at = (uint64_t)row.tok - (view.head + i * V);
#pragma unroll
                    for (uint32_t k = 0; k < V; ++k)
                        f[k] = at == k ? row.token_value(f[k]) : row.value(f[k]);
                    st_stream16(out + i, pack<T>(f));
                }
            }
        }
        if (part == 0)
            for (uint32_t k = tid; k < view.head + view.tail; k += kLpThreads) {
                const uint64_t i = view.single(k);
                const float f = to_f32(x[i]);
                d[i] = from_f32<T>((uint64_t)row.tok == i ? row.token_value(f) : row.value(f));
            }
    } else { // a value a thread
        const uint64_t e0 = p.vocab * part / split, e1 = p.vocab * (part + 1) / split;
        for (uint64_t i0 = e0 + tid; i0 < e1; i0 += 8 * kLpThreads) {
            T q[8];
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u)
                if (i0 + u * kLpThreads < e1)
                    q[u] = x[i0 + u * kLpThreads];
#pragma unroll
            for (uint32_t u = 0; u < 8; ++u) {
                const uint64_t i = i0 + u * kLpThreads;
                if (i < e1) {
                    const float f = to_f32(q[u]);
                    d[i] = from_f32<T>((uint64_t)row.tok == i ? row.token_value(f) : row.value(f));
                }
            }
        }
    }
}

namespace {

// CTAs a row, in powers of two: enough for `ctas` in all while a CTA keeps at
// least `least` values
uint32_t row_split(uint64_t rows, uint64_t vocab, uint64_t ctas, uint64_t least)
{
    uint32_t s = 1;
    while (s < 8 && rows * s < ctas && vocab / (2 * s) >= least)
        s *= 2;
    return s;
}

cudaLaunchConfig_t row_config(uint64_t rows, uint32_t split, size_t smem, cudaLaunchAttribute *at, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * split));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = split;
    at->val.clusterDim.y = at->val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cfg;
}

template <typename T> ecc_status logprob_launch(const LogprobParams &p, cudaStream_t st)
{
    const int sms = sm_count();
    const size_t smem = sizeof(LogprobShared);
    if (sms <= 0 || occupancy((const void *)logprob_kernel<T>, kLpThreads, smem) <= 0)
        return ECC_ERR_CUDA;
    const uint32_t split = row_split(p.rows, p.vocab, 2ull * sms, 2048);
    if (p.rows >= (1ull << 31) / split)
        return ECC_ERR_ARG;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = row_config(p.rows, split, smem, &at, st);
    return launch_status(cudaLaunchKernelEx(&cfg, logprob_kernel<T>, p, split));
}

template <typename T> ecc_status logprob_grad_launch(const LogprobGradParams &p, cudaStream_t st)
{
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    const uint32_t split = row_split(p.rows, p.vocab, 8ull * sms, 4096);
    if (p.rows >= (1ull << 31) / split)
        return ECC_ERR_ARG;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = row_config(p.rows, split, 0, &at, st);
    return launch_status(cudaLaunchKernelEx(&cfg, logprob_grad_kernel<T>, p, split));
}

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" {

ecc_status ecc_token_logprob(const void *logits, uint64_t ld, uint32_t type, const int64_t *tokens, uint64_t rows,
                             uint64_t vocab, float scale, uint32_t top, float *logprob, float *entropy, float *lse,
                             float *top_logprob, int32_t *top_index, void *stream)
{
    if (!wide_type(type) || !vocab || vocab >= (1ull << 31) || !(scale > 0.f) || !std::isfinite(scale * 2.f) ||
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
    return type == ECC_F32    ? logprob_launch<float>(p, st)
           : type == ECC_BF16 ? logprob_launch<bf16>(p, st)
                              : logprob_launch<__half>(p, st);
}

ecc_status ecc_token_logprob_grad(const void *logits, uint64_t ld, uint32_t type, const int64_t *tokens,
                                  uint64_t rows, uint64_t vocab, float scale, const float *lse,
                                  const float *entropy, const float *dlogprob, const float *dentropy, void *dlogits,
                                  uint64_t ldd, void *stream)
{
    if (!wide_type(type) || !vocab || vocab >= (1ull << 31) || !(scale > 0.f) || !std::isfinite(scale * 2.f))
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
    return type == ECC_F32    ? logprob_grad_launch<float>(p, st)
           : type == ECC_BF16 ? logprob_grad_launch<bf16>(p, st)
                              : logprob_grad_launch<__half>(p, st);
}

} // extern "C"
