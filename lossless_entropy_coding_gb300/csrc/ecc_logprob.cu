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
        if (m == -INFINITY) { // no token has a probability
            lse = -INFINITY;
            entropy = 0.f;
        } else if (m == INFINITY) {
            lse = INFINITY;
            entropy = NAN;
        } else {
            lse = m * scale + logs; // (infinite where m * scale leaves float32; the rest does without it)
            entropy = logs - t / s;
        }
    }
    __device__ __forceinline__ float logprob(float x) const
    {
        return m == -INFINITY ? -INFINITY : m == INFINITY ? x - m : (x - m) * scale - logs;
    }
};

// log p in the gradient: from lse, unless lse is so large that rounding it
// to float32 (2^-24 |lse|) would show; the row's maximum and log sum are then
// found again.  So they are where lse is infinite and a scale above 1 may
// have made it so (a row of the type's lowest value).
constexpr float kLseMost = 256.f;

// ---------------------------------------------------------------- rows in vectors
// A row of logits as `head` single values, `vecs` 16-byte aligned vectors and
// `tail` single values (fewer than 2^31 values in all).
template <typename T> struct RowView {
    static constexpr uint32_t V = 16 / sizeof(T); // values of a vector
    static constexpr uint32_t U = 32 / V;         // vectors of a group: a thread takes 32 values at a time
    const T *x;
    uint32_t head, tail, vecs;
    __device__ __forceinline__ RowView(const T *row, uint64_t n) : x(row)
    {
        head = min((16u - ((uint32_t)(uintptr_t)row & 15u) & 15u) / (uint32_t)sizeof(T), (uint32_t)n);
        vecs = ((uint32_t)n - head) / V;
        tail = ((uint32_t)n - head) % V;
    }
    __device__ __forceinline__ const uint4 *vec(uint32_t i) const { return reinterpret_cast<const uint4 *>(x + head) + i; }
    // the k-th of the head and tail values (k < head + tail): its index
    __device__ __forceinline__ uint32_t single(uint32_t k) const { return k < head ? k : vecs * V + k; }
};

__device__ __forceinline__ float max_nan(float a, float b) // NaN if either is
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
constexpr uint32_t kSlots = 16;    // slot maxima kept for each column of a block, and of a warp
constexpr uint32_t kWarpSlots = 8;
constexpr int kSelThreads = 128;   // selecting threads of a block
constexpr uint32_t kStages = 4;    // stages of a block's ring
constexpr uint32_t kStageVecs = 4 * kLpThreads;
constexpr uint32_t kStageBytes = kStageVecs * 16;

// A team of N threads (a warp, or a block's four selecting warps) finds a row's
// alternatives from the group maxima of C columns of vectors: column t holds
// the vectors t, t + C, ... of the team's share.
template <int N, int C> struct Team {
    static constexpr uint32_t threads = N, columns = C, keys = N == 32 ? 256 : 512; // keys: candidates that are ranked
    unsigned long long key[keys];
    unsigned long long best[ECC_MAX_TOP]; // the alternatives, in order
    uint16_t pair[C * (N == 32 ? kWarpSlots : kSlots)]; // slot << 8 | column
    uint32_t low[N / 32];
    float sum[3];
    uint16_t kept[N == 32 ? 1 : keys];
    uint32_t n_key, n_pair, n_kept, hit[2];

    static __device__ __forceinline__ void sync()
    {
        __syncwarp();
        if constexpr (N > 32) // (the form that allows a warp to arrive in parts)
            asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
    }
    static __device__ __forceinline__ uint32_t thread() { return threadIdx.x % N; }
};
using WarpTeam = Team<32, 32>;
using BlockTeam = Team<kSelThreads, kLpThreads>;

// The `top` largest of key[0, n) in order (a key's rank is the number of
// larger ones; keys differ), four threads a key; missing ones are 0.
template <typename Tm> __device__ __forceinline__ void rank_keys(Tm &sh, uint32_t n, uint32_t top)
{
    const uint32_t tid = Tm::thread(), q = tid & 3;
    for (uint32_t i0 = 0; i0 < n; i0 += Tm::threads / 4) {
        const uint32_t i = i0 + tid / 4;
        const unsigned long long k = i < n ? sh.key[i] : ~0ull;
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t j = q; j < n; j += 4)
            rank += sh.key[j] > k;
        rank += __shfl_xor_sync(~0u, rank, 1);
        rank += __shfl_xor_sync(~0u, rank, 2);
        if (q == 0 && i < n && rank < top)
            sh.best[rank] = k;
    }
    for (uint32_t i = n + tid; i < top; i += Tm::threads)
        sh.best[i] = 0;
}

// A team's share of a row: vectors [v0, v1), and the single values at the
// row's ends for the first share.
template <typename T> struct Share {
    RowView<T> row;
    uint32_t v0, v1, n, singles;
};

// A group of a thread's values, `big` the largest, into the softmax.  Without the cut
// of Softmax::add, two values at a time; where that meets 0 * infinity (a
// masked value), again with the cut.
template <int P> __device__ __forceinline__ float largest_of(const float2 *f)
{
    float big = max_nan(f[0].x, f[0].y), more = -INFINITY;
#pragma unroll
    for (int i = 1; i < P; ++i)
        (i & 1 ? more : big) = max_nan(i & 1 ? more : big, f[i].x, f[i].y);
    return max_nan(big, more);
}
template <int P> __device__ __forceinline__ void add_group(Softmax &sm, const float2 (&f)[P], float big, float c)
{
    if (!(big <= sm.m))
        sm.raise(max_nan(sm.m, big), c);
    const float2 minus = both(sm.m == -INFINITY ? 0.f : -sm.m), c2 = both(c);
    float2 s0 = both(0.f), s1 = s0, t0 = s0, t1 = s0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 d = mul2(add2(f[i], minus), c2), e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
        if (i & 1) {
            s1 = add2(s1, e);
            t1 = fma2(e, d, t1);
        } else {
            s0 = add2(s0, e);
            t0 = fma2(e, d, t0);
        }
    }
    s0 = add2(s0, s1);
    t0 = add2(t0, t1);
    const float t = t0.x + t0.y;
    if (t == t) {
        sm.s += s0.x + s0.y;
        sm.t += t;
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            sm.add(f[i].x, c);
            sm.add(f[i].y, c);
        }
    }
}

// The share's alternatives -> sh.best.  gmax[k][t] is the largest logit of
// slot k of column t: its vectors [k << shift, (k + 1) << shift).  A bound
// that at least `top` slots reach is a bound that every alternative reaches;
// only the slots that reach it are read again (a few dozen, a lane a value,
// from L2), and the values that do are ranked.  For a warp the bound is the
// top-th largest slot, to 24 bits, found bit by bit; for a block first the
// minimum over its warps of the r-th largest of the lanes' columns, r = top /
// warps, then the top-th largest of the slots that reach it (two or three
// times `top`: reading all those again took longer than a row's softmax).
// `single` is the value of the row's ends that this thread holds.
template <typename T, typename Tm>
__device__ __forceinline__ void select_top(Tm &sh, const float (*gmax)[Tm::columns], const Share<T> &a, uint32_t top,
                                           uint32_t slots, uint32_t shift, bool has_single, float single,
                                           uint32_t single_at)
{
    constexpr uint32_t V = RowView<T>::V, N = Tm::threads, C = Tm::columns;
    const uint32_t tid = Tm::thread(), lane = tid & 31, warp = tid >> 5;
    const T *x = a.row.x;
    uint32_t bound = order_bits(-INFINITY) + 1; // -infinity is no candidate
    if (tid == 0)
        sh.n_key = sh.n_pair = sh.n_kept = 0;
    if constexpr (N == 32) {
        uint32_t key[kWarpSlots], low = 0;
#pragma unroll
        for (uint32_t k = 0; k < kWarpSlots; ++k)
            key[k] = k < slots ? order_bits(gmax[k][lane]) : 0;
        for (uint32_t bit = 0x80000000u; bit >= 0x100u; bit >>= 1) {
            uint32_t n = 0;
#pragma unroll
            for (uint32_t k = 0; k < kWarpSlots; ++k)
                n += key[k] >= (low | bit);
            if (__reduce_add_sync(~0u, n) >= top)
                low |= bit;
        }
        bound = max(bound, low);
        Tm::sync();
    } else {
        float own = -INFINITY;
#pragma unroll 2
        for (uint32_t k = 0; k < slots; ++k)
#pragma unroll
            for (uint32_t t = 0; t < C; t += N)
                own = max_nan(own, gmax[k][t + tid]);
        // warps whose lanes all have a vector; with none, every value above -infinity is a candidate
        const uint32_t full = min(N / 32, (a.v1 - a.v0) / 32), take = full ? (top + full - 1) / full : 0;
        uint32_t mine = order_bits(own), low = 0;
#pragma unroll 1
        for (uint32_t i = 0; i < take; ++i) {
            low = __reduce_max_sync(~0u, mine);
            if (lane == __ffs(__ballot_sync(~0u, mine == low)) - 1)
                mine = 0;
        }
        if (lane == 0)
            sh.low[warp] = low;
        Tm::sync();
        if (full) {
            uint32_t b = 0xFFFFFFFFu;
            for (uint32_t w = 0; w < full; ++w)
                b = min(b, sh.low[w]);
            bound = max(bound, b);
        }
    }
#pragma unroll 1
    for (uint32_t k = 0; k < slots; ++k)
#pragma unroll 1
        for (uint32_t t = 0; t < C; t += N) {
            const uint32_t bits = order_bits(gmax[k][t + tid]);
            if (bits >= bound) {
                const uint32_t n = atomicAdd(&sh.n_pair, 1u);
                sh.pair[n] = (uint16_t)(k << 8 | (t + tid));
                if (n < Tm::keys)
                    sh.key[n] = (unsigned long long)bits << 32 | n;
            }
        }
    Tm::sync();
    const uint16_t *pair = sh.pair;
    uint32_t pairs = sh.n_pair;
    if constexpr (N > 32) {
        if (pairs > top && pairs <= Tm::keys) {
            rank_keys(sh, pairs, top);
            Tm::sync();
            bound = (uint32_t)(sh.best[top - 1] >> 32);
            for (uint32_t i = tid; i < pairs; i += N)
                if ((uint32_t)(sh.key[i] >> 32) >= bound)
                    sh.kept[atomicAdd(&sh.n_kept, 1u)] = sh.pair[i];
            Tm::sync();
            pair = sh.kept;
            pairs = sh.n_kept;
        }
    }
    if (has_single && order_bits(single) >= bound)
        sh.key[atomicAdd(&sh.n_key, 1u)] = order_key(single, single_at); // at most 14
    Tm::sync();
    // the slots' values, eight loads a thread at a time
    const uint32_t log_v = sizeof(T) == 4 ? 2 : 3, log_slot = shift + log_v, items = pairs << log_slot;
    for (uint32_t i0 = tid; i0 < items; i0 += 8 * N) {
        if (*(volatile uint32_t *)&sh.n_key > Tm::keys)
            break; // too many (all threads will see it)
        T q[8];
        uint32_t at[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t i = i0 + j * N;
            at[j] = ~0u;
            if (i < items) {
                const uint32_t slot = pair[i >> log_slot], e = i & ((1u << log_slot) - 1);
                const uint32_t v = a.v0 + (((slot >> 8) << shift) + (e >> log_v)) * C + (slot & 0xFFu);
                if (v < a.v1) {
                    at[j] = a.row.head + v * V + (e & (V - 1));
                    q[j] = x[at[j]];
                }
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
            if (at[j] != ~0u) {
                const float f = to_f32(q[j]);
                if (order_bits(f) >= bound) {
                    const uint32_t n = atomicAdd(&sh.n_key, 1u);
                    if (n < Tm::keys)
                        sh.key[n] = order_key(f, at[j]);
                }
            }
    }
    Tm::sync();
    const uint32_t n = sh.n_key;
    const uint32_t first = a.singles ? 0 : a.row.head + a.v0 * V, last = a.row.head + a.v1 * V;
    if (n <= Tm::keys) {
        rank_keys(sh, n, top);
        Tm::sync();
        if (n < top && warp == 0) { // fewer than asked for: tokens without probability, lowest index first
            uint32_t have = n;
            for (uint32_t i0 = first; have < top; i0 += 32) {
                uint32_t i = i0 + lane;
                bool in = i < last;
                if (!in && a.singles) { // behind the vectors: the tail
                    i = a.row.head + a.row.vecs * V + (i - last);
                    in = i < a.n;
                }
                const bool hit = in && order_bits(to_f32(x[in ? i : 0])) < bound;
                const uint32_t hits = __ballot_sync(~0u, hit), at = have + __popc(hits & ((1u << lane) - 1));
                if (hit && at < top)
                    sh.best[at] = order_key(-INFINITY, i);
                have += __popc(hits);
                if (!__any_sync(~0u, in))
                    break;
            }
        }
    } else {
        // More candidates than are ranked at a time, as among many equal values: the share is read again with the best
        // so far in hand.  Where the next candidates might not fit, the best `top` stay, and the last of them is
        // what the rest have to exceed: equal values that follow do not, so a constant row costs little more than
        // reading it again (top 32, a pass for each alternative and now: 4096 x 50021 float32 zeros 10.6 and 0.92 ms,
        // 4096 x 131072 bf16 27.2 and 1.47, 5184 x 1375 f16 0.27 and 0.12).
        constexpr uint32_t U = 4;
        unsigned long long least = (unsigned long long)bound << 32; // keys from here on
        Tm::sync(); // (n is read)
        if (tid == 0)
            sh.n_key = sh.hit[0] = sh.hit[1] = 0;
        Tm::sync();
        uint32_t have = 0;
        auto take = [&](bool in, uint32_t i) { // a value of each thread
            const unsigned long long key = in ? order_key(to_f32(x[i]), i) : 0;
            if (in && key >= least)
                sh.key[atomicAdd(&sh.n_key, 1u)] = key;
            Tm::sync();
            have = sh.n_key;
            if (have > Tm::keys - N) {
                rank_keys(sh, have, top);
                Tm::sync();
                if (tid < top)
                    sh.key[tid] = sh.best[tid];
                if (tid == 0)
                    sh.n_key = top;
                least = sh.best[top - 1];
                have = top;
            }
            Tm::sync();
        };
        take(tid < a.singles, tid < a.singles ? a.row.single(tid) : 0);
        uint32_t chunk = 0; // U vectors a thread; `hit` in turn for the odd and the even ones, set by any thread
#pragma unroll 1
        for (uint32_t v0 = a.v0 + tid; v0 - tid < a.v1; v0 += U * N, ++chunk) {
            uint4 q[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                if (v0 + u * N < a.v1)
                    q[u] = *a.row.vec(v0 + u * N);
            bool hit = false;
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                if (v0 + u * N < a.v1) {
                    float2 f[V / 2];
                    unpack2<T>(q[u], f);
                    const uint32_t i = a.row.head + (v0 + u * N) * V;
#pragma unroll
                    for (uint32_t k = 0; k < V; ++k)
                        hit |= order_key(k & 1 ? f[k / 2].y : f[k / 2].x, i + k) >= least;
                }
            if (hit)
                sh.hit[chunk & 1] = chunk + 1;
            Tm::sync();
            if (*(volatile uint32_t *)&sh.hit[chunk & 1] != chunk + 1)
                continue;
#pragma unroll 1
            for (uint32_t k = 0; k < U * V; ++k) {
                const uint32_t v = v0 + k / V * N;
                take(v < a.v1, a.row.head + v * V + k % V);
            }
        }
        rank_keys(sh, have, top);
    }
    Tm::sync();
}

// a warp's sums, on every lane
__device__ __forceinline__ void join_lanes(Softmax &sm, float c)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sm.join(__shfl_xor_sync(~0u, sm.m, o), __shfl_xor_sync(~0u, sm.s, o), __shfl_xor_sync(~0u, sm.t, o), c);
}

// the row's outputs from sh.sum and sh.best; thread 0 knows the token and its logit
template <typename Tm>
__device__ __forceinline__ void write_row(const LogprobParams &p, const Tm &sh, uint64_t r, int64_t tok, float xtok)
{
    const uint32_t tid = Tm::thread();
    // (t is in units of log2(e))
    const RowResult res(sh.sum[0], sh.sum[1], sh.sum[2] * 0.69314718f, p.scale);
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

// Short rows: a warp a row, four a block, no block barriers.
template <typename T> __global__ void __launch_bounds__(128, 6) logprob_warp_kernel(LogprobParams p)
{
    __shared__ WarpTeam teams[4];
    __shared__ float gmax[4][kWarpSlots][32];
    constexpr uint32_t V = RowView<T>::V, U = RowView<T>::U;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    WarpTeam &sh = teams[warp];
    const uint64_t r = (uint64_t)blockIdx.x * 4 + warp;
    if (r >= p.rows)
        return;
    const T *x = static_cast<const T *>(p.logits) + r * p.ld;
    const RowView<T> row(x, p.vocab);
    const Share<T> a{row, 0, row.vecs, (uint32_t)p.vocab, row.head + row.tail};
    const float c = p.scale * 1.44269504f;
    const int64_t tok = p.tokens ? p.tokens[r] : -1;
    const float xtok = tok >= 0 && tok < (int64_t)p.vocab ? to_f32(x[tok]) : 0.f;
    const bool has_single = lane < a.singles;
    const uint32_t single_at = has_single ? row.single(lane) : 0;
    const float single = has_single ? to_f32(x[single_at]) : -INFINITY;
    const uint32_t groups = (row.vecs + U * 32 - 1) / (U * 32);
    uint32_t shift = 0; // vectors of a slot: a power of two
    while ((kWarpSlots * 32u << shift) < row.vecs)
        ++shift;
    Softmax sm;
    float slot_max = -INFINITY;
    for (uint32_t g = 0; g < groups; ++g) {
        const uint32_t i0 = g * U * 32 + lane;
        uint4 q[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u)
            if (i0 + u * 32 < row.vecs)
                q[u] = ld_stream16(row.vec(i0 + u * 32));
        float2 f[16];
        float big = -INFINITY;
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (i0 + u * 32 < row.vecs) {
                unpack2<T>(q[u], f + u * V / 2);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < V / 2; ++i)
                    f[u * V / 2 + i] = both(-INFINITY);
            }
            const float m = largest_of<V / 2>(f + u * V / 2);
            big = max_nan(big, m);
            slot_max = max_nan(slot_max, m);
            const uint32_t next = g * U + u + 1; // vectors of this lane so far
            if (p.top && ((next & ((1u << shift) - 1)) == 0 || next == groups * U)) {
                const uint32_t k = (next - 1) >> shift;
                if (k < kWarpSlots)
                    gmax[warp][k][lane] = slot_max;
                slot_max = -INFINITY;
            }
        }
        add_group(sm, f, big, c);
    }
    if (has_single) {
        if (!(single <= sm.m))
            sm.raise(max_nan(sm.m, single), c);
        sm.add(single, c);
    }
    __syncwarp();
    join_lanes(sm, c);
    if (lane == 0) {
        sh.sum[0] = sm.m;
        sh.sum[1] = sm.s;
        sh.sum[2] = sm.t;
    }
    __syncwarp();
    if (p.top)
        select_top<T>(sh, gmax[warp], a, p.top, min(kWarpSlots, (groups * U + (1u << shift) - 1) >> shift), shift,
                      has_single, single, single_at);
    write_row(p, sh, r, tok, xtok);
}

// Long rows.  A block walks the rows b, b + blocks, ... (split = 1), or a
// cluster of `split` blocks shares one row and joins its parts through
// distributed shared memory.  A copy warp streams the rows' vectors into a
// ring (16 KB bulk copies, several in flight, on over the end of a row);
// eight warps run the softmax and leave each row's sums and group maxima in
// one of two buffers; four warps select the alternatives and write the row
// meanwhile.  (With the eight warps selecting, the ring idled for most of a
// row: 4096 rows of 50021 float32, top 20: 221 us.)  One pass over the logits,
// bound by HBM.  If a bounded wait runs out, the block's remaining rows get
// NaN.
constexpr int kStreamThreads = kLpThreads + kSelThreads + 32;
struct RowBuffer {
    float gmax[kSlots][kLpThreads];
    float m[kLpWarps], s[kLpWarps], t[kLpWarps];
    uint32_t failed;
};
struct StreamShared {
    RowBuffer row[2];
    BlockTeam team;
    uint64_t full[kStages], empty[kStages];
};
// Hand a buffer over between the eight and the four warps (barriers 2 to 5).
// A warp arrives as a whole: had it split at the branch before (a lane that
// writes for its warp), the aligned form would count it twice.
__device__ __forceinline__ void buffer_arrive(uint32_t id)
{
    __syncwarp();
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "n"(kLpThreads + kSelThreads) : "memory");
}
__device__ __forceinline__ void buffer_sync(uint32_t id)
{
    __syncwarp();
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(kLpThreads + kSelThreads) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kStreamThreads, 2) logprob_stream_kernel(LogprobParams p, uint32_t split)
{
    extern __shared__ __align__(128) uint8_t raw[];
    constexpr uint32_t V = RowView<T>::V, U = RowView<T>::U;
    uint8_t *ring = raw;
    StreamShared &ss = *reinterpret_cast<StreamShared *>(raw + kStages * kStageBytes);
    BlockTeam &sh = ss.team;
    const uint32_t rank = split > 1 ? cluster_rank() : 0;
    const uint64_t step = split > 1 ? p.rows : gridDim.x, r0 = blockIdx.x / split;
    const float c = p.scale * 1.44269504f;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(&ss.full[i], 1);
            mbar_init(&ss.empty[i], kLpWarps);
        }
        fence_mbar_init();
        fence_proxy_async();
        ss.row[0].failed = ss.row[1].failed = 0;
    }
    __syncthreads();
    int64_t row_tok = -1; // of the cluster's one row
    float row_xtok = 0.f;
    auto share_of = [&](uint64_t r) {
        const RowView<T> row(static_cast<const T *>(p.logits) + r * p.ld, p.vocab);
        // (split is a power of two)
        const uint32_t shift = 31 - __clz(split);
        return Share<T>{row, (uint32_t)((uint64_t)row.vecs * rank >> shift), (uint32_t)((uint64_t)row.vecs * (rank + 1) >> shift),
                        (uint32_t)p.vocab, rank == 0 ? row.head + row.tail : 0};
    };
    auto groups_of = [&](const Share<T> &a) { return (a.v1 - a.v0 + U * kLpThreads - 1) / (U * kLpThreads); };
    auto per_slot_of = [&](uint32_t groups) { // a power of two
        uint32_t n = 1;
        while (n * kSlots < groups)
            n *= 2;
        return n;
    };
    if (threadIdx.x >= kLpThreads + kSelThreads) { // the copy warp
        if (threadIdx.x == kLpThreads + kSelThreads) {
            uint32_t st = 0, ph = 0, issued = 0;
            bool ok = true;
            // the ring may be full while an earlier row's alternatives are looked for: at worst (every value a new
            // best one, ranked 352 at a time) that takes some 50 ns a value
            const uint64_t limit = kWaitLimitNs + 200 * p.vocab;
            for (uint64_t r = r0; r < p.rows && ok; r += step) {
                const Share<T> a = share_of(r);
                for (uint32_t v = a.v0; v < a.v1; v += kStageVecs) {
                    if (!(ok = mbar_wait(&ss.empty[st], ph ^ 1, limit)))
                        break;
                    const uint32_t bytes = min(kStageVecs, a.v1 - v) * 16;
                    mbar_expect_tx(&ss.full[st], bytes);
                    bulk_g2s(ring + st * kStageBytes, a.row.vec(v), bytes, &ss.full[st]);
                    ++issued;
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) // the copies in flight: a last wait each
                for (uint32_t i = 0; i < min(issued, kStages); ++i) {
                    if (st == 0) {
                        st = kStages;
                        ph ^= 1;
                    }
                    --st;
                    (void)mbar_wait(&ss.full[st], ph, kWaitLimitNs);
                }
        }
    } else if (threadIdx.x < kLpThreads) { // the softmax
        const uint32_t tid = threadIdx.x;
        uint32_t st = 0, ph = 0, b = 0;
        bool ok = true; // a wait that runs out ends the block's loads
        for (uint64_t r = r0; r < p.rows; r += step, b ^= 1) {
            RowBuffer &buf = ss.row[b];
            if (r >= r0 + 2 * step)
                buffer_sync(4 + b); // the row before last is written
            const Share<T> a = share_of(r);
            const uint32_t nv = a.v1 - a.v0, groups = groups_of(a), whole = nv / (U * kLpThreads);
            const uint32_t per_slot = per_slot_of(groups);
            Softmax sm;
            uint32_t slot = 0;
            float slot_max = -INFINITY;
            uint32_t left = per_slot; // groups left of the slot
            for (uint32_t g = 0; g < groups; ++g) {
                float2 f[16];
#pragma unroll
                for (uint32_t h = 0; h < U / 4; ++h) { // a group's stages
                    uint32_t count = kStageVecs;
                    if (g == whole) {
                        const uint32_t done = g * U * kLpThreads + h * kStageVecs;
                        count = done < nv ? min(kStageVecs, nv - done) : 0;
                    }
                    if (count && !(ok = ok && mbar_wait(&ss.full[st], ph, kWaitLimitNs)))
                        break;
                    const uint4 *q = reinterpret_cast<const uint4 *>(ring + st * kStageBytes) + tid;
                    if (count == kStageVecs) {
#pragma unroll
                        for (uint32_t u = 0; u < 4; ++u)
                            unpack2<T>(q[u * kLpThreads], f + (h * 4 + u) * V / 2);
                    } else {
#pragma unroll
                        for (uint32_t u = 0; u < 4; ++u)
                            if (tid + u * kLpThreads < count) {
                                unpack2<T>(q[u * kLpThreads], f + (h * 4 + u) * V / 2);
                            } else {
#pragma unroll
                                for (uint32_t i = 0; i < V / 2; ++i)
                                    f[(h * 4 + u) * V / 2 + i] = both(-INFINITY);
                            }
                    }
                    if (count) {
                        // The values have to be in registers before the copy warp may fill the stage again: an
                        // arrival alone does not wait for this warp's loads (float32 values, which nothing
                        // converts, were still on their way).
                        fence_proxy_async();
                        __syncwarp();
                        if ((tid & 31) == 0)
                            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&ss.empty[st])) : "memory");
                        if (++st == kStages) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                }
                if (!ok) {
                    ss.row[0].failed = ss.row[1].failed = 1;
                    break;
                }
                const float big = largest_of<16>(f);
                add_group(sm, f, big, c);
                slot_max = max_nan(slot_max, big);
                if (--left == 0 || g + 1 == groups) {
                    if (p.top)
                        buf.gmax[slot][tid] = slot_max;
                    ++slot;
                    left = per_slot;
                    slot_max = -INFINITY;
                }
            }
            __syncwarp();
            join_lanes(sm, c);
            if ((tid & 31) == 0) {
                buf.m[tid >> 5] = sm.m;
                buf.s[tid >> 5] = sm.s;
                buf.t[tid >> 5] = sm.t;
            }
            buffer_arrive(2 + b);
        }
    } else { // the alternatives and the outputs
        const uint32_t tid = BlockTeam::thread();
        // asked for a row ahead: the token, its logit, the values at the row's ends (threads 8 to 21)
        struct {
            int64_t tok;
            T logit, single;
        } next{-1, T(0.f), T(0.f)};
        auto token_of = [&](uint64_t r) { return r < p.rows && p.tokens && tid == 0 && rank == 0 ? p.tokens[r] : (int64_t)-1; };
        auto ask = [&](uint64_t r) {
            if (r >= p.rows)
                return;
            const Share<T> a = share_of(r);
            if (next.tok >= 0 && next.tok < (int64_t)p.vocab)
                next.logit = a.row.x[next.tok];
            if (tid >= 8 && tid - 8 < a.singles)
                next.single = a.row.x[a.row.single(tid - 8)];
        };
        next.tok = token_of(r0);
        ask(r0);
        uint32_t b = 0;
        for (uint64_t r = r0; r < p.rows; r += step, b ^= 1) {
            RowBuffer &buf = ss.row[b];
            const Share<T> a = share_of(r);
            const int64_t tok = next.tok;
            const float xtok = to_f32(next.logit);
            const bool has_single = tid >= 8 && tid - 8 < a.singles;
            const uint32_t single_at = has_single ? a.row.single(tid - 8) : 0;
            const float single = has_single ? to_f32(next.single) : -INFINITY;
            next.tok = token_of(r + step);
            const uint32_t groups = groups_of(a);
            const uint32_t per_slot = per_slot_of(groups);
            buffer_sync(2 + b);
            const bool failed = buf.failed;
            if (tid < 32) {
                Softmax sm;
                if (tid < kLpWarps) {
                    sm.m = failed ? NAN : buf.m[tid];
                    sm.s = buf.s[tid];
                    sm.t = buf.t[tid];
                } else if (has_single) {
                    sm.m = single;
                    sm.add(single, c);
                }
                join_lanes(sm, c);
                if (tid == 0) {
                    sh.sum[0] = sm.m;
                    sh.sum[1] = sm.s;
                    sh.sum[2] = sm.t;
                }
            }
            if (failed) {
                for (uint32_t i = tid; i < p.top; i += kSelThreads)
                    sh.best[i] = order_key(NAN, 0);
            } else if (p.top) {
                select_top<T>(sh, buf.gmax, a, p.top, (groups + per_slot - 1) / per_slot, 31 - __clz(per_slot * U),
                              has_single, single, single_at);
            }
            BlockTeam::sync();
            if (r + 2 * step < p.rows)
                buffer_arrive(4 + b);
            if (split > 1) { // one row a cluster; its parts are joined below
                row_tok = tok;
                row_xtok = xtok;
                break;
            }
            ask(r + step);
            write_row(p, sh, r, tok, xtok);
            BlockTeam::sync(); // the next row writes what write_row reads
        }
    }
    if (split == 1)
        return;
    __syncwarp();
    cluster_sync(); // every part is there
    if (rank == 0 && threadIdx.x >= kLpThreads && threadIdx.x < kLpThreads + kSelThreads) {
        const uint32_t tid = BlockTeam::thread();
        if (tid < 32) {
            Softmax sm;
            if (tid < split) {
                const uint32_t at = cluster_addr(smem_u32(sh.sum), tid);
                sm.m = cluster_load(at);
                sm.s = cluster_load(at + 4);
                sm.t = cluster_load(at + 8);
            }
            join_lanes(sm, c);
            if (tid == 0) {
                sh.sum[0] = sm.m;
                sh.sum[1] = sm.s;
                sh.sum[2] = sm.t;
            }
        }
        // the blocks' lists are in order (a short one ends in zeros): a key's rank is its place and the
        // number of larger keys in each other list
        const uint32_t n = split * p.top; // at most 256
        for (uint32_t i = tid; i < n; i += kSelThreads) {
            const uint32_t at = cluster_addr(smem_u32(sh.best + i % p.top), i / p.top);
            const uint32_t lo = __float_as_uint(cluster_load(at)), hi = __float_as_uint(cluster_load(at + 4));
            sh.key[i] = (unsigned long long)hi << 32 | lo;
        }
        BlockTeam::sync();
#pragma unroll 1
        for (uint32_t i = tid; i < n; i += kSelThreads) {
            const unsigned long long key = sh.key[i];
            const uint32_t own = i / p.top;
            uint32_t rank_of = i - own * p.top;
            for (uint32_t q = 0; q < split; ++q) {
                uint32_t count = 0; // keys of list q above this one
#pragma unroll
                for (uint32_t step = 16; step; step >>= 1)
                    if (count + step <= p.top && sh.key[q * p.top + count + step - 1] > key)
                        count += step;
                if (q != own)
                    rank_of += count < p.top && sh.key[q * p.top + count] > key ? count + 1 : count;
            }
            if (key && rank_of < p.top)
                sh.best[rank_of] = key;
        }
        BlockTeam::sync();
        write_row(p, sh, r0, row_tok, row_xtok);
    }
    __syncwarp();
    cluster_sync(); // the first block has read the others' parts
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
    __device__ __forceinline__ float log2p(float x) const { return fmaxf(fmaf(x - m, c, -l), -200.f); }
    __device__ __forceinline__ float value(float x) const
    {
        const float g = log2p(x);
        return exp2_fast(g) * fmaf(B, g, A);
    }
    __device__ __forceinline__ float2 value2(float2 x) const
    {
        float2 g = fma2(add2(x, both(-m)), both(c), both(-l));
        g = make_float2(fmaxf(g.x, -200.f), fmaxf(g.y, -200.f));
        return mul2(make_float2(exp2_fast(g.x), exp2_fast(g.y)), fma2(both(B), g, both(A)));
    }
    __device__ __forceinline__ float token_value(float x) const
    {
        const float g = log2p(x);
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
    bool none = lse == -INFINITY, nan = !(lse < INFINITY);
    if (fabsf(lse) > kLseMost && (fabsf(lse) < INFINITY || p.scale > 1.f)) {
        float m = -INFINITY, s = 0.f;
        for (uint64_t i = tid; i < p.vocab; i += kLpThreads)
            m = fmaxf(m, to_f32(x[i]));
        row.m = block_reduce(m, [](float a, float b) { return fmaxf(a, b); });
        none = row.m == -INFINITY;
        nan = row.m == INFINITY;
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
    if (none) { // no token has a probability
        row.A = row.B = row.m = row.l = 0.f;
        row.tok = -1;
    } else if (nan) { // every value is NaN, the token's too
        row.A = NAN;
        row.tok = -1;
    }
    const RowView<T> view(x, p.vocab);
    if ((((uintptr_t)x ^ (uintptr_t)d) & 15) == 0) { // both rows' vectors start at the same value
        const uint32_t v0 = (uint64_t)view.vecs * part / split, v1 = (uint64_t)view.vecs * (part + 1) / split;
        uint4 *out = reinterpret_cast<uint4 *>(d + view.head);
        // the token's vector, if it lies in one
        const uint64_t tv = row.tok >= (int64_t)view.head ? (uint64_t)(row.tok - view.head) / V : ~0ull;
        for (uint32_t i0 = v0 + tid; i0 < v1; i0 += 4 * kLpThreads) {
            uint4 q[4];
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                if (i0 + u * kLpThreads < v1)
                    q[u] = load_once(view.vec(i0 + u * kLpThreads));
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                const uint32_t i = i0 + u * kLpThreads;
                if (i < v1) {
                    float2 f[V / 2], o[V / 2];
                    unpack2<T>(q[u], f);
#pragma unroll
                    for (uint32_t k = 0; k < V / 2; ++k)
                        o[k] = row.value2(f[k]);
                    if (i == tv) {
                        const uint32_t at = (uint32_t)(row.tok - view.head) % V;
#pragma unroll
                        for (uint32_t k = 0; k < V / 2; ++k) {
                            if (at == 2 * k)
                                o[k].x = row.token_value(f[k].x);
                            if (at == 2 * k + 1)
                                o[k].y = row.token_value(f[k].y);
                        }
                    }
                    st_stream16(out + i, pack2<T>(o));
                }
            }
        }
        if (part == 0)
            for (uint32_t k = tid; k < view.head + view.tail; k += kLpThreads) {
                const uint32_t i = view.single(k);
                const float f = to_f32(x[i]);
                d[i] = from_f32<T>((uint64_t)row.tok == i ? row.token_value(f) : row.value(f));
            }
    } else { // the gradient's vectors begin elsewhere: the logits are read across boundaries
        const RowView<T> out_view(d, p.vocab);
        const uint32_t v0 = (uint64_t)out_view.vecs * part / split, v1 = (uint64_t)out_view.vecs * (part + 1) / split;
        uint4 *out = reinterpret_cast<uint4 *>(d + out_view.head);
        const T *from = x + out_view.head;
        const void *begin = p.logits, *end = static_cast<const T *>(p.logits) + (p.rows - 1) * p.ld + p.vocab;
        const uint64_t tv = row.tok >= (int64_t)out_view.head ? (uint64_t)(row.tok - out_view.head) / V : ~0ull;
        for (uint32_t i0 = v0 + tid; i0 < v1; i0 += 2 * kLpThreads) {
            uint4 q[2];
#pragma unroll
            for (uint32_t u = 0; u < 2; ++u)
                if (i0 + u * kLpThreads < v1)
                    q[u] = load_anywhere(from + (uint64_t)(i0 + u * kLpThreads) * V, begin, end);
#pragma unroll
            for (uint32_t u = 0; u < 2; ++u) {
                const uint32_t i = i0 + u * kLpThreads;
                if (i < v1) {
                    float2 f[V / 2], o[V / 2];
                    unpack2<T>(q[u], f);
#pragma unroll
                    for (uint32_t k = 0; k < V / 2; ++k)
                        o[k] = row.value2(f[k]);
                    if (i == tv) {
                        const uint32_t at = (uint32_t)(row.tok - out_view.head) % V;
#pragma unroll
                        for (uint32_t k = 0; k < V / 2; ++k) {
                            if (at == 2 * k)
                                o[k].x = row.token_value(f[k].x);
                            if (at == 2 * k + 1)
                                o[k].y = row.token_value(f[k].y);
                        }
                    }
                    st_stream16(out + i, pack2<T>(o));
                }
            }
        }
        if (part == 0)
            for (uint32_t k = tid; k < out_view.head + out_view.tail; k += kLpThreads) {
                const uint32_t i = out_view.single(k);
                const float f = to_f32(x[i]);
                d[i] = from_f32<T>((uint64_t)row.tok == i ? row.token_value(f) : row.value(f));
            }
    }
}

namespace {

// CTAs a row, in powers of two: at most `ctas` in all while a CTA keeps at
// least `least` values
uint32_t row_split(uint64_t rows, uint64_t vocab, uint64_t ctas, uint64_t least)
{
    uint32_t s = 1;
    while (s < 8 && rows * s * 2 <= ctas && vocab / (2 * s) >= least)
        s *= 2;
    return s;
}

cudaLaunchConfig_t row_config(uint64_t rows, uint32_t split, int threads, size_t smem, cudaLaunchAttribute *at, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * split));
    cfg.blockDim = dim3(threads);
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
    if (sms <= 0)
        return ECC_ERR_CUDA;
    // a warp a row where that fills the GPU, or where a block would have
    // fewer than eight values a thread
    if (p.vocab <= 2048 || (p.vocab <= 8192 && p.rows >= 8ull * sms)) {
        if (p.rows > (1ull << 32))
            return ECC_ERR_ARG;
        logprob_warp_kernel<T><<<(unsigned)((p.rows + 3) / 4), 128, 0, st>>>(p);
        return launch_status(cudaGetLastError());
    }
    const size_t smem = kStages * kStageBytes + sizeof(StreamShared);
    if (occupancy((const void *)logprob_stream_kernel<T>, kStreamThreads, smem) <= 0)
        return ECC_ERR_CUDA;
    const uint32_t split = row_split(p.rows, p.vocab, 2ull * sms, 4096);
    const uint64_t rows = split > 1 ? p.rows : std::min<uint64_t>(p.rows, 2ull * sms);
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = row_config(rows, split, kStreamThreads, smem, &at, st);
    return launch_status(cudaLaunchKernelEx(&cfg, logprob_stream_kernel<T>, p, split));
}

template <typename T> ecc_status logprob_grad_launch(const LogprobGradParams &p, cudaStream_t st)
{
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    const uint32_t split = row_split(p.rows, p.vocab, 16ull * sms, 4096);
    if (p.rows >= (1ull << 31) / split)
        return ECC_ERR_ARG;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = row_config(p.rows, split, kLpThreads, 0, &at, st);
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
