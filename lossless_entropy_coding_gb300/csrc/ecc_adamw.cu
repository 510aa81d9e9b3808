// ecc_adamw.cu -- AdamW over many tensors in one launch, states in float32 or
// in e4m3 bytes with a scale for each kAdamGroup values.
//
// Each value is read, updated and written once.  A warp takes a group of 256
// values, so that the largest magnitude of an 8-bit state's group is one warp
// reduction; the tensors' pointers travel as kernel parameters, so nothing is
// copied to the device first and a captured call keeps them.

#include <algorithm>
#include <cmath>
#include <limits>
#include <utility>
#include <vector>

#include "ecc_act.cuh"

namespace ecc {

constexpr uint32_t kAdamGroup = ECC_ADAMW_GROUP;
constexpr uint32_t kAdamVectors = 16; // of a tensor's kind: 16-byte accesses

struct AdamTensor {
    void *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale, *master;
    uint64_t n;
};
struct AdamHyper {
    float beta1, beta2, gain1, gain2; // gain = 1 - beta
    float log_beta1, log_beta2, eps, weight_decay, lr, grad_scale;
    float rate, root; // 1 / (1 - beta1^step), sqrt(1 / (1 - beta2^step))
    uint32_t seed, step;
    const float *lr_at, *grad_scale_at;
    const int64_t *step_at;
};
// Up to CAP tensors: their first tiles, and kinds (types of parameter and
// gradient, 2 bits each, and the bit above).
template <int CAP> struct AdamArgs {
    AdamHyper h;
    uint32_t count;
    uint32_t first[CAP + 1];
    AdamTensor t[CAP];
    uint8_t kind[CAP];
};

// A mixing of 32-bit numbers: two multiplications between three shifts, with
// the constants that C. Wellons published for it ("Prospecting for Hash
// Functions", 2018).
__host__ __device__ inline uint32_t mix32(uint32_t x)
{
    x = (x ^ x >> 16) * 0x7FEB352Du;
    x = (x ^ x >> 15) * 0x846CA68Bu;
    return x ^ x >> 16;
}

// what a step's values have in common
struct AdamStep {
    float beta1, beta2, gain1, gain2, eps, keep, rate, root, grad_scale;
    uint32_t key;
};
__device__ __forceinline__ AdamStep step_of(const AdamHyper &h)
{
    AdamStep s;
    const float lr = h.lr_at ? *h.lr_at : h.lr;
    s.beta1 = h.beta1;
    s.beta2 = h.beta2;
    s.gain1 = h.gain1;
    s.gain2 = h.gain2;
    s.eps = h.eps;
    s.keep = 1.f - lr * h.weight_decay;
    s.grad_scale = h.grad_scale_at ? *h.grad_scale_at : h.grad_scale;
    uint32_t step = h.step;
    s.rate = h.rate;
    s.root = h.root;
    if (h.step_at) {
        const int64_t t = *h.step_at;
        step = (uint32_t)t;
        s.rate = -1.f / expm1f((float)t * h.log_beta1);
        s.root = sqrtf(-1.f / expm1f((float)t * h.log_beta2));
    }
    s.rate *= lr;
    s.key = mix32(mix32(h.seed) + step);
    return s;
}

__device__ __forceinline__ float rsqrt_approx(float x)
{
    float y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// sqrt(x), x >= 0: a Newton step on the approximate reciprocal root (the
// result is the nearest float32 but for about one in a million).  The step is
// NaN, from 0 times infinity, where x is its own root: 0 and infinity.
__device__ __forceinline__ float2 root2(float2 x)
{
    const float2 y = make_float2(rsqrt_approx(x.x), rsqrt_approx(x.y)), r = mul2(x, y);
    const float2 e = fma2(mul2(r, both(-1.f)), r, x), f = fma2(e, mul2(y, both(0.5f)), r);
    return make_float2(f.x == f.x ? f.x : x.x, f.y == f.y ? f.y : x.y);
}

// p, m, v of two values.  The roundings of the moments are those of separate
// multiplications and sums, so that a step can be followed to the bit; the
// parameter takes this step's moments as they are before they are stored.
// Returns sqrt(v).
__device__ __forceinline__ float2 update2(const AdamStep &s, float2 g, float2 &p, float2 &m, float2 &v)
{
    g = mul2(g, both(s.grad_scale));
    // (packed sums of packed products would be fused)
    const float2 a = mul2(m, both(s.beta1)), b = mul2(g, both(s.gain1));
    m = make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
    const float2 c = mul2(v, both(s.beta2)), d = mul2(mul2(g, g), both(s.gain2));
    v = make_float2(__fadd_rn(c.x, d.x), __fadd_rn(c.y, d.y));
    const float2 r = root2(v);
    p = fma2(p, both(s.keep), mul2(mul2(m, both(-s.rate)), rcp_both(fma2(r, both(s.root), both(s.eps)))));
    return r;
}

// The e4m3 code of a magnitude of at most 448, in the top byte: one of its two
// neighbours, the upper one with the probability that the remainder is of
// their distance (16 random bits, at bit 8 of d, added below the kept 3 bits of
// the mantissa; d's top byte takes the difference of the exponents' biases).  Below 2^-6, where the neighbours are 2^-9
// apart, that is done behind a shift into the binade that has this distance;
// the larger of the two results is the right one everywhere: above 2^-6 the
// shifted value's neighbours are further apart, below 2^-6 the value's own
// code, taken as a normal one, is the smaller.
__device__ __forceinline__ uint32_t dithered(float a, uint32_t d)
{
    const uint32_t n = (__float_as_uint(fmaxf(a, 0.0078125f)) << 4) + d;
    return max(n, (__float_as_uint(a + 0.015625f) << 4) + d - (8u << 24));
}
// The same for a value of at least 2^-6, of any sign, that may exceed 448 by a
// few last places (which the addition does not carry over).
__device__ __forceinline__ uint32_t dithered_normal(float y, uint32_t d) { return (__float_as_uint(y) << 4) + d; }
__device__ __forceinline__ uint32_t m_bits(uint32_t d) { return __byte_perm(d, 0x40000000u, 0x7324); }
__device__ __forceinline__ uint32_t v_bits(uint32_t d) { return __byte_perm(d, 0x40000000u, 0x7104); }
// the larger one, or NaN if there is one
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// for m (signed) and sqrt(v), from 448 / the group's largest
__device__ __forceinline__ uint32_t m_dithered(float y, uint32_t d)
{
    return dithered(fminf(fabsf(y), 448.f), m_bits(d));
}
__device__ __forceinline__ uint32_t v_dithered(float y, uint32_t d)
{
    return dithered(y > 0.f ? fminf(fmaxf(y, 0.001953125f), 448.f) : 0.f, v_bits(d));
}
// the top bytes of four words
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// A group's scales from the bits of its largest magnitudes (a NaN or infinity
// lies above all others); returns 448 / largest, which is finite from
// kAdamLeast on, or 0 below it.
constexpr float kAdamLeast = 1.5046328e-36f; // 2^-119; 448 / float32's largest is 1.3166e-36
__device__ __forceinline__ float group_scale(float *scale, uint32_t bits, bool root, bool finite, bool write)
{
    float top = __uint_as_float(bits);
    if (root)
        top = root2(both(top)).x;
    if (write)
        *scale = finite ? __fmul_rn(top, 1.f / 448.f) : __int_as_float(0x7FC00000);
    return finite && top >= kAdamLeast ? __fmul_rn(__frcp_rn(top), 448.f) : 0.f;
}

// 8 values from element i, as read: 4-byte types fill both vectors
__device__ __forceinline__ void read8(const void *p, uint64_t i, bool wide, uint4 (&q)[2])
{
    if (wide) {
        q[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i));
        q[1] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i) + 1);
    } else {
        q[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
    }
}
__device__ __forceinline__ void unpack8(const uint4 (&q)[2], uint32_t type, float2 (&f)[4])
{
    if (type == ECC_F32) {
        unpack2<float>(q[0], f);
        unpack2<float>(q[1], f + 2);
    } else if (type == ECC_BF16) {
        unpack2<bf16>(q[0], f);
    } else {
        unpack2<__half>(q[0], f);
    }
}
__device__ __forceinline__ void write8(void *p, uint64_t i, uint32_t type, const float2 (&f)[4])
{
    if (type == ECC_F32) {
        __stcs(reinterpret_cast<uint4 *>(static_cast<float *>(p) + i), pack2<float>(f));
        __stcs(reinterpret_cast<uint4 *>(static_cast<float *>(p) + i) + 1, pack2<float>(f + 2));
    } else {
        __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i), type == ECC_BF16 ? pack2<bf16>(f) : pack2<__half>(f));
    }
}
__device__ __forceinline__ void unpack_e4m3(uint2 q, float scale, float2 (&f)[4])
{
    const uint32_t w[4] = {q.x & 0xFFFFu, q.x >> 16, q.y & 0xFFFFu, q.y >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w[k], __NV_E4M3);
        f[k] = mul2(__half22float2(__half2(h)), both(scale));
    }
}

// Value k of a lane's 8 in a group: 8 neighbours where the tensor's arrays
// start on 16-byte boundaries (8 for byte states) and the group is whole,
// else one of each 32, so that the lanes are neighbours.
template <bool VECTORS> __device__ __forceinline__ uint32_t place_of(uint32_t lane, int k) { return VECTORS ? lane * 8 + k : k * 32 + lane; }

// 8 values, by type
template <typename T>
__device__ __forceinline__ void read_each(const void *p, uint64_t e0, uint32_t left, uint32_t lane, float2 (&f)[4])
{
    const T *q = static_cast<const T *>(p) + e0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t i = place_of<false>(lane, k);
        (k & 1 ? f[k / 2].y : f[k / 2].x) = i < left ? to_f32(q[i]) : 0.f;
    }
}
__device__ __forceinline__ void read_each(const void *p, uint64_t e0, uint32_t left, uint32_t lane, uint32_t type, float2 (&f)[4])
{
    if (type == ECC_F32)
        read_each<float>(p, e0, left, lane, f);
    else if (type == ECC_BF16)
        read_each<bf16>(p, e0, left, lane, f);
    else
        read_each<__half>(p, e0, left, lane, f);
}
template <typename T>
__device__ __forceinline__ void write_each(void *p, uint64_t e0, uint32_t left, uint32_t lane, const float2 (&f)[4])
{
    T *q = static_cast<T *>(p) + e0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t i = place_of<false>(lane, k);
        if (i < left)
            q[i] = from_f32<T>(k & 1 ? f[k / 2].y : f[k / 2].x);
    }
}
template <bool VECTORS>
__device__ __forceinline__ void write_values(void *p, uint64_t e0, uint32_t left, uint32_t lane, uint32_t type, const float2 (&f)[4])
{
    if constexpr (VECTORS)
        write8(p, e0 + lane * 8, type, f);
    else if (type == ECC_F32)
        write_each<float>(p, e0, left, lane, f);
    else if (type == ECC_BF16)
        write_each<bf16>(p, e0, left, lane, f);
    else
        write_each<__half>(p, e0, left, lane, f);
}

// A warp's group; everything is asked for before anything is used.  (67 M bf16
// values with 8-bit states 235 us by values, 187 by vectors, with float32 states
// 282 and 229.)
template <bool BYTES, bool VECTORS>
__device__ __forceinline__ void update_group(const AdamTensor &t, uint32_t kind, uint64_t e0, uint32_t lane, const AdamStep &s)
{
    const uint32_t ptype = kind & 3, gtype = kind >> 2 & 3;
    const uint32_t left = (uint32_t)min(t.n - e0, (uint64_t)kAdamGroup);
    const void *from = t.master ? t.master : t.param;
    const uint32_t from_type = t.master ? (uint32_t)ECC_F32 : ptype;
    float2 p[4], g[4], m[4], v[4];
    float *msp = nullptr, *vsp = nullptr;
    float ms = 1.f, vs = 1.f;
    if constexpr (BYTES) {
        msp = t.m_scale + e0 / kAdamGroup;
        vsp = t.v_scale + e0 / kAdamGroup;
    }
    if constexpr (VECTORS) {
        const uint64_t i = e0 + lane * 8;
        uint4 pq[2], gq[2], mq[2], vq[2];
        if constexpr (BYTES) {
            const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.m) + i));
            const uint2 b = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.v) + i));
            mq[0] = make_uint4(a.x, a.y, 0, 0);
            vq[0] = make_uint4(b.x, b.y, 0, 0);
            ms = *msp;
            vs = *vsp;
        } else {
            read8(t.m, i, true, mq);
            read8(t.v, i, true, vq);
        }
        read8(from, i, from_type == ECC_F32, pq);
        read8(t.grad, i, gtype == ECC_F32, gq);
        unpack8(pq, from_type, p);
        unpack8(gq, gtype, g);
        if constexpr (BYTES) {
            unpack_e4m3(make_uint2(mq[0].x, mq[0].y), ms, m);
            unpack_e4m3(make_uint2(vq[0].x, vq[0].y), vs, v);
        } else {
            unpack8(mq, ECC_F32, m);
            unpack8(vq, ECC_F32, v);
        }
    } else {
        if constexpr (BYTES) {
            read_each<e4m3>(t.m, e0, left, lane, m);
            read_each<e4m3>(t.v, e0, left, lane, v);
            ms = *msp;
            vs = *vsp;
        } else {
            read_each<float>(t.m, e0, left, lane, m);
            read_each<float>(t.v, e0, left, lane, v);
        }
        read_each(from, e0, left, lane, from_type, p);
        read_each(t.grad, e0, left, lane, gtype, g);
        if constexpr (BYTES)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = mul2(m[k], both(ms));
                v[k] = mul2(v[k], both(vs));
            }
    }
    if constexpr (BYTES) {
        float m_most = 0.f, v_most = 0.f, m_least = INFINITY, r_least = INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = mul2(v[k], v[k]);
            const float2 r = update2(s, g[k], p[k], m[k], v[k]);
            m_most = max_nan(max_nan(m_most, fabsf(m[k].x)), fabsf(m[k].y));
            v_most = max_nan(max_nan(v_most, v[k].x), v[k].y);
            m_least = fminf(fminf(m_least, fabsf(m[k].x)), fabsf(m[k].y));
            r_least = fminf(fminf(r_least, r.x), r.y);
            v[k] = r;
        }
        if (t.master)
            write_values<VECTORS>(t.master, e0, left, lane, ECC_F32, p);
        write_values<VECTORS>(t.param, e0, left, lane, ptype, p);
        const uint32_t mm = __reduce_max_sync(~0u, __float_as_uint(m_most)), vm = __reduce_max_sync(~0u, __float_as_uint(v_most));
        const bool finite = mm < 0x7F800000u && vm < 0x7F800000u;
        const float mi = group_scale(msp, mm, false, finite, lane == 0);
        const float vi = group_scale(vsp, vm, true, finite, lane == 0);
        const uint32_t key = mix32(s.key + (uint32_t)(e0 >> 32)), low = (uint32_t)e0;
        uint32_t mw[2] = {0, 0}, vw[2] = {0, 0};
        // (no value so small that its neighbours are 2^-9 apart, which few groups have: a third fewer instructions)
        const bool normal = __all_sync(~0u, finite && __fmul_rn(m_least, mi) >= 0.015625f && __fmul_rn(r_least, vi) >= 0.015625f);
        if (finite) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t mc[4], vc[4], sign[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t d = mix32((low + place_of<VECTORS>(lane, h * 4 + k)) ^ key);
                    const float2 y2 = mul2(m[h * 2 + k / 2], both(mi)), z2 = mul2(v[h * 2 + k / 2], both(vi));
                    const float y = k & 1 ? y2.y : y2.x, z = k & 1 ? z2.y : z2.x;
                    sign[k] = __float_as_uint(y);
                    if (normal) {
                        mc[k] = dithered_normal(y, m_bits(d));
                        vc[k] = dithered_normal(z, v_bits(d));
                    } else {
                        mc[k] = m_dithered(y, d);
                        vc[k] = v_dithered(z, d);
                    }
                }
                mw[h] = top_bytes(mc[0], mc[1], mc[2], mc[3]) | (top_bytes(sign[0], sign[1], sign[2], sign[3]) & 0x80808080u);
                vw[h] = top_bytes(vc[0], vc[1], vc[2], vc[3]);
            }
        }
        uint8_t *mp = static_cast<uint8_t *>(t.m) + e0, *vp = static_cast<uint8_t *>(t.v) + e0;
        if constexpr (VECTORS) {
            __stcs(reinterpret_cast<uint2 *>(mp + lane * 8), make_uint2(mw[0], mw[1]));
            __stcs(reinterpret_cast<uint2 *>(vp + lane * 8), make_uint2(vw[0], vw[1]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t i = place_of<false>(lane, k);
                if (i < left) {
                    mp[i] = (uint8_t)(mw[k / 4] >> k % 4 * 8);
                    vp[i] = (uint8_t)(vw[k / 4] >> k % 4 * 8);
                }
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            update2(s, g[k], p[k], m[k], v[k]);
        write_values<VECTORS>(t.m, e0, left, lane, ECC_F32, m);
        write_values<VECTORS>(t.v, e0, left, lane, ECC_F32, v);
        if (t.master)
            write_values<VECTORS>(t.master, e0, left, lane, ECC_F32, p);
        write_values<VECTORS>(t.param, e0, left, lane, ptype, p);
    }
}

template <int CAP, bool BYTES>
__global__ void __launch_bounds__(BYTES ? 1024 : 256, BYTES ? 1 : 2) adamw_kernel(const __grid_constant__ AdamArgs<CAP> a)
{
    const AdamStep s = step_of(a.h);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t at = 0;
    for (uint32_t tile = blockIdx.x; tile < a.first[a.count]; tile += gridDim.x) {
        if (tile >= a.first[at + 1]) { // the last tensor that starts at or before this tile
            uint32_t lo = at + 1, hi = a.count - 1;
            while (lo < hi) {
                const uint32_t mid = (lo + hi + 1) / 2;
                if (a.first[mid] <= tile)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            at = lo;
        }
        const AdamTensor &t = a.t[at];
        const uint32_t kind = a.kind[at];
        const uint64_t e0 = ((uint64_t)(tile - a.first[at]) * (blockDim.x / 32) + warp) * kAdamGroup;
        if (e0 >= t.n)
            continue;
        if ((kind & kAdamVectors) && e0 + kAdamGroup <= t.n)
            update_group<BYTES, true>(t, kind, e0, lane, s);
        else
            update_group<BYTES, false>(t, kind, e0, lane, s);
    }
}

namespace {

// Types and pointers of a tensor; nothing of an empty one is looked at.
bool tensor_ok(const ecc_adamw_tensor &t)
{
    if (!wide_type(t.param_type) || !wide_type(t.grad_type) || (t.state_type != ECC_F32 && t.state_type != ECC_E4M3) || t.reserved)
        return false;
    if (!t.n)
        return true;
    if (t.n >= 1ull << 40 || !t.param || !t.grad || !t.m || !t.v || !aligned_to(t.param, t.param_type) ||
        !aligned_to(t.grad, t.grad_type) || !aligned_to(t.m, t.state_type) || !aligned_to(t.v, t.state_type) ||
        !aligned_to(t.master, ECC_F32))
        return false;
    return t.state_type == ECC_F32 ||
           (t.m_scale && t.v_scale && aligned_to(t.m_scale, ECC_F32) && aligned_to(t.v_scale, ECC_F32));
}

bool by_vectors(const ecc_adamw_tensor &t)
{
    const uintptr_t states = (uintptr_t)t.m | (uintptr_t)t.v;
    return (((uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.master) & 15) == 0 &&
           (states & (t.state_type == ECC_E4M3 ? 7 : 15)) == 0;
}

// Whether nothing that is written overlaps anything else (a tensor given twice
// would be updated by two warps at once, a gradient in another's parameter read
// before or after its update).
bool apart(const ecc_adamw_job &j)
{
    using Span = std::pair<uintptr_t, uintptr_t>; // first byte, end
    const auto by_first = [](const Span &a, const Span &b) { return a.first < b.first; };
    std::vector<Span> spans; // that are written, in order
    spans.reserve(j.count * 6);
    auto add = [&](const void *p, uint64_t bytes) {
        if (p)
            spans.emplace_back((uintptr_t)p, (uintptr_t)p + bytes);
    };
    for (uint64_t i = 0; i < j.count; ++i) {
        const ecc_adamw_tensor &t = j.tensors[i];
        if (!t.n)
            continue;
        const uint64_t state = t.n * type_bytes(t.state_type), scales = (t.n + kAdamGroup - 1) / kAdamGroup * sizeof(float);
        add(t.param, t.n * type_bytes(t.param_type));
        add(t.m, state);
        add(t.v, state);
        add(t.master, t.n * sizeof(float));
        if (t.state_type == ECC_E4M3) {
            add(t.m_scale, scales);
            add(t.v_scale, scales);
        }
    }
    std::sort(spans.begin(), spans.end(), by_first);
    for (size_t i = 1; i < spans.size(); ++i)
        if (spans[i].first < spans[i - 1].second)
            return false;
    // the last one that starts before an array's end has ended before it starts
    const auto clear_of = [&](const void *p, uint64_t bytes) {
        const auto next = std::lower_bound(spans.begin(), spans.end(), Span((uintptr_t)p + bytes, 0), by_first);
        return !p || next == spans.begin() || (next - 1)->second <= (uintptr_t)p;
    };
    for (uint64_t i = 0; i < j.count; ++i)
        if (j.tensors[i].n && !clear_of(j.tensors[i].grad, j.tensors[i].n * type_bytes(j.tensors[i].grad_type)))
            return false;
    return clear_of(j.step_at, sizeof(int64_t)) && clear_of(j.lr_at, sizeof(float)) && clear_of(j.grad_scale_at, sizeof(float));
}

// A launch's threads a block and blocks an SM.  Float32 states are bound by HBM,
// where fewer accesses in flight are better: two blocks of 256 (170 M values with
// masters: 793 us, 6.4 TB/s; three 859, one of 1024 877).  8-bit states are
// bound by instructions, and take 1024 threads an SM: in one block while
// parameters and gradients are of 16 bits (265 M values: 650 us, 4.1 TB/s; in
// four 688, 768 threads 722), in four of 256 where more bytes move with a value
// (67 M values with float32 gradients and masters: 240 us, in one 263; all in
// float32 211 and 233).
struct AdamShape {
    int threads, blocks;
};
AdamShape adam_shape(const ecc_adamw_job &j, bool bytes)
{
    if (!bytes)
        return {256, 2};
    double total = 0, values = 0; // bytes of parameters, masters and gradients
    for (uint64_t i = 0; i < j.count; ++i) {
        const ecc_adamw_tensor &t = j.tensors[i];
        if (t.state_type != ECC_E4M3)
            continue;
        total += (double)t.n * (type_bytes(t.param_type) * (t.master ? 1 : 2) + type_bytes(t.grad_type) + (t.master ? 8 : 0));
        values += (double)t.n;
    }
    return total < 8 * values ? AdamShape{1024, 1} : AdamShape{256, 4};
}

// the next tensors with states of the one kind
template <int CAP, bool BYTES>
ecc_status launch_tensors(const ecc_adamw_job &j, const AdamHyper &h, AdamShape shape, uint64_t &next, cudaStream_t st)
{
    const uint64_t tile = (uint64_t)shape.threads / 32 * kAdamGroup; // values of a block's step
    AdamArgs<CAP> a;
    a.h = h;
    a.count = 0;
    uint64_t tiles = 0;
    for (; next < j.count && a.count < CAP; ++next) {
        const ecc_adamw_tensor &t = j.tensors[next];
        if ((t.state_type == ECC_E4M3) != BYTES)
            continue;
        const uint64_t own = (t.n + tile - 1) / tile;
        if (!own)
            continue;
        if (tiles + own >= 1ull << 31)
            break; // (one tensor has fewer than 2^29 tiles)
        a.first[a.count] = (uint32_t)tiles;
        a.t[a.count] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n};
        a.kind[a.count] = (uint8_t)(t.param_type | t.grad_type << 2 | (by_vectors(t) ? kAdamVectors : 0));
        ++a.count;
        tiles += own;
    }
    if (!a.count)
        return ECC_OK;
    a.first[a.count] = (uint32_t)tiles;
    const int sms = sm_count();
    if (sms <= 0)
        return ECC_ERR_CUDA;
    adamw_kernel<CAP, BYTES><<<(unsigned)std::min(tiles, (uint64_t)sms * shape.blocks), shape.threads, 0, st>>>(a);
    return launch_status(cudaGetLastError());
}

bool job_ok(const ecc_adamw_job &j)
{
    const auto number = [](double v) { return std::isfinite((float)v); };
    if ((j.count && !j.tensors) || j.reserved || !number(j.lr) || !(j.beta1 >= 0 && j.beta1 < 1) ||
        !(j.beta2 >= 0 && j.beta2 < 1) || !(j.eps >= 0) || !number(j.eps) || !number(j.weight_decay) || !number(j.grad_scale) ||
        (!j.step_at && j.step < 1) || ((uintptr_t)j.step_at & 7) || !aligned_to(j.lr_at, ECC_F32) ||
        !aligned_to(j.grad_scale_at, ECC_F32))
        return false;
    for (uint64_t i = 0; i < j.count; ++i)
        if (!tensor_ok(j.tensors[i]))
            return false;
    return true;
}

} // namespace
} // namespace ecc

using namespace ecc;

extern "C" ecc_status ecc_adamw(const ecc_adamw_job *job, void *stream)
try {
    if (!job || !job_ok(*job) || !apart(*job))
        return ECC_ERR_ARG;
    const ecc_adamw_job &j = *job;
    AdamHyper h{};
    h.beta1 = (float)j.beta1;
    h.beta2 = (float)j.beta2;
    h.gain1 = (float)(1 - j.beta1);
    h.gain2 = (float)(1 - j.beta2);
    // (beta = 0: 1 - beta^step is 1 for every step)
    h.log_beta1 = j.beta1 > 0 ? (float)std::log(j.beta1) : -200.f;
    h.log_beta2 = j.beta2 > 0 ? (float)std::log(j.beta2) : -200.f;
    // (the reciprocal takes a subnormal denominator for 0, and 0 / eps is 0)
    h.eps = j.eps > 0 ? std::max((float)j.eps, std::numeric_limits<float>::min()) : 0.f;
    h.weight_decay = (float)j.weight_decay;
    h.lr = (float)j.lr;
    h.grad_scale = (float)j.grad_scale;
    h.seed = j.seed;
    if (!j.step_at) {
        h.step = (uint32_t)j.step;
        h.rate = (float)(1 / (1 - std::pow(j.beta1, (double)j.step)));
        h.root = (float)std::sqrt(1 / (1 - std::pow(j.beta2, (double)j.step)));
    }
    h.lr_at = j.lr_at;
    h.grad_scale_at = j.grad_scale_at;
    h.step_at = j.step_at;
    ecc_status rc = ECC_OK;
    // (parameters of 2 KiB or of 31 KiB: the launch copies them)
    cudaStream_t st = (cudaStream_t)stream;
    const AdamShape wide = adam_shape(j, false), bytes = adam_shape(j, true);
    for (uint64_t next = 0; rc == ECC_OK && next < j.count;)
        rc = j.count - next <= 24 ? launch_tensors<24, false>(j, h, wide, next, st) : launch_tensors<448, false>(j, h, wide, next, st);
    for (uint64_t next = 0; rc == ECC_OK && next < j.count;)
        rc = j.count - next <= 24 ? launch_tensors<24, true>(j, h, bytes, next, st) : launch_tensors<448, true>(j, h, bytes, next, st);
    return rc;
} catch (...) { // no memory for the list of spans
    return ECC_ERR_ARG;
}
