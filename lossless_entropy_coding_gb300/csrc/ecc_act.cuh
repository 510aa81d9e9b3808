// ecc_act.cuh -- the linear operators' activations and their slopes, two
// values at a time.
//
// The Gaussian ones share Phi(a) = 1 - q for a >= 0 and q for a < 0, with q =
// erfc(|a| / sqrt 2) / 2 by Abramowitz and Stegun 7.1.26: erfc(x) = (c1 t + ...
// + c5 t^5) e^(-x^2), t = 1 / (1 + 0.3275911 x), off by at most 1.5e-7 (a
// last place of float32 at 1), and phi(a) from the same e^(-a^2 / 2): about
// nine instructions a value, where erff and expf took the backward pass's
// elementwise kernel 35.
#pragma once

#include "ecc_lm.cuh"

namespace ecc {

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 exp2_both(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_both(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }

// Phi(a) and e^(-a^2 / 2)
__device__ __forceinline__ void gauss2(float2 a, float2 &Phi, float2 &e)
{
    const float2 x = make_float2(fabsf(a.x), fabsf(a.y));
    const float2 t = rcp_both(fma2(x, both(0.3275911f * 0.70710678f), both(1.f)));
    e = exp2_both(mul2(mul2(a, a), both(-0.72134752f))); // log2(e) / 2
    float2 q = fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
    q = fma2(q, t, both(0.5f * 1.421413741f));
    q = fma2(q, t, both(0.5f * -0.284496736f));
    q = fma2(q, t, both(0.5f * 0.254829592f));
    q = mul2(mul2(q, t), e);
    const float2 p = fma2(q, both(-1.f), both(1.f));
    Phi = make_float2(a.x < 0.f ? q.x : p.x, a.y < 0.f ? q.y : p.y);
}
// 1 / (1 + e^-u)
__device__ __forceinline__ float2 logistic2(float2 u)
{
    return rcp_both(add2(exp2_both(mul2(u, both(-1.44269504f))), both(1.f)));
}
// 2 sqrt(2 / pi) (a + 0.044715 a^3): (1 + tanh(u / 2)) / 2 = logistic(u)
__device__ __forceinline__ float2 tanh_argument2(float2 a)
{
    return mul2(a, fma2(mul2(a, a), both(1.59576912f * 0.044715f), both(1.59576912f)));
}

template <uint32_t ACT> __device__ __forceinline__ float2 act_value2(float2 a)
{
    if constexpr (ACT == ECC_ACT_RELU) { // NaN stays
        return make_float2(a.x < 0.f ? 0.f : a.x, a.y < 0.f ? 0.f : a.y);
    } else if constexpr (ACT == ECC_ACT_GELU) {
        float2 Phi, e;
        gauss2(a, Phi, e);
        return mul2(a, Phi);
    } else if constexpr (ACT == ECC_ACT_GELU_TANH) {
        return mul2(a, logistic2(tanh_argument2(a)));
    } else if constexpr (ACT == ECC_ACT_SILU) {
        return mul2(a, logistic2(a));
    } else {
        return a;
    }
}

template <uint32_t ACT> __device__ __forceinline__ float2 act_slope2(float2 a)
{
    if constexpr (ACT == ECC_ACT_RELU) {
        return make_float2(a.x > 0.f ? 1.f : (a.x != a.x ? a.x : 0.f), a.y > 0.f ? 1.f : (a.y != a.y ? a.y : 0.f));
    } else if constexpr (ACT == ECC_ACT_GELU) { // Phi(a) + a phi(a)
        float2 Phi, e;
        gauss2(a, Phi, e);
        return fma2(mul2(a, both(0.39894228f)), e, Phi);
    } else if constexpr (ACT == ECC_ACT_GELU_TANH) { // h + a h (1 - h) u'
        // (a h (1 - h) first, and a finite u': for large a it is 0 times what overflows)
        const float2 h = logistic2(tanh_argument2(a));
        const float2 du = fma2(mul2(a, a), both(3.f * 1.59576912f * 0.044715f), both(1.59576912f));
        const float2 t = mul2(a, fma2(mul2(h, both(-1.f)), h, h));
        return fma2(t, make_float2(fminf(du.x, 3e38f), fminf(du.y, 3e38f)), h);
    } else if constexpr (ACT == ECC_ACT_SILU) { // h (1 + a (1 - h))
        const float2 h = logistic2(a);
        return fma2(a, fma2(mul2(h, both(-1.f)), h, h), h);
    } else {
        return both(1.f);
    }
}

} // namespace ecc
