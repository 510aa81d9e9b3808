// ecc_lm.cuh -- element types, conversions and block reductions shared by the
// language-model operators (layer norm, matrix product, token log
// probabilities).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/ecc_lm.h"
#include "ecc_launch.h"

namespace ecc {

using bf16 = __nv_bfloat16;
struct e4m3 {
    uint8_t b;
};

template <typename T> struct TypeCode;
template <> struct TypeCode<float> { static constexpr uint32_t value = ECC_F32; };
template <> struct TypeCode<bf16> { static constexpr uint32_t value = ECC_BF16; };
template <> struct TypeCode<__half> { static constexpr uint32_t value = ECC_F16; };
template <> struct TypeCode<e4m3> { static constexpr uint32_t value = ECC_E4M3; };

inline uint32_t type_bytes(uint32_t t) { return t == ECC_F32 ? 4u : t == ECC_E4M3 ? 1u : 2u; }
inline bool wide_type(uint32_t t) { return t == ECC_F32 || t == ECC_BF16 || t == ECC_F16; }
inline bool aligned_to(const void *p, uint32_t t) { return ((uintptr_t)p & (type_bytes(t) - 1)) == 0; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(e4m3 v)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v.b, __NV_E4M3)));
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ e4m3 from_f32<e4m3>(float v)
{
    return e4m3{(uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3)};
}

// element i of an array whose type is known at run time
__device__ __forceinline__ float load_any(const void *p, uint64_t i, uint32_t type)
{
    if (type == ECC_F32)
        return static_cast<const float *>(p)[i];
    if (type == ECC_BF16)
        return to_f32(static_cast<const bf16 *>(p)[i]);
    return to_f32(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, uint64_t i, uint32_t type, float v)
{
    if (type == ECC_F32)
        static_cast<float *>(p)[i] = v;
    else if (type == ECC_BF16)
        static_cast<bf16 *>(p)[i] = from_f32<bf16>(v);
    else if (type == ECC_F16)
        static_cast<__half *>(p)[i] = from_f32<__half>(v);
    else
        static_cast<e4m3 *>(p)[i] = from_f32<e4m3>(v);
}

// two float32 operations in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)),
          "l"(reinterpret_cast<const unsigned long long &>(c)));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 16 bytes as 16 / sizeof(T) float32 values, in pairs
template <typename T> __device__ __forceinline__ void unpack2(const uint4 &v, float2 *f);
template <> __device__ __forceinline__ void unpack2<float>(const uint4 &v, float2 *f)
{
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <> __device__ __forceinline__ void unpack2<bf16>(const uint4 &v, float2 *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
template <> __device__ __forceinline__ void unpack2<__half>(const uint4 &v, float2 *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
}
// and back, rounded
template <typename T> __device__ __forceinline__ uint4 pack2(const float2 *f);
template <> __device__ __forceinline__ uint4 pack2<float>(const float2 *f)
{
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
}
template <> __device__ __forceinline__ uint4 pack2<bf16>(const float2 *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 pack2<__half>(const float2 *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 b = __floats2half2_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 of the 32 bytes of a and b, from byte off (below 16) on.  BRANCH: by a
// branch on the word, which a warp mostly takes as one, in place of selects.
// (Layer norm of 16384 x 4097 bf16 behind loads from HBM: 98 us with the
// branch, 112 with selects; its gradient, from shared memory: 204 and 194.)
template <bool BRANCH> __device__ __forceinline__ uint4 shift16(const uint4 &a, const uint4 &b, uint32_t off)
{
    const uint32_t s = (off & 3) * 8;
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    auto from = [&](const int k) {
        return make_uint4(__funnelshift_r(w[k], w[k + 1], s), __funnelshift_r(w[k + 1], w[k + 2], s),
                          __funnelshift_r(w[k + 2], w[k + 3], s), __funnelshift_r(w[k + 3], w[k + 4], s));
    };
    if constexpr (BRANCH) {
        switch (off >> 2) {
        case 0: return from(0);
        case 1: return from(1);
        case 2: return from(2);
        default: return from(3);
        }
    }
    if (off & 8) {
#pragma unroll
        for (int k = 0; k < 6; ++k)
            w[k] = w[k + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int k = 0; k < 5; ++k)
            w[k] = w[k + 1];
    }
    return from(0);
}

// 16 bytes at p, on any boundary of an element: the two aligned vectors around
// them, shifted together.  Only vectors that lie inside [begin, end), the
// bytes of the whole array, are read; where one does not, single elements.
template <typename T>
__device__ __forceinline__ uint4 load_anywhere(const T *p, const void *begin, const void *end)
{
    const uintptr_t at = (uintptr_t)p, low = at & ~(uintptr_t)15;
    const uint32_t off = (uint32_t)(at - low);
    if (off == 0)
        return *reinterpret_cast<const uint4 *>(p);
    if (low < (uintptr_t)begin || low + 32 > (uintptr_t)end) {
        struct alignas(16) {
            T v[16 / sizeof(T)];
        } t;
#pragma unroll
        for (int k = 0; k < (int)(16 / sizeof(T)); ++k)
            t.v[k] = p[k];
        return *reinterpret_cast<const uint4 *>(&t);
    }
    return shift16<true>(*reinterpret_cast<const uint4 *>(low), *reinterpret_cast<const uint4 *>(low + 16), off);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A kernel that a call launches behind another of its own may start before
// that one has ended (launch_behind): it waits here before it touches
// anything; the one before says early that it may start.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_behind(void (*f)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, args...);
}

} // namespace ecc
