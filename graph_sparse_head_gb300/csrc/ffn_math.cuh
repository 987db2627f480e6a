// The gate's activation and its derivative, shared by the feed-forward
// kernels. `fast` forms serve the bf16 block, whose hidden values are rounded
// to 8 bits of mantissa (2^-9 relative) right after; float32 blocks take the
// library's expf, erff and division.
#pragma once

#include <math.h>

#include "pmha_internal.h"

namespace pmha {
namespace {

// Two float32 values in one 64-bit register: one instruction for both on this
// architecture's packed adders and multipliers.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ uint32_t to_bf16x2(F2 x)
{
    float a, b;
    split(x, a, b);
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the larger, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// 1 / a and 1 / b from one reciprocal of their product, for 1 <= a, b <= 2^59.
// The special-function unit gives 16 results a clock and SM, and the tensor
// pipe passes 128 x 64 hidden values in 770 clocks: four of them for a pair of
// values would take longer than the products, three do not.
__device__ __forceinline__ F2 rcp2(F2 d)
{
    float a, b;
    split(d, a, b);
    return f2(b, a) * f2(rcp(a * b));
}

template <int ACT>
struct Act;

template <>
struct Act<PMHA_ACT_SILU> {
    static __device__ __forceinline__ float exact(float g, float *slope)
    {
        const float p = 1.f / (1.f + expf(-g));
        *slope = p * (1.f + g * (1.f - p));
        return g * p;
    }
    static __device__ __forceinline__ float exact(float g) { return g / (1.f + expf(-g)); }
    // sigmoid(g) with g held at -40 (where g sigmoid(g) is -2e-16, and a NaN stays):
    // a product of two denominators is then at most 2^116
    static __device__ __forceinline__ F2 sigmoid(F2 &g)
    {
        float a, b;
        split(g, a, b);
        g = f2(max_nan(a, -40.f), max_nan(b, -40.f));
        split(g * f2(-1.44269504f), a, b);
        return rcp2(f2(fminf(ex2(a), 2.9e17f), fminf(ex2(b), 2.9e17f)) + f2(1.f));
    }
    static __device__ __forceinline__ F2 fast(F2 g)
    {
        const F2 p = sigmoid(g);
        return g * p;
    }
    static __device__ __forceinline__ F2 fast(F2 g, F2 *slope)
    {
        const F2 p = sigmoid(g), a = g * p;
        *slope = fma2(a, fma2(p, f2(-1.f), f2(1.f)), p);
        return a;
    }
};

template <>
struct Act<PMHA_ACT_GELU> {
    static __device__ __forceinline__ float exact(float g, float *slope)
    {
        const float p = 0.5f * erfcf(-0.70710678f * g);
        *slope = fmaf(g, 0.39894228f * expf(-0.5f * g * g), p);
        return g * p;
    }
    static __device__ __forceinline__ float exact(float g) { return g * (0.5f * erfcf(-0.70710678f * g)); }
    // Phi(g), from Phi(-|g|) = erfc(z) / 2, z = |g| / sqrt(2), by the rational form 7.1.26
    // of Abramowitz and Stegun (error below 1.5e-7): a polynomial in t = 1 / (1 + p z)
    // times e^(-z^2), which also gives the density that the slope needs.
    static __device__ __forceinline__ F2 phi(F2 g, F2 *e)
    {
        float a, b;
        split(g, a, b);
        // past |g| = 64 the exponential is 0 whatever t is
        const F2 t = rcp2(fma2(f2(fminf(fabsf(a), 64.f), fminf(fabsf(b), 64.f)), f2(0.3275911f * 0.70710678f), f2(1.f)));
        float u, v;
        split(g * g * f2(-0.72134752f), u, v);
        *e = f2(ex2(u), ex2(v));
        F2 q = fma2(t, f2(0.5f * 1.061405429f), f2(-0.5f * 1.453152027f));
        q = fma2(t, q, f2(0.5f * 1.421413741f));
        q = fma2(t, q, f2(-0.5f * 0.284496736f));
        q = fma2(t, q, f2(0.5f * 0.254829592f));
        q = q * t * *e;
        const F2 r = fma2(q, f2(-1.f), f2(1.f));
        float q0, q1, r0, r1;
        split(q, q0, q1);
        split(r, r0, r1);
        return f2(a < 0.f ? q0 : r0, b < 0.f ? q1 : r1);
    }
    static __device__ __forceinline__ F2 fast(F2 g)
    {
        F2 e;
        return g * phi(g, &e);
    }
    static __device__ __forceinline__ F2 fast(F2 g, F2 *slope)
    {
        F2 e;
        const F2 p = phi(g, &e);
        *slope = fma2(g * f2(0.39894228f), e, p);
        return g * p;
    }
};

}  // namespace
}  // namespace pmha
