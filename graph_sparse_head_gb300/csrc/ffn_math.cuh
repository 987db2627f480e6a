// The gate's activation and its derivative, shared by the feed-forward
// kernels. `fast` forms serve the bf16 block, whose hidden values are rounded
// to 8 bits of mantissa (2^-9 relative) right after; float32 blocks take the
// library's expf, erff and division.
#pragma once

#include <math.h>

#include "pmha_internal.h"

namespace pmha {
namespace {

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
    static __device__ __forceinline__ float sigmoid(float g)
    {
        // 2^(-g log2 e) overflows to infinity for g < -88, and the quotient is then 0
        return __fdividef(1.f, 1.f + exp2f_approx(-1.44269504f * g));
    }
    static __device__ __forceinline__ float fast(float g) { return g * sigmoid(g); }
    static __device__ __forceinline__ float fast(float g, float *slope)
    {
        const float p = sigmoid(g), a = g * p;
        *slope = fmaf(a, 1.f - p, p);
        return a;
    }
    static __device__ __forceinline__ float exp2f_approx(float x)
    {
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
        return y;
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
    // Phi(-|g|) = erfc(z) / 2, z = |g| / sqrt(2), by the rational form 7.1.26 of
    // Abramowitz and Stegun (error below 1.5e-7): polynomial in t = 1 / (1 + p z)
    // times e^(-z^2), which also gives the density the slope needs.
    static __device__ __forceinline__ float lower(float g, float *e)
    {
        const float z = fabsf(g) * 0.70710678f;
        const float t = __fdividef(1.f, fmaf(0.3275911f, z, 1.f));
        *e = Act<PMHA_ACT_SILU>::exp2f_approx(-0.72134752f * g * g);
        float q = fmaf(t, 1.061405429f, -1.453152027f);
        q = fmaf(t, q, 1.421413741f);
        q = fmaf(t, q, -0.284496736f);
        q = fmaf(t, q, 0.254829592f);
        return 0.5f * q * t * *e;
    }
    static __device__ __forceinline__ float fast(float g)
    {
        float e;
        const float q = lower(g, &e);
        return g * (g < 0.f ? q : 1.f - q);
    }
    static __device__ __forceinline__ float fast(float g, float *slope)
    {
        float e;
        const float q = lower(g, &e), p = g < 0.f ? q : 1.f - q;
        *slope = fmaf(g * 0.39894228f, e, p);
        return g * p;
    }
};

}  // namespace
}  // namespace pmha
