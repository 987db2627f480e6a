// The gate's activation and its derivative, shared by the feed-forward
// kernels. `hidden` and `fast` serve the bf16 block, whose hidden values are rounded
// to 8 bits of mantissa (2^-9 relative) right after; float32 blocks take the
// library's expf, erff and division.
#pragma once

#include <math.h>

#include "pmha_internal.h"

namespace pmha {
namespace {

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

// The fast forms take the gate and the other factor times constants (kGate,
// kUp) that the caller folds into scales and biases: with the gate times
// -log2(e) the exponential needs no product of its own, and -ln(2) on the other
// side undoes it: two special-function results and seven other instructions a
// value. Packed float32 pairs and one reciprocal for two values were measured
// slower (register moves: 15 instructions a value).
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
    static constexpr float kGate = -1.44269504f, kUp = -0.69314718f;
    // g sigmoid(g) u; a gate far below 0 gives 1 / infinity = 0, also where gate times up would overflow
    static __device__ __forceinline__ float hidden(float gate, float up)
    {
        return gate * rcp(1.f + ex2(gate)) * up;
    }
    // act(g) and its slope, from the plain gate
    static __device__ __forceinline__ float fast(float g, float *slope)
    {
        const float p = rcp(1.f + ex2(kGate * g)), a = g * p;
        *slope = fmaf(a, 1.f - p, p);
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
    static constexpr float kGate = 1.f, kUp = 1.f;
    // Phi(-z) for z = min(|g|, 64) (0 from 14 on), by the rational form 7.1.26 of Abramowitz
    // and Stegun for erfc(z / sqrt(2)) (error below 1.5e-7; relative to the tail 0.16 % at z = 5, where it is 3e-7, and
    // 2 % at 10): a polynomial in
    // t = 1 / (1 + p z) times e = exp(-g^2 / 2), which the slope needs as well.
    static __device__ __forceinline__ float lower(float g, float z, float *e)
    {
        const float t = rcp(fmaf(z, 0.3275911f * 0.70710678f, 1.f));
        *e = ex2(g * g * -0.72134752f);
        float q = fmaf(t, 0.5f * 1.061405429f, -0.5f * 1.453152027f);
        q = fmaf(t, q, 0.5f * 1.421413741f);
        q = fmaf(t, q, -0.5f * 0.284496736f);
        q = fmaf(t, q, 0.5f * 0.254829592f);
        return q * t * *e;
    }
    // g Phi(g) = max(g, 0) - |g| Phi(-|g|)
    static __device__ __forceinline__ float hidden(float gate, float up)
    {
        float e;
        const float z = fminf(fabsf(gate), 64.f);
        return fmaf(-z, lower(gate, z, &e), fmaxf(gate, 0.f)) * up;
    }
    static __device__ __forceinline__ float fast(float g, float *slope)
    {
        float e;
        const float z = fminf(fabsf(g), 64.f), q = lower(g, z, &e);
        *slope = fmaf(g * 0.39894228f, e, 0.5f + copysignf(0.5f - q, g));
        return fmaf(-z, q, fmaxf(g, 0.f));
    }
};

}  // namespace
}  // namespace pmha
