// The gate's activation and its derivative, shared by the feed-forward
// kernels. `hidden` and `fast` serve the bf16 block, whose hidden values are rounded
// to 8 bits of mantissa (2^-9 relative) right after; float32 blocks take the
// library's expf, erff and division.
#pragma once

#include <math.h>

#include "pair.cuh"
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
// value. In the bf16 kernels packed float32 pairs and one reciprocal for two values were
// measured slower (register moves: 15 instructions a value); the 4-bit kernel, whose accumulators come from tensor memory
// in register pairs, takes hidden2.
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
    static __device__ __forceinline__ Pair hidden2(Pair gate, Pair up)
    {
        float g0, g1, d0, d1;
        gate.get(g0, g1);
        add2(Pair(ex2(g0), ex2(g1)), Pair(1.f, 1.f)).get(d0, d1);
        return mul2(mul2(gate, Pair(rcp(d0), rcp(d1))), up);
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
    static constexpr float kP = 0.3275911f * 0.70710678f, kE = -0.72134752f;  // of z in t; -log2(e) / 2
    static constexpr float kA1 = 0.5f * 0.254829592f, kA2 = -0.5f * 0.284496736f, kA3 = 0.5f * 1.421413741f,
                           kA4 = -0.5f * 1.453152027f, kA5 = 0.5f * 1.061405429f;
    static __device__ __forceinline__ float lower(float g, float z, float *e)
    {
        const float t = rcp(fmaf(z, kP, 1.f));
        *e = ex2(g * g * kE);
        float q = fmaf(t, kA5, kA4);
        q = fmaf(t, q, kA3);
        q = fmaf(t, q, kA2);
        q = fmaf(t, q, kA1);
        return q * t * *e;
    }
    static __device__ __forceinline__ Pair lower2(Pair g, Pair z)
    {
        float t0, t1, e0, e1;
        fma2(z, Pair(kP, kP), Pair(1.f, 1.f)).get(t0, t1);
        const Pair t(rcp(t0), rcp(t1));
        mul2(mul2(g, g), Pair(kE, kE)).get(e0, e1);
        Pair q = fma2(t, Pair(kA5, kA5), Pair(kA4, kA4));
        q = fma2(t, q, Pair(kA3, kA3));
        q = fma2(t, q, Pair(kA2, kA2));
        q = fma2(t, q, Pair(kA1, kA1));
        return mul2(mul2(q, t), Pair(ex2(e0), ex2(e1)));
    }
    // g Phi(g) = max(g, 0) - |g| Phi(-|g|)
    static __device__ __forceinline__ float hidden(float gate, float up)
    {
        float e;
        const float z = fminf(fabsf(gate), 64.f);
        return fmaf(-z, lower(gate, z, &e), fmaxf(gate, 0.f)) * up;
    }
    static __device__ __forceinline__ Pair hidden2(Pair gate, Pair up)
    {
        float g0, g1;
        gate.get(g0, g1);
        const float z0 = fminf(fabsf(g0), 64.f), z1 = fminf(fabsf(g1), 64.f);
        return mul2(fma2(Pair(-z0, -z1), lower2(gate, Pair(z0, z1)), Pair(fmaxf(g0, 0.f), fmaxf(g1, 0.f))), up);
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
