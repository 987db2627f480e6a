// Two float32 values in a register pair, one instruction for both (fma, mul and add .f32x2).
#pragma once

#include <stdint.h>

namespace pmha {
namespace {

struct Pair {
    uint64_t v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
// An array of values as pairs, and one value for all of them
template <int N>
struct Values {
    Pair p[N / 2];
    __device__ __forceinline__ Values() {}
    __device__ __forceinline__ explicit Values(const float (&f)[N])
    {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i] = Pair(f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void get(float (&f)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i].get(f[2 * i], f[2 * i + 1]);
    }
    // sum of a[i] b[i]
    static __device__ __forceinline__ float dot(const Values &a, const Values &b)
    {
        Pair s = mul2(a.p[0], b.p[0]);
#pragma unroll
        for (int i = 1; i < N / 2; ++i) s = fma2(a.p[i], b.p[i], s);
        float x, y;
        s.get(x, y);
        return x + y;
    }
};
template <int N>
__device__ __forceinline__ Values<N> times(const Values<N> &a, const Values<N> &b)
{
    Values<N> d;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) d.p[i] = mul2(a.p[i], b.p[i]);
    return d;
}
template <int N>
__device__ __forceinline__ Values<N> times(const Values<N> &a, float b)
{
    Values<N> d;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) d.p[i] = mul2(a.p[i], Pair(b, b));
    return d;
}
// a b + c
template <int N>
__device__ __forceinline__ Values<N> times_plus(const Values<N> &a, const Values<N> &b, const Values<N> &c)
{
    Values<N> d;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) d.p[i] = fma2(a.p[i], b.p[i], c.p[i]);
    return d;
}
template <int N>
__device__ __forceinline__ Values<N> times_plus(const Values<N> &a, float b, const Values<N> &c)
{
    Values<N> d;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) d.p[i] = fma2(a.p[i], Pair(b, b), c.p[i]);
    return d;
}

}  // namespace
}  // namespace pmha
