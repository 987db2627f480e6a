// What the kernels over token rows share (norm.cu, join.cu): vector loads and
// stores, the kernel shape of a width, the power of two that brings a large row
// into float32's range, sums over a block, pairs of floats.
#pragma once

#include <math.h>

#include "pmha_internal.h"

namespace pmha {
namespace {  // each translation unit keeps its own copy

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;
// A row whose squares' sum leaves float32 is taken again times the power of two
// that brings its largest magnitude into [2, 4) (exact but for values 2^-120 of
// it), with eps times its square: the norm does not change, and no sum of up to 2^24 squares
// overflows. A fixed factor would not do: 2^-64, taken before, left rows from 2^128 / sqrt(width) infinite.
constexpr float kMostSquares = 3.0e38f;
__device__ __forceinline__ float down_scale(float most)
{
    const uint32_t e = __float_as_uint(most) >> 23;  // exponent + 127
    return e >= 128 && e < 255 ? __uint_as_float((255 - e) << 23) : 1.f;  // 1 for infinities and NaN too
}

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC consecutive values as one load or store (16, 4 or 2 bytes), or as two of 16.
struct alignas(16) TwoPieces {
    uint4 a, b;
};
template <typename T, int VEC> struct Pack;
template <> struct Pack<float, 8> { using type = TwoPieces; };
template <> struct Pack<__nv_bfloat16, 16> { using type = TwoPieces; };
template <> struct Pack<float, 4> { using type = uint4; };
template <> struct Pack<float, 1> { using type = uint32_t; };
template <> struct Pack<__nv_bfloat16, 8> { using type = uint4; };
template <> struct Pack<__nv_bfloat16, 2> { using type = uint32_t; };
template <> struct Pack<__nv_bfloat16, 1> { using type = uint16_t; };
// VEC bytes
template <int VEC> struct Bytes;
template <> struct Bytes<16> { using type = uint4; };
template <> struct Bytes<8> { using type = uint2; };
template <> struct Bytes<4> { using type = uint32_t; };
template <> struct Bytes<2> { using type = uint16_t; };
template <> struct Bytes<1> { using type = uint8_t; };

template <typename T, int VEC>
__device__ __forceinline__ void load(const T *p, T (&v)[VEC])
{
    *reinterpret_cast<typename Pack<T, VEC>::type *>(v) = *reinterpret_cast<const typename Pack<T, VEC>::type *>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T *p, const T (&v)[VEC])
{
    *reinterpret_cast<typename Pack<T, VEC>::type *>(p) = *reinterpret_cast<const typename Pack<T, VEC>::type *>(v);
}
template <typename T, int VEC> struct alignas(alignof(typename Pack<T, VEC>::type)) Vals {
    T v[VEC];
};

// The bits, as float32, of the largest magnitude of some values; compared as integers, so that infinities and NaN come last.
template <typename T, int VEC>
__device__ __forceinline__ uint32_t most_bits(const Vals<T, VEC> &v)
{
    uint32_t most = 0;
    if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v.v);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) most = __vmaxu2(most, w[i] & 0x7fff7fffu);
        return max(most & 0xffff0000u, most << 16);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) most = max(most, __float_as_uint(to_f<T>(v.v[i])) & 0x7fffffffu);
        return most;
    }
}
// VEC consecutive values of a row that need not lie on a boundary: one by one, those past the row's end zeros (left alone).
// The same cache line serves a lane's values and its neighbours'.
template <typename T, int VEC, bool ALIGNED>
__device__ __forceinline__ void load_some(const T *p, int left, Vals<T, VEC> &v)
{
    if constexpr (ALIGNED) {
        load<T, VEC>(p, v.v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < left) v.v[i] = p[i];
    }
}

// The low bytes of VEC words
template <int VEC>
__device__ __forceinline__ typename Bytes<VEC>::type low_bytes(const uint32_t (&w)[VEC])
{
    auto four = [&](int i) {
        return __byte_perm(__byte_perm(w[i], w[i + 1], 0x0040), __byte_perm(w[i + 2], w[i + 3], 0x0040), 0x5410);
    };
    if constexpr (VEC == 4) return four(0);
    else if constexpr (VEC == 8) return make_uint2(four(0), four(4));
    else return make_uint4(four(0), four(4), four(8), four(12));
}

// An unevaluated sum hi + lo (about 46 bits).
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(Two a, Two b)
{
    const Two s = two_sum(a.hi, b.hi);
    return {s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo))};
}
__device__ __forceinline__ float block_sum(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sh[i];
    __syncthreads();
    return v;
}

__device__ __forceinline__ float block_max(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v = fmaxf(v, sh[i]);
    __syncthreads();
    return v;
}

// 16 bytes from global to shared memory, or zeros
__device__ __forceinline__ void copy16(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
// ---------------------------------------------------------------- host side
inline bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    if (!a || !b || !an || !bn) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + bn && y < x + an;
}
struct Span {
    const void *p;
    size_t n;
};
// Whether an output overlaps an input or another output.
template <int NI, int NO>
inline bool any_overlap(const Span (&in)[NI], const Span (&out)[NO])
{
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return true;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return true;
    }
    return false;
}
inline bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline size_t bytes_of(pmha_dtype dt) { return dt == PMHA_BF16 ? 2 : 4; }

inline pmha_status check_rows(const char *who, pmha_dtype dt, int64_t rows, int64_t width)
{
    if (dt != PMHA_F32 && dt != PMHA_BF16) {
        set_error("%s: dtype %d is neither PMHA_F32 nor PMHA_BF16", who, (int)dt);
        return PMHA_ERR_INVALID_ARG;
    }
    if (rows < 0 || width < 1 || width > ((int64_t)1 << 24) || rows > ((int64_t)1 << 31) - 1 ||
        rows * width > (int64_t)1 << 46) {
        set_error("%s: rows %lld must be 0 .. 2^31 - 1, width %lld 1 .. 2^24, and their product at most 2^46", who,
                  (long long)rows, (long long)width);
        return PMHA_ERR_INVALID_ARG;
    }
    return PMHA_OK;
}

// The kernel shape of a width: values a piece, pieces a lane, lanes a row; 0 lanes: one block a row.
struct Shape {
    int vec, nv, lpr;
};
inline Shape shape_of(pmha_dtype dt, int64_t width)
{
    const int v = dt == PMHA_BF16 ? 8 : 4;
    const int vec = width % v == 0 ? v : (dt == PMHA_BF16 && width % 2 == 0 ? 2 : 1);
    if (width > 1024) return {vec, 0, 0};
    const int64_t pieces = width / vec;
    if (vec == v) {
        if (pieces <= 8) return {vec, 1, 8};
        if (pieces <= 16) return {vec, 1, 16};
        if (pieces <= 32) return {vec, 1, 32};
        if (pieces <= 64) return {vec, 2, 32};
        if (pieces <= 128) return {vec, 4, 32};
        return {vec, 8, 32};
    }
    return pieces <= 256 / vec ? Shape{vec, 8 / vec, 32} : Shape{vec, 32 / vec, 32};
}

// F(type tag, vec, nv, lpr) for every shape that shape_of gives.
template <typename T, int V, int N, int L> struct Tag {
    using type = T;
    static constexpr int vec = V, nv = N, lpr = L;
};
template <typename F>
void dispatch(pmha_dtype dt, Shape s, F f)
{
    using B = __nv_bfloat16;
    if (dt == PMHA_BF16) {
        if (s.vec == 8) {
            if (s.lpr == 8) f(Tag<B, 8, 1, 8>());
            else if (s.lpr == 16) f(Tag<B, 8, 1, 16>());
            else if (s.nv == 1) f(Tag<B, 8, 1, 32>());
            else if (s.nv == 2) f(Tag<B, 8, 2, 32>());
            else f(Tag<B, 8, 4, 32>());
        } else if (s.vec == 2) {
            if (s.nv == 4) f(Tag<B, 2, 4, 32>());
            else f(Tag<B, 2, 16, 32>());
        } else {
            if (s.nv == 8) f(Tag<B, 1, 8, 32>());
            else f(Tag<B, 1, 32, 32>());
        }
    } else if (s.vec == 4) {
        if (s.lpr == 8) f(Tag<float, 4, 1, 8>());
        else if (s.lpr == 16) f(Tag<float, 4, 1, 16>());
        else if (s.nv == 1) f(Tag<float, 4, 1, 32>());
        else if (s.nv == 2) f(Tag<float, 4, 2, 32>());
        else if (s.nv == 4) f(Tag<float, 4, 4, 32>());
        else f(Tag<float, 4, 8, 32>());
    } else {
        if (s.nv == 8) f(Tag<float, 1, 8, 32>());
        else f(Tag<float, 1, 32, 32>());
    }
}
template <typename F>
void dispatch_wide(pmha_dtype dt, int vec, F f)
{
    using B = __nv_bfloat16;
    if (dt == PMHA_BF16) {
        if (vec == 8) f(Tag<B, 8, 1, 32>());
        else if (vec == 2) f(Tag<B, 2, 1, 32>());
        else f(Tag<B, 1, 1, 32>());
    } else if (vec == 4) f(Tag<float, 4, 1, 32>());
    else f(Tag<float, 1, 1, 32>());
}


}  // namespace
}  // namespace pmha
