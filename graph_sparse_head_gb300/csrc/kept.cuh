// Tensors kept in 8 bits between the forward and the backward pass: a row of
// `width` values as int8 codes with a bfloat16 scale for every 32 of them.
//
//   scale = max|group| / 127 rounded up to bfloat16, at least 2^-100;  code = v / scale to the nearest integer
//   v ~ code scale, off by half a scale: 1/254 of the group's largest magnitude (and the 2^-7 by which it was rounded up)
//
// Integers rather than E4M3: a group of normally distributed values has its
// largest near 2.5 sigma, a code is then off by 0.006 sigma (root mean square),
// an E4M3 value by 0.025. Codes are those of exact arithmetic, ties to even.
#pragma once

#include "rows.cuh"

namespace pmha {
namespace {

constexpr int kGroup = 32;
constexpr float kKeptLeast = 7.88860905e-31f;  // 2^-100

struct Kept {
    const int8_t *codes;
    const __nv_bfloat16 *scale;
};
struct KeptOut {
    int8_t *codes;
    __nv_bfloat16 *scale;
};

// The scale of a group from the bits of its largest magnitude (compared as integers, infinities and NaN come last).
__device__ __forceinline__ float kept_scale(uint32_t most)
{
    if (most >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    const float up = __fdiv_ru(__uint_as_float(most), 127.f);
    const uint32_t b = (__float_as_uint(up) + 0xffffu) & 0xffff0000u;  // up again: that of the exact quotient
    return fmaxf(__uint_as_float(b), kKeptLeast);
}
// v / scale to the nearest integer, in the low byte. A bfloat16 v and scale: the quotient is at least 2^-10 away from a
// half unless it is one, and a product with the reciprocal is within 2^-17 of it, so that rounding it to a grid of 2^-11
// first gives back the halves. A float32 v: the rounded quotient is a half only if the exact one is (the half times the
// scale has 16 bits, v is then at least its last bit away).
template <typename T>
__device__ __forceinline__ uint32_t kept_code(float v, float scale, float inv)
{
    float y;
    if constexpr (sizeof(T) == 2) y = __fsub_rn(__fmaf_rn(v, inv, 6144.f), 6144.f);
    else y = __fdiv_rn(v, scale);
    return __float_as_uint(__fadd_rn(y, 12582912.f)) & 0xffu;  // 1.5 * 2^23
}

// Keeps VEC values at column c of a row whose group's other values lie in the neighbouring lanes; every lane of the warp
// comes here, those past the width with zeros and in == false.
template <typename T, int VEC>
__device__ __forceinline__ void keep(const KeptOut &k, long long row, int c, int width, bool in, const T (&v)[VEC])
{
    constexpr int kLanes = kGroup / VEC;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) most = max(most, __float_as_uint(to_f<T>(v[i])) & 0x7fffffffu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
    const float scale = kept_scale(most);
    const bool fine = most < 0x7f800000u;
    const float inv = __fdiv_rn(1.f, scale);
    alignas(8) uint8_t b[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) b[i] = fine ? (uint8_t)kept_code<T>(to_f<T>(v[i]), scale, inv) : (uint8_t)0;
    if (!in) return;
    *reinterpret_cast<typename Bytes<VEC>::type *>(k.codes + row * width + c) = *reinterpret_cast<typename Bytes<VEC>::type *>(b);
    if (c % kGroup == 0) k.scale[row * ((width + kGroup - 1) / kGroup) + c / kGroup] = __float2bfloat16_rn(scale);
}
// VEC kept values, in float32
template <int VEC>
__device__ __forceinline__ void unkeep(const typename Bytes<VEC>::type &codes, float scale, float (&v)[VEC])
{
    alignas(8) int8_t b[VEC];
    *reinterpret_cast<typename Bytes<VEC>::type *>(b) = codes;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (float)b[i] * scale;
}
template <int VEC>
__device__ __forceinline__ void load_kept(const Kept &k, long long row, int c, int width, float (&v)[VEC])
{
    const typename Bytes<VEC>::type codes =
        *reinterpret_cast<const typename Bytes<VEC>::type *>(k.codes + row * width + c);
    unkeep<VEC>(codes, __bfloat162float(k.scale[row * ((width + kGroup - 1) / kGroup) + c / kGroup]), v);
}

}  // namespace
}  // namespace pmha
