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

#include "pair.cuh"
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

// The scale of a group from the bits of its largest magnitude (compared as integers, infinities and NaN come last): the
// least bfloat16 c with 127 c >= max (127 c is exact in float32), found beside an approximate quotient.
__device__ __forceinline__ float kept_scale(uint32_t bits)
{
    if (bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    const float most = __uint_as_float(bits);
    uint32_t c = (__float_as_uint(most * (1.f / 127.f)) + 0xffffu) & 0xffff0000u;
    if (c >= __float_as_uint(kKeptLeast)) {  // normal numbers, and their neighbours below
        if (127.f * __uint_as_float(c) < most) c += 0x10000u;
        else if (127.f * __uint_as_float(c - 0x10000u) >= most) c -= 0x10000u;
    }
    return fmaxf(__uint_as_float(c), kKeptLeast);
}
__device__ __forceinline__ float kept_inverse(float scale)  // within 2^-22
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(scale));
    return y;
}
// v / scale to the nearest integer, in the low byte, ties to even. A bfloat16 v and scale, two values at once: the quotient is
// at least 2^-10 away from a half unless it is one, and its product with the inverse is within 2^-15 of it, so that rounding it
// to a grid of 2^-11 first (6144 off: a multiple of the grid and of 256) gives back the halves. (Of a group with an infinity or
// a NaN any code will do: its scale is NaN.)
constexpr float kRound = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ void kept_code2(float v0, float v1, float inv, uint32_t &c0, uint32_t &c1)
{
    float a, b;
    add2(fma2(Pair(v0, v1), Pair(inv, inv), Pair(6144.f, 6144.f)), Pair(kRound, kRound)).get(a, b);
    c0 = __float_as_uint(a), c1 = __float_as_uint(b);
}
// A float32 v: the remainder of the product's nearest integer q is exact (both v and q scale are multiples of its last bit)
// and says whether the neighbour is nearer, or as near and even.
__device__ __forceinline__ uint32_t kept_code(float v, float scale, float inv)
{
    const float m = __fmaf_rn(v, inv, kRound), q = __fsub_rn(m, kRound);
    const float e = __fmaf_rn(-q, scale, v), half = 0.5f * scale;
    const bool move = fabsf(e) > half || (fabsf(e) == half && (__float_as_uint(m) & 1u));
    return __float_as_uint(m) + (move ? (e > 0.f ? 1u : 0xffffffffu) : 0u);
}

// The codes of VEC values of a group whose others lie in the neighbouring lanes, in the low bytes, and the group's scale;
// every lane of the warp comes here, those without a value with zeros.
template <typename T, int VEC>
__device__ __forceinline__ float kept_codes(const Vals<T, VEC> &v, uint32_t (&w)[VEC])
{
    uint32_t most = most_bits<T, VEC>(v);
#pragma unroll
    for (int o = kGroup / VEC / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
    const float scale = kept_scale(most), inv = kept_inverse(scale);
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
        if constexpr (sizeof(T) == 2) {
            kept_code2(to_f<T>(v.v[i]), to_f<T>(v.v[i + 1]), inv, w[i], w[i + 1]);
        } else {
            w[i] = kept_code(v.v[i], scale, inv);
            w[i + 1] = kept_code(v.v[i + 1], scale, inv);
        }
    }
    return scale;
}
// Keeps them at these places; `first`: the group's first lane, which writes the scale.
template <typename T, int VEC>
__device__ __forceinline__ void keep(const KeptOut &at, bool first, bool in, const Vals<T, VEC> &v)
{
    uint32_t w[VEC];
    const float scale = kept_codes<T, VEC>(v, w);
    if (!in) return;
    *reinterpret_cast<typename Bytes<VEC>::type *>(at.codes) = low_bytes<VEC>(w);
    if (first) *at.scale = __float2bfloat16_rn(scale);
}
// VEC kept values, in float32: a byte b ^ 0x80 in the last place of 2^23 is 2^23 + 128 + b
template <int VEC>
__device__ __forceinline__ void unkeep(const typename Bytes<VEC>::type &codes, float scale, float (&v)[VEC])
{
    uint32_t w[(VEC + 3) / 4] = {};
    *reinterpret_cast<typename Bytes<VEC>::type *>(w) = codes;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const uint32_t b = __byte_perm(w[i / 4] ^ 0x80808080u, 0x4b000000u, 0x7540 + (i & 3));
        v[i] = __uint_as_float(b);
    }
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            mul2(add2(Pair(v[i], v[i + 1]), Pair(-8388736.f, -8388736.f)), Pair(scale, scale)).get(v[i], v[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __fsub_rn(v[i], 8388736.f) * scale;
    }
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
