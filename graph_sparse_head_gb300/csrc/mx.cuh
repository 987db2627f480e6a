// Matrices in microscaled 4-bit floating point: rows of E2M1 values in blocks of
// 32 along the row, each block with a power of two for its scale (E8M0 byte, 2^(byte - 127)).
//
//   2^e = the least power of two, e >= -127, with max|block| <= 6 2^e;  code = value / 2^e to the nearest of
//   0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives (ties to the even code)
//
// Nothing is clipped. (The largest power of two below max|block| / 4 for the scale would clip values above 6.)
// Codes: two a byte, the lower column in the low half, ceil(width / 32) * 16 bytes a row, zeros past the width.
// Scales: tiles of 128 rows by 4 blocks (512 bytes), the tiles of a row block side by side; byte of row r (of 128) and
// block k (of 4) at 16 (r % 32) + 4 (r / 32) + k, zeros past the rows and blocks: a tile goes to tensor memory as it is.
#pragma once

#include <cuda_fp4.h>

#include "pmha_internal.h"

namespace pmha {

struct Mx {
    const uint8_t *codes, *scale;
};
inline int64_t mx_blocks(int64_t width) { return (width + 31) / 32; }
inline int64_t mx_pitch(int64_t width) { return mx_blocks(width) * 16; }
inline size_t mx_code_bytes(int64_t rows, int64_t width) { return (size_t)rows * (size_t)mx_pitch(width); }
inline size_t mx_scale_bytes(int64_t rows, int64_t width)
{
    return (size_t)((rows + 127) / 128) * (size_t)((mx_blocks(width) + 3) / 4) * 512;
}

// Tensor-core products (mx_tc.cu). K: width of the rows of both operands.
struct MxLinear {
    Mx x, w;  // (M, K), (N, K)
    const void *bias, *residual;
    void *out;  // (M, N) bf16
    int64_t M, N, K;
};
pmha_status mx_tc_linear(const MxLinear &a, const char *stage, cudaStream_t s);
struct MxGated {
    Mx x, wg, wu;  // (M, K), (F, K), (F, K)
    const void *bg, *bu;
    uint8_t *h_codes, *h_scale;  // (M, F) in 4 bits
    int64_t M, F, K;
    pmha_act act;
};
pmha_status mx_tc_gated(const MxGated &a, cudaStream_t s);

#ifdef __CUDACC__
namespace {

// The scale byte of a block from the bits of its largest magnitude (compared as integers); 255 (NaN) for infinities and NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t most)
{
    const int e = (int)(most >> 23);
    const int b = e - ((most & 0x7fffffu) <= 0x400000u ? 2 : 1);  // 6 2^e = 1.5 2^(e + 2)
    return e >= 255 ? 255u : (uint32_t)max(b, 0);
}
// 2^(127 - byte), for bytes up to 253; 0 for 255 (of a block whose scale is NaN any code will do)
__device__ __forceinline__ float mx_inverse(uint32_t byte) { return __uint_as_float((uint32_t)max(254 - (int)byte, 0) << 23); }
// 2^(byte - 127), NaN for 255
__device__ __forceinline__ float mx_scale_value(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7fc00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x400000u);
}
// Two values, already times the inverse scale, as a byte
__device__ __forceinline__ uint32_t mx_byte(float low, float high)
{
    return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(low, high), __NV_E2M1, cudaRoundNearest);
}
// Eight values as codes, the first in the lowest half byte
__device__ __forceinline__ uint32_t mx_word(const float *f)
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace
#endif

}  // namespace pmha
