// Root-mean-square norm of token rows, with the residual's addition before it
// and an optional output in 8 bits with a scale a row; and its backward pass.
//
//   s = round(x + residual)          (kept in the layer type; the norm is of the kept sum)
//   r = (mean(s^2) + eps)^(-1/2),    y = s r w
//   dx = r (a - s r^2 mean(a s)) + dsum with a = dy w,    dw = sum over rows of dy s r
//
// All of it is bound by memory: each row is read once into registers (widths
// up to 1024), by as many lanes of a warp as its 16-byte pieces need, so that
// narrow rows share a warp and the statistics are a few shuffles. Wider rows
// take a block each and read their row again from L1/L2 for the second pass.
// bf16 with a residual: 320,000 x 128 in 50.5 us, 6.5 TB/s (96 % of a copy). The
// 8-bit output is bound by its some 30 instructions a value: 64,000 x 128 in 17 us.
#include <cuda_fp8.h>

#include <algorithm>

#include "rows.cuh"

namespace pmha {
namespace {

constexpr float kScaleMin = 5.42101086e-20f;  // 2^-64
// The 8-bit output's statistics are pairs of floats, and the second float of 1 / (mean square) is a normal
// number up to 2^102: its rows are scaled from 2^96 on.
constexpr float kMostPairs = 7.9228163e28f;
// ---------------------------------------------------------------- pairs of floats
// An unevaluated sum hi + lo (about 46 bits), for the 8-bit output: a value
// next to a border of the E4M3 grid must fall where exact arithmetic puts it,
// and 32-bit sums and products would move about 5 values in a million.
__device__ __forceinline__ Two two_mul(float a, float b)
{
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a / b for normal b: an approximate quotient (some 22 bits) and its exact
// remainder's quotient; hi and lo may overlap in two bits.
__device__ __forceinline__ Two div(Two a, float b)
{
    const float r = rcp(b), q = __fmul_rn(a.hi, r);
    return {q, __fmul_rn(__fadd_rn(__fmaf_rn(-q, b, a.hi), a.lo), r)};
}
__device__ __forceinline__ Two mul(Two a, Two b)
{
    Two p = two_mul(a.hi, b.hi);
    p.lo = __fadd_rn(p.lo, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi)));
    return p;
}
// 1 / sqrt(m): one Newton step with its second-order term from the library's root
__device__ __forceinline__ Two inv_sqrt(Two m)
{
    const float y = rsqrtf(m.hi);
    const Two p = two_mul(y, y);
    float e = __fmaf_rn(-m.hi, p.hi, 1.f);
    e = __fsub_rn(e, __fmaf_rn(m.hi, p.lo, __fmul_rn(m.lo, p.hi)));
    return {y, __fmul_rn(y, __fmaf_rn(__fmul_rn(0.375f, e), e, __fmul_rn(0.5f, e)))};
}
struct NormArgs {
    Two inv_width;
    const void *x, *res, *w;
    void *sum, *out;
    uint8_t *q;
    float *scale;
    long long rows;
    int width;
    float eps;
};

// The row's scale and the factor r / scale of its 8-bit values.
struct Quant {
    float scale;
    Two c;
};
__device__ __forceinline__ Quant quant(Two ss, Two amax, Two inv_width, float eps)
{
    Two m = add(mul(ss, inv_width), Two{eps, 0.f});
    const float mh = __fadd_rn(m.hi, m.lo);
    m = {mh, __fsub_rn(m.lo, __fsub_rn(mh, m.hi))};
    const Two r = inv_sqrt(m);
    const Two s = mul(mul(amax, r), Two{1.f / 448.f, (float)(1.0 / 448.0 - (double)(1.f / 448.f))});
    Quant z;
    z.scale = __fadd_rn(s.hi, s.lo);
    if (z.scale < kScaleMin) z.scale = kScaleMin;  // a NaN stays
    if (!(ss.hi <= 3.4e38f)) z.scale = __int_as_float(0x7fffffff);
    z.c = div(r, z.scale);
    return z;
}
// The product of two bf16 values, and a bf16 value's square, have at most 16
// significant bits: one float holds them (EXACT), which leaves some 30
// instructions a value instead of 120.
template <bool EXACT>
__device__ __forceinline__ Two product(float a, float b)
{
    if constexpr (EXACT) return {__fmul_rn(a, b), 0.f};
    else return two_mul(a, b);
}
// f w c, cut to a float whose last bit is set where anything was cut ("to
// odd"): a later rounding to fewer bits then falls as that of the exact product.
template <bool EXACT>
__device__ __forceinline__ float quant_value(float f, float w, Two c)
{
    const Two p = product<EXACT>(f, w);
    const float e = EXACT ? __fmul_rn(p.hi, c.lo) : __fmaf_rn(p.hi, c.lo, __fmul_rn(p.lo, c.hi));
    const float s = __fmaf_rz(p.hi, c.hi, e);
    const float cut = __fadd_rn(__fmaf_rn(p.hi, c.hi, -s), e);
    return __int_as_float(__float_as_int(s) | (cut != 0.f ? 1 : 0));
}
template <bool EXACT>
__device__ __forceinline__ void take_max(Two &m, Two o)
{
    if constexpr (EXACT) m.hi = fmaxf(m.hi, o.hi);
    else if (o.hi > m.hi || (o.hi == m.hi && o.lo > m.lo)) m = o;
}
template <bool EXACT>
__device__ __forceinline__ Two abs_mul(float f, float w)
{
    Two p = product<EXACT>(f, w);
    if constexpr (EXACT) p.hi = fabsf(p.hi);
    else if (p.hi < 0.f) p = {-p.hi, -p.lo};
    return p;
}
template <bool EXACT>
__device__ __forceinline__ void square_into(Two &ss, float f)
{
    const Two p = product<EXACT>(f, f);
    const Two t = two_sum(ss.hi, p.hi);
    if constexpr (EXACT) ss = {t.hi, __fadd_rn(ss.lo, t.lo)};
    else ss = {t.hi, __fadd_rn(ss.lo, __fadd_rn(t.lo, p.lo))};
}
__device__ __forceinline__ uint8_t to_e4m3(float v) { return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }

// ---------------------------------------------------------------- forward
// LPR lanes share a row; lane l holds pieces l, l + LPR, ... of VEC values, NV of them.
template <typename T, int VEC, int NV, int LPR, bool Q8>
__global__ void __launch_bounds__(kThreads) k_rms_norm(NormArgs a)
{
    constexpr int kRows = 32 / LPR;  // rows of a warp
    constexpr bool kExact = sizeof(T) == 2;
    const int lane = threadIdx.x & 31, l = lane % LPR;
    const long long row = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + lane / LPR;
    const bool live = row < a.rows;
    const T *x = (const T *)a.x, *res = (const T *)a.res, *w = (const T *)a.w;
    const long long base = row * a.width;
    Vals<T, VEC> v[NV], e[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + l) * VEC;
        if (live && c < a.width) {
            load<T, VEC>(x + base + c, v[j].v);
            if (res) load<T, VEC>(res + base + c, e[j].v);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j].v[i] = e[j].v[i] = from_f<T>(0.f);
        }
    }
    Vals<T, VEC> wv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + l) * VEC;
        if (w && c < a.width) load<T, VEC>(w + c, wv[j].v);
        else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) wv[j].v[i] = from_f<T>(1.f);
        }
    }
    if (res) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j].v[i] = from_f<T>(__fadd_rn(to_f<T>(v[j].v[i]), to_f<T>(e[j].v[i])));
    }
    if (a.sum) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + l) * VEC;
            if (live && c < a.width) store<T, VEC>((T *)a.sum + base + c, v[j].v);
        }
    }
    float sc = 1.f;  // v holds the row times this
    auto scale_rows = [&](bool over) {
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) most = fmaxf(most, fabsf(to_f<T>(v[j].v[i])));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
        const float by = over ? down_scale(most) : 1.f;
        sc *= by;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j].v[i] = from_f<T>(to_f<T>(v[j].v[i]) * by);
    };
    if (a.out) {
        auto squares = [&]() {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float f = to_f<T>(v[j].v[i]);
                    ss = fmaf(f, f, ss);
                }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            return ss;
        };
        float ss = squares();
        if (__any_sync(kFull, ss > kMostSquares)) {
            scale_rows(ss > kMostSquares);
            ss = squares();
        }
        const float r = rsqrtf(ss / (float)a.width + a.eps * sc * sc);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + l) * VEC;
            Vals<T, VEC> y;
#pragma unroll
            for (int i = 0; i < VEC; ++i) y.v[i] = from_f<T>(to_f<T>(v[j].v[i]) * r * to_f<T>(wv[j].v[i]));
            if (live && c < a.width) store<T, VEC>((T *)a.out + base + c, y.v);
        }
    }
    if constexpr (Q8) {
        Two ss, am;
        auto stats = [&]() {
            ss = am = Two{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float f = to_f<T>(v[j].v[i]);
                    square_into<kExact>(ss, f);
                    take_max<kExact>(am, abs_mul<kExact>(f, to_f<T>(wv[j].v[i])));
                }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                ss = add(ss, Two{__shfl_xor_sync(kFull, ss.hi, o), __shfl_xor_sync(kFull, ss.lo, o)});
                take_max<kExact>(am, Two{__shfl_xor_sync(kFull, am.hi, o), __shfl_xor_sync(kFull, am.lo, o)});
            }
        };
        stats();
        const bool over = !(ss.hi <= kMostPairs && am.hi <= kMostSquares);  // squares, or products with the weight
        if (__any_sync(kFull, over)) {
            scale_rows(over);
            stats();
        }
        const Quant z = quant(ss, am, a.inv_width, a.eps * sc * sc);
        if (live && l == 0) a.scale[row] = z.scale;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + l) * VEC;
            if (!(live && c < a.width)) continue;
            alignas(8) uint8_t b[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                b[i] = to_e4m3(quant_value<kExact>(to_f<T>(v[j].v[i]), to_f<T>(wv[j].v[i]), z.c));
            *reinterpret_cast<typename Bytes<VEC>::type *>(a.q + base + c) =
                *reinterpret_cast<typename Bytes<VEC>::type *>(b);
        }
    }
}

// Rows of more than 1024 values: one block a row.
template <typename T, int VEC, bool Q8>
__global__ void __launch_bounds__(kThreads) k_rms_norm_wide(NormArgs a)
{
    __shared__ float sh[kThreads / 32];
    __shared__ Two sh2[kThreads / 32], shm[kThreads / 32];
    constexpr bool kExact = sizeof(T) == 2;
    const long long row = blockIdx.x, base = row * a.width;
    const T *x = (const T *)a.x, *res = (const T *)a.res, *w = (const T *)a.w;
    auto kept = [&](int c, Vals<T, VEC> &v) {
        load<T, VEC>(x + base + c, v.v);
        if (res) {
            Vals<T, VEC> e;
            load<T, VEC>(res + base + c, e.v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v.v[i] = from_f<T>(__fadd_rn(to_f<T>(v.v[i]), to_f<T>(e.v[i])));
        }
    };
    auto weight = [&](int c, Vals<T, VEC> &v) {
        if (w) load<T, VEC>(w + c, v.v);
        else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v.v[i] = from_f<T>(1.f);
        }
    };
    float ss, sc = 1.f;
    Two s2, am;
    auto stats = [&](bool keep) {
        ss = 0.f;
        s2 = am = Two{0.f, 0.f};
        for (int c = threadIdx.x * VEC; c < a.width; c += kThreads * VEC) {
            Vals<T, VEC> v, wv;
            kept(c, v);
            if (keep) store<T, VEC>((T *)a.sum + base + c, v.v);
            if constexpr (Q8) weight(c, wv);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float f = to_f<T>(v.v[i]) * sc;
                ss = fmaf(f, f, ss);
                if constexpr (Q8) {
                    square_into<kExact>(s2, f);
                    take_max<kExact>(am, abs_mul<kExact>(f, to_f<T>(wv.v[i])));
                }
            }
        }
        ss = block_sum(ss, sh);
        if constexpr (Q8) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                s2 = add(s2, Two{__shfl_xor_sync(kFull, s2.hi, o), __shfl_xor_sync(kFull, s2.lo, o)});
                take_max<kExact>(am, Two{__shfl_xor_sync(kFull, am.hi, o), __shfl_xor_sync(kFull, am.lo, o)});
            }
            if ((threadIdx.x & 31) == 0) {
                sh2[threadIdx.x >> 5] = s2;
                shm[threadIdx.x >> 5] = am;
            }
            __syncthreads();
            s2 = am = Two{0.f, 0.f};
            for (int i = 0; i < kThreads / 32; ++i) {
                s2 = add(s2, sh2[i]);
                take_max<kExact>(am, shm[i]);
            }
            __syncthreads();  // read before a second pass writes there
        }
    };
    stats(a.sum != nullptr);
    if (!(ss <= (Q8 ? kMostPairs : kMostSquares) && am.hi <= kMostSquares)) {  // the same in every thread
        float most = 0.f;
        for (int c = threadIdx.x * VEC; c < a.width; c += kThreads * VEC) {
            Vals<T, VEC> v;
            kept(c, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) most = fmaxf(most, fabsf(to_f<T>(v.v[i])));
        }
        sc = down_scale(block_max(most, sh));
        stats(false);
    }
    Quant z;
    if constexpr (Q8) {
        z = quant(s2, am, a.inv_width, a.eps * sc * sc);
        if (threadIdx.x == 0) a.scale[row] = z.scale;
    }
    const float r = rsqrtf(ss / (float)a.width + a.eps * sc * sc);
    for (int c = threadIdx.x * VEC; c < a.width; c += kThreads * VEC) {
        Vals<T, VEC> v, wv, y;
        kept(c, v);
        weight(c, wv);
        if (a.out) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) y.v[i] = from_f<T>(to_f<T>(v.v[i]) * sc * r * to_f<T>(wv.v[i]));
            store<T, VEC>((T *)a.out + base + c, y.v);
        }
        if constexpr (Q8) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                a.q[base + c + i] = to_e4m3(quant_value<kExact>(to_f<T>(v.v[i]) * sc, to_f<T>(wv.v[i]), z.c));
        }
    }
}

// ---------------------------------------------------------------- backward
struct NormBwdArgs {
    const void *x, *w, *dy, *ds;
    void *dx;
    float *part;  // (grid, width) partial weight gradients, or null
    long long rows;
    int width;
    float eps;
};

template <typename T, int VEC, int NV>
constexpr int kRingOf = VEC * sizeof(T) == 16 && NV <= 2 ? 4 / NV : 0;

// Steps of a block: so many terms of the weight gradient at most are added in
// float32, one after the other. Where there are more rows, there are more
// blocks, whose partial rows are added as pairs of floats: the error does not
// grow with the rows. 1,280,000 x 256: 395 us, with four blocks a SM and 263
// steps each 476 (three are resident, the rest ran behind them alone). Sums put
// aside every 128 steps inside one loop over all rows: 507, for the barriers and a slower loop.
constexpr int kSteps = 128;

// A warp walks its rows and keeps its columns' weight gradient in registers; a
// block sums its warps' through shared memory and writes one partial row.
// 1,280,000 x 256 bf16 with dsum: 395 us, 6.6 TB/s.
template <typename T, int VEC, int NV, int LPR>
__global__ void __launch_bounds__(kThreads) k_rms_norm_bwd(NormBwdArgs a)
{
    extern __shared__ float shw[];  // width values
    constexpr int kRows = 32 / LPR;
    const int lane = threadIdx.x & 31, l = lane % LPR, warp = threadIdx.x >> 5;
    const T *x = (const T *)a.x, *w = (const T *)a.w, *dy = (const T *)a.dy, *ds = (const T *)a.ds;
    float dw[NV][VEC], wf[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + l) * VEC;
        Vals<T, VEC> wv;
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv.v[i] = from_f<T>(1.f);
        if (w && c < a.width) load<T, VEC>(w + c, wv.v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            dw[j][i] = 0.f;
            wf[j][i] = to_f<T>(wv.v[i]);
        }
    }
    const long long step = (long long)gridDim.x * (kThreads / 32) * kRows;
    const float inv_width = 1.f / (float)a.width;
    Vals<T, VEC> v[NV], g[NV], s[NV];
    // Rows of 16-byte pieces come through a ring of kRing rows a warp, each lane
    // copying and reading its own pieces (no barrier): what is in flight does
    // not take registers, and 150 KB an SM of it keep memory busy. Others are
    // loaded when they are needed.
    constexpr int kRing = kRingOf<T, VEC, NV>;
    uint8_t *ring = (uint8_t *)shw + ((a.width * 4 + 15) & ~15) + threadIdx.x * 16;
    auto fetch = [&](long long row0, int slot) {
        const long long row = row0 + lane / LPR, base = row * a.width;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + l) * VEC;
            const bool in = row < a.rows && c < a.width;
            if constexpr (kRing > 0) {
                uint8_t *p = ring + (slot * NV + j) * 3 * kThreads * 16;
                const size_t at = in ? base + c : 0;
                copy16(p, x + at, in);
                copy16(p + kThreads * 16, dy + at, in);
                if (ds) copy16(p + 2 * kThreads * 16, ds + at, in);
            } else if (in) {
                load<T, VEC>(x + base + c, v[j].v);
                load<T, VEC>(dy + base + c, g[j].v);
                if (ds) load<T, VEC>(ds + base + c, s[j].v);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[j].v[i] = g[j].v[i] = s[j].v[i] = from_f<T>(0.f);
            }
        }
        if constexpr (kRing > 0) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const long long row_first = ((long long)blockIdx.x * (kThreads / 32) + warp) * kRows;
    if constexpr (kRing > 0)
        for (int i = 0; i < kRing - 1; ++i) fetch(row_first + i * step, i);
    int slot = 0;
    for (long long row0 = row_first; row0 < a.rows; row0 += step) {
        const long long row = row0 + lane / LPR, base = row * a.width;
        const bool live = row < a.rows;
        if constexpr (kRing > 0) {
            fetch(row0 + (kRing - 1) * step, slot ? slot - 1 : kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint8_t *p = ring + (slot * NV + j) * 3 * kThreads * 16;
                load<T, VEC>((const T *)p, v[j].v);
                load<T, VEC>((const T *)(p + kThreads * 16), g[j].v);
                if (ds) load<T, VEC>((const T *)(p + 2 * kThreads * 16), s[j].v);
            }
            slot = slot + 1 == kRing ? 0 : slot + 1;
        } else {
            fetch(row0, 0);
        }
        float f[NV][VEC], da[NV][VEC], ss, as;
        auto stats = [&]() {
            ss = as = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    ss = fmaf(f[j][i], f[j][i], ss);
                    as = fmaf(da[j][i], f[j][i], as);
                }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(kFull, ss, o);
                as += __shfl_xor_sync(kFull, as, o);
            }
        };
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[j][i] = to_f<T>(v[j].v[i]);
                da[j][i] = to_f<T>(g[j].v[i]) * wf[j][i];
            }
        stats();
        float sc = 1.f;
        // the sum of a s is of s as it is, too: s of 2^58 and a of 2^64 are ordinary numbers
        const bool over = ss > kMostSquares || !(fabsf(as) <= kMostSquares);
        if (__any_sync(kFull, over)) {
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) most = fmaxf(most, fabsf(f[j][i]));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
            sc = over ? down_scale(most) : 1.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[j][i] *= sc;
            stats();
        }
        const float r = rsqrtf(ss / (float)a.width + a.eps * sc * sc);  // of s sc
        const float k = as * inv_width * r * r;                         // dx = sc r (a - s sc k)
        const float rd = r * sc;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + l) * VEC;
            Vals<T, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                dw[j][i] = fmaf(to_f<T>(g[j].v[i]), f[j][i] * r, dw[j][i]);
                const float d = fmaf(-f[j][i], k, da[j][i]);
                o.v[i] = from_f<T>(ds ? fmaf(rd, d, to_f<T>(s[j].v[i])) : rd * d);
            }
            if (a.dx && live && c < a.width) store<T, VEC>((T *)a.dx + base + c, o.v);
        }
    }
    // the last steps' copies (zeros past the rows) land before the block's shared memory can go to another
    if constexpr (kRing > 0) asm volatile("cp.async.wait_all;" ::: "memory");
    if (!a.part) return;
    // the warp's row groups, then the warps one after the other
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) dw[j][i] += __shfl_xor_sync(kFull, dw[j][i], o);
    for (int t = 0; t < kThreads / 32; ++t) {
        if (warp == t && lane < LPR) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * LPR + l) * VEC;
                if (c < a.width)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) shw[c + i] = t ? shw[c + i] + dw[j][i] : dw[j][i];
            }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < a.width; c += kThreads) a.part[(long long)blockIdx.x * a.width + c] = shw[c];
}

// Wide rows: a block walks its rows; the partial weight gradient of the block
// lives in its row of `part` (each column belongs to one thread).
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_rms_norm_bwd_wide(NormBwdArgs a)
{
    __shared__ float sh[kThreads / 32];
    const T *x = (const T *)a.x, *w = (const T *)a.w, *dy = (const T *)a.dy, *ds = (const T *)a.ds;
    float *part = a.part ? a.part + (long long)blockIdx.x * a.width : nullptr;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const long long base = row * a.width;
        float ss, as, sc = 1.f;
        auto stats = [&]() {
            ss = as = 0.f;
            for (int c = threadIdx.x * VEC; c < a.width; c += kThreads * VEC) {
                Vals<T, VEC> v, g, wv;
                load<T, VEC>(x + base + c, v.v);
                load<T, VEC>(dy + base + c, g.v);
                if (w) load<T, VEC>(w + c, wv.v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float f = to_f<T>(v.v[i]) * sc, wi = w ? to_f<T>(wv.v[i]) : 1.f;
                    ss = fmaf(f, f, ss);
                    as = fmaf(to_f<T>(g.v[i]) * wi, f, as);
                }
            }
            ss = block_sum(ss, sh);
            as = block_sum(as, sh);
        };
        stats();
        if (ss > kMostSquares || !(fabsf(as) <= kMostSquares)) {  // the same in every thread
            float most = 0.f;
            for (int c = threadIdx.x * VEC; c < a.width; c += kThreads * VEC) {
                Vals<T, VEC> v;
                load<T, VEC>(x + base + c, v.v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) most = fmaxf(most, fabsf(to_f<T>(v.v[i])));
            }
            sc = down_scale(block_max(most, sh));
            stats();
        }
        const float r = rsqrtf(ss / (float)a.width + a.eps * sc * sc);
        const float k = as / (float)a.width * r * r, rd = r * sc;
        for (int c = threadIdx.x * VEC; c < a.width; c += kThreads * VEC) {
            Vals<T, VEC> v, g, wv, s, o;
            load<T, VEC>(x + base + c, v.v);
            load<T, VEC>(dy + base + c, g.v);
            if (w) load<T, VEC>(w + c, wv.v);
            if (ds) load<T, VEC>(ds + base + c, s.v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float f = to_f<T>(v.v[i]) * sc, gi = to_f<T>(g.v[i]), wi = w ? to_f<T>(wv.v[i]) : 1.f;
                if (part) part[c + i] = row == blockIdx.x ? gi * (f * r) : fmaf(gi, f * r, part[c + i]);
                float d = rd * fmaf(-f, k, gi * wi);
                if (ds) d += to_f<T>(s.v[i]);
                o.v[i] = from_f<T>(d);
            }
            if (a.dx) store<T, VEC>((T *)a.dx + base + c, o.v);
        }
    }
}

// dw[c] = sum of n partial rows, 32 threads a column in a fixed order, as pairs
__global__ void __launch_bounds__(kThreads) k_sum_rows(const float *__restrict__ part, int n, int width, float *dw)
{
    __shared__ Two sh[32][8];
    const int c8 = threadIdx.x & 7, c = blockIdx.x * 8 + c8, t = threadIdx.x >> 3;
    Two s = {0.f, 0.f};
    if (c < width)
#pragma unroll 4
        for (int i = t; i < n; i += 32) s = add(s, Two{part[(long long)i * width + c], 0.f});
    sh[t][c8] = s;
    __syncthreads();
    if (t == 0 && c < width) {
        for (int i = 1; i < 32; ++i) s = add(s, sh[i][c8]);
        dw[c] = s.hi + s.lo;
    }
}

// ---------------------------------------------------------------- host side
// Blocks of the backward pass, each of which writes one partial row: four a SM keep its memory pipe full, more where a
// block would take more than kSteps steps. Blocks that take one wide row at a time come in whole fives a SM, which are
// resident (100,000 x 2,048: 677 us, with four a SM 715, with just as many as kSteps needs 782); for the others
// just as many is faster (1,280,000 x 256: 382 us, 405 in threes a SM, of which those are resident).
int64_t bwd_blocks(pmha_dtype dt, int64_t rows, int64_t width)
{
    const Shape s = shape_of(dt, width);
    const int64_t per = s.lpr ? (int64_t)(kThreads / 32) * (32 / s.lpr) : 1, steps = (rows + per - 1) / per;
    const int64_t full = (int64_t)num_sms() * (s.lpr ? 4 : 5);
    const int64_t least = s.lpr ? (steps + kSteps - 1) / kSteps : (steps + full * kSteps - 1) / (full * kSteps) * full;
    return std::max<int64_t>(1, std::min(steps, std::max(full, least)));
}

}  // namespace
}  // namespace pmha

using namespace pmha;

extern "C" {

pmha_status pmha_rms_norm(pmha_dtype dtype, int64_t rows, int64_t width, const void *x, const void *residual,
                          const void *weight, float eps, void *sum, void *out, void *out_q, float *scale,
                          pmha_stream stream)
{
    pmha_status st = check_rows("pmha_rms_norm", dtype, rows, width);
    if (st != PMHA_OK) return st;
    if (!(eps >= 1e-30f) || !isfinite(eps)) {
        set_error("pmha_rms_norm: eps %g must be finite and at least 1e-30", (double)eps);
        return PMHA_ERR_INVALID_ARG;
    }
    if (rows == 0) return PMHA_OK;
    if ((!out && !out_q) || (out_q == nullptr) != (scale == nullptr)) {
        set_error("pmha_rms_norm: out or out_q is needed, and out_q and scale go together");
        return PMHA_ERR_INVALID_ARG;
    }
    if (!x || !aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) ||
        !aligned(out, 16) || !aligned(out_q, 16) || !aligned(scale, 16)) {
        set_error("pmha_rms_norm: x is NULL, or a pointer is not 16-byte aligned");
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t n = (size_t)(rows * width), nb = n * bytes_of(dtype), wb = (size_t)width * bytes_of(dtype);
    const void *outs[4] = {sum, out, out_q, scale};
    const size_t out_n[4] = {nb, nb, n, (size_t)rows * 4};
    for (int i = 0; i < 4; ++i) {
        bool bad = overlap(outs[i], out_n[i], x, nb) || overlap(outs[i], out_n[i], residual, nb) ||
                   overlap(outs[i], out_n[i], weight, wb);
        for (int j = 0; j < i; ++j) bad |= overlap(outs[i], out_n[i], outs[j], out_n[j]);
        if (bad) {
            set_error("pmha_rms_norm: an output overlaps an input or another output");
            return PMHA_ERR_INVALID_ARG;
        }
    }
    const double inv = 1.0 / (double)width;
    NormArgs a{Two{(float)inv, (float)(inv - (double)(float)inv)}, x, residual, weight, sum, out, (uint8_t *)out_q, scale, rows, (int)width, eps};
    const Shape s = shape_of(dtype, width);
    cudaStream_t cs = (cudaStream_t)stream;
    {
        StageTimer timer(out_q ? "rms_norm_quantized" : "rms_norm", cs);
        if (s.lpr) {
            const int64_t per = (int64_t)(kThreads / 32) * (32 / s.lpr);
            const unsigned grid = (unsigned)((rows + per - 1) / per);
            dispatch(dtype, s, [&](auto t) {
                using G = decltype(t);
                if (out_q) k_rms_norm<typename G::type, G::vec, G::nv, G::lpr, true><<<grid, kThreads, 0, cs>>>(a);
                else k_rms_norm<typename G::type, G::vec, G::nv, G::lpr, false><<<grid, kThreads, 0, cs>>>(a);
            });
        } else {
            dispatch_wide(dtype, s.vec, [&](auto t) {
                using G = decltype(t);
                if (out_q) k_rms_norm_wide<typename G::type, G::vec, true><<<(unsigned)rows, kThreads, 0, cs>>>(a);
                else k_rms_norm_wide<typename G::type, G::vec, false><<<(unsigned)rows, kThreads, 0, cs>>>(a);
            });
        }
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

size_t pmha_rms_norm_backward_workspace_size(pmha_dtype dtype, int64_t rows, int64_t width)
{
    if (check_rows("pmha_rms_norm_backward", dtype, rows, width) != PMHA_OK) return 0;
    return (((size_t)bwd_blocks(dtype, rows, width) * (size_t)width * 4) + 255) & ~(size_t)255;
}

pmha_status pmha_rms_norm_backward(pmha_dtype dtype, int64_t rows, int64_t width, const void *x, const void *weight,
                                   float eps, const void *dout, const void *dsum, void *dx, float *dweight,
                                   void *workspace, size_t workspace_bytes, pmha_stream stream)
{
    pmha_status st = check_rows("pmha_rms_norm_backward", dtype, rows, width);
    if (st != PMHA_OK) return st;
    if (!(eps >= 1e-30f) || !isfinite(eps)) {
        set_error("pmha_rms_norm_backward: eps %g must be finite and at least 1e-30", (double)eps);
        return PMHA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = (cudaStream_t)stream;
    if (!aligned(dweight, 16)) {
        set_error("pmha_rms_norm_backward: dweight is not 16-byte aligned");
        return PMHA_ERR_INVALID_ARG;
    }
    if (rows == 0) {
        if (dweight) PMHA_CUDA_TRY(cudaMemsetAsync(dweight, 0, (size_t)width * 4, cs));
        return PMHA_OK;
    }
    if (!x || !dout || !aligned(x, 16) || !aligned(weight, 16) || !aligned(dout, 16) || !aligned(dsum, 16) ||
        !aligned(dx, 16)) {
        set_error("pmha_rms_norm_backward: x or dout is NULL, or a pointer is not 16-byte aligned");
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t nb = (size_t)(rows * width) * bytes_of(dtype), wb = (size_t)width * bytes_of(dtype);
    const void *ins[4] = {x, dout, dsum, weight};
    const size_t in_n[4] = {nb, nb, nb, wb};
    const size_t need = pmha_rms_norm_backward_workspace_size(dtype, rows, width);
    bool bad = overlap(dx, nb, dweight, (size_t)width * 4);
    for (int i = 0; i < 4; ++i)
        bad |= overlap(dx, nb, ins[i], in_n[i]) || overlap(dweight, (size_t)width * 4, ins[i], in_n[i]);
    if (bad) {
        set_error("pmha_rms_norm_backward: an output overlaps an input or another output");
        return PMHA_ERR_INVALID_ARG;
    }
    if (!dx && !dweight) return PMHA_OK;
    if (dweight && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))) {
        set_error("pmha_rms_norm_backward: workspace needs %zu bytes, 256-byte aligned (got %zu at %p)", need,
                  workspace_bytes, workspace);
        return PMHA_ERR_WORKSPACE;
    }
    const int64_t grid = bwd_blocks(dtype, rows, width);
    NormBwdArgs a{x, weight, dout, dsum, dx, dweight ? (float *)workspace : nullptr, rows, (int)width, eps};
    const Shape s = shape_of(dtype, width);
    cudaError_t attr = cudaSuccess;
    {
        StageTimer timer("rms_norm_backward", cs);
        if (s.lpr)
            dispatch(dtype, s, [&](auto t) {
                using G = decltype(t);
                using T = typename G::type;
                // the block's weight gradient, then the ring: below 48 KB + 4 KB
                const size_t smem = (((size_t)width * 4 + 15) & ~(size_t)15) +
                                    (size_t)kRingOf<T, G::vec, G::nv> * G::nv * 3 * kThreads * 16;
                auto kern = k_rms_norm_bwd<T, G::vec, G::nv, G::lpr>;
                attr = smem > 48 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                        : cudaSuccess;
                if (attr == cudaSuccess) kern<<<(unsigned)grid, kThreads, smem, cs>>>(a);
            });
        else
            dispatch_wide(dtype, s.vec, [&](auto t) {
                using G = decltype(t);
                k_rms_norm_bwd_wide<typename G::type, G::vec><<<(unsigned)grid, kThreads, 0, cs>>>(a);
            });
    }
    PMHA_CUDA_TRY(attr);
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    if (dweight) {
        StageTimer timer("rms_norm_dweight", cs);
        k_sum_rows<<<(unsigned)((width + 7) / 8), kThreads, 0, cs>>>(a.part, (int)grid, (int)width, dweight);
        count_launch();
        PMHA_CUDA_TRY(cudaGetLastError());
    }
    return PMHA_OK;
}

}  // extern "C"
