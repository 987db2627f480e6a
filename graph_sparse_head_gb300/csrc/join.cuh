// What the forward and the backward kernels of the join share.
#pragma once

#include <algorithm>

#include "kept.cuh"

namespace pmha {
namespace {

__host__ __device__ inline int64_t groups_of(int64_t width) { return (width + kGroup - 1) / kGroup; }

// A tensor of the layer type, or one kept in 8 bits (codes set), or none.
struct Source {
    const void *p;
    Kept k;
    __device__ __forceinline__ bool any() const { return p || k.codes; }
};
template <typename T, int VEC>
__device__ __forceinline__ void load_source(const Source &s, long long row, int c, int width, float (&v)[VEC])
{
    if (s.p) {
        Vals<T, VEC> t;
        load<T, VEC>((const T *)s.p + row * width + c, t.v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f<T>(t.v[i]);
    } else {
        load_kept<VEC>(s.k, row, c, width, v);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void load_row(const void *p, long long at, float (&v)[VEC])
{
    Vals<T, VEC> t;
    load<T, VEC>((const T *)p + at, t.v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f<T>(t.v[i]);
}

// VEC values rounded to the type, two to an instruction in bf16; v holds them as rounded afterwards
template <typename T, int VEC>
__device__ __forceinline__ Vals<T, VEC> rounded(float (&v)[VEC])
{
    Vals<T, VEC> r;
    if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
        uint32_t *w = reinterpret_cast<uint32_t *>(r.v);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[i], v[i + 1]);
            w[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
            v[i] = __uint_as_float(w[i / 2] << 16);
            v[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            r.v[i] = from_f<T>(v[i]);
            v[i] = to_f<T>(r.v[i]);
        }
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void widen(const Vals<T, VEC> &r, float *v)
{
    if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(r.v);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            v[i] = __uint_as_float(w[i / 2] << 16);
            v[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f<T>(r.v[i]);
    }
}
// 16 bytes of values, or their codes, into the ring
__device__ __forceinline__ void ring_copy(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int VEC>
__device__ __forceinline__ void ring_codes(uint32_t dst, const int8_t *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(VEC == 8 ? 8 : 4) : "memory");
}

// A row is shared by LPR threads ("a team"), lanes of one warp or whole warps of
// a block, each with some eight values in registers. Sums over a team of warps go through
// shared memory: a warp writes to one of two places in turn, so that one barrier for up to three sums is enough
// (who writes to a place again has passed the barrier behind which all have read it).
struct TeamSums {
    float v[2][3][kThreads / 32];
};
template <int LPR, bool MAX, int K>
__device__ __forceinline__ void team_reduce(float (&v)[K], TeamSums &sh, int &turn)
{
    static_assert(K <= 3, "places in TeamSums");
    constexpr int kLanes = LPR < 32 ? LPR : 32;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float t = __shfl_xor_sync(kFull, v[k], o);
            v[k] = MAX ? fmaxf(v[k], t) : v[k] + t;
        }
    if constexpr (LPR > 32) {
        constexpr int kWarps = LPR / 32;
        const int warp = threadIdx.x >> 5, first = warp / kWarps * kWarps;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) sh.v[turn][k][warp] = v[k];
        }
        if constexpr (LPR == kThreads) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / LPR), "n"(LPR) : "memory");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = sh.v[turn][k][first];
#pragma unroll
            for (int i = 1; i < kWarps; ++i)
                v[k] = MAX ? fmaxf(v[k], sh.v[turn][k][first + i]) : v[k] + sh.v[turn][k][first + i];
        }
        turn ^= 1;
    }
}
template <int N>
__device__ __forceinline__ float squares_of(const float (&f)[N])
{
    const Values<N> v(f);
    return Values<N>::dot(v, v);
}
// The power of two that a team's row is scaled by, in place, where `over`.
template <int N, int LPR>
__device__ __forceinline__ float scale_row(float (&f)[N], bool over, TeamSums &sh, int &turn)
{
    float most[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) most[0] = fmaxf(most[0], fabsf(f[i]));
    team_reduce<LPR, true>(most, sh, turn);
    const float sc = over ? down_scale(most[0]) : 1.f;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] *= sc;
    return sc;
}
// The row's 1 / rms; a row whose squares leave float32 is scaled in place by *sc first.
template <int N, int LPR>
__device__ __forceinline__ float row_root(float (&f)[N], float inv_width, float eps, float *sc, TeamSums &sh, int &turn)
{
    float ss[1] = {squares_of(f)};
    team_reduce<LPR, false>(ss, sh, turn);
    *sc = 1.f;
    if (__any_sync(kFull, ss[0] > kMostSquares)) {  // a team of warps comes here together: they have one row
        *sc = scale_row<N, LPR>(f, ss[0] > kMostSquares, sh, turn);
        ss[0] = squares_of(f);
        team_reduce<LPR, false>(ss, sh, turn);
    }
    return rsqrtf(fmaf(ss[0], inv_width, eps * *sc * *sc));
}

// The kernel shape of a width up to 2048: values a piece, pieces a thread, threads a row; 0 threads: one block walks the
// row. Eight values a thread, or four of float32 rows that fit a warp so: with 32 values a thread (a warp for every
// row) the backward pass spills.
inline Shape join_shape(pmha_dtype dt, int64_t width)
{
    const int vec = shape_of(dt, width).vec;
    if (width > 2048) return {vec, 0, 0};
    if (vec < 4) return {vec, 8 / vec, width <= 256 ? 32 : 256};
    if (vec == 4 && width <= 128) return {vec, 1, width <= 32 ? 8 : width <= 64 ? 16 : 32};
    int lpr = vec == 4 ? 32 : 8;
    while (lpr * 8 < width) lpr *= 2;
    return {vec, 8 / vec, lpr};
}
template <typename F>
void join_dispatch(pmha_dtype dt, Shape s, F f)
{
    using B = __nv_bfloat16;
    if (s.vec == 8) {
        if (s.lpr == 8) f(Tag<B, 8, 1, 8>());
        else if (s.lpr == 16) f(Tag<B, 8, 1, 16>());
        else if (s.lpr == 32) f(Tag<B, 8, 1, 32>());
        else if (s.lpr == 64) f(Tag<B, 8, 1, 64>());
        else if (s.lpr == 128) f(Tag<B, 8, 1, 128>());
        else f(Tag<B, 8, 1, 256>());
    } else if (s.vec == 4) {
        if (s.lpr == 8) f(Tag<float, 4, 1, 8>());
        else if (s.lpr == 16) f(Tag<float, 4, 1, 16>());
        else if (s.lpr == 32 && s.nv == 1) f(Tag<float, 4, 1, 32>());
        else if (s.lpr == 32) f(Tag<float, 4, 2, 32>());
        else if (s.lpr == 64) f(Tag<float, 4, 2, 64>());
        else if (s.lpr == 128) f(Tag<float, 4, 2, 128>());
        else f(Tag<float, 4, 2, 256>());
    } else if (s.vec == 2) {
        if (s.lpr == 32) f(Tag<B, 2, 4, 32>());
        else f(Tag<B, 2, 4, 256>());
    } else if (dt == PMHA_BF16) {
        if (s.lpr == 32) f(Tag<B, 1, 8, 32>());
        else f(Tag<B, 1, 8, 256>());
    } else {
        if (s.lpr == 32) f(Tag<float, 1, 8, 32>());
        else f(Tag<float, 1, 8, 256>());
    }
}

// 1 / rms of a row that a block shares, from its squares' sum ss and largest magnitude: taken again times *sc where the
// squares leave float32. squares(sc) and most() walk the row.
template <typename F, typename G>
__device__ __forceinline__ float block_root(float *sh, int width, float eps, float *sc, F squares, G most)
{
    *sc = 1.f;
    float ss = block_sum(squares(1.f), sh);
    if (ss > kMostSquares) {  // the same in every thread
        *sc = down_scale(block_max(most(), sh));
        ss = block_sum(squares(*sc), sh);
    }
    return rsqrtf(ss / (float)width + eps * *sc * *sc);
}

// ---------------------------------------------------------------- host side
inline Span codes_of(const pmha_kept *k, int64_t rows, int64_t width)
{
    return k ? Span{k->codes, (size_t)(rows * width)} : Span{nullptr, 0};
}
inline Span scales_of(const pmha_kept *k, int64_t rows, int64_t width)
{
    return k ? Span{k->scale, (size_t)(rows * groups_of(width)) * 2} : Span{nullptr, 0};
}
inline bool whole(const pmha_kept *k)  // absent, or with both of its arrays
{
    return !k || (k->codes && k->scale && aligned(k->codes, 16) && aligned(k->scale, 16));
}
inline Source source(const void *p, const pmha_kept *k)
{
    return Source{p, Kept{k ? (const int8_t *)k->codes : nullptr, k ? (const __nv_bfloat16 *)k->scale : nullptr}};
}
inline KeptOut kept_out(const pmha_kept *k)
{
    return KeptOut{k ? (int8_t *)k->codes : nullptr, k ? (__nv_bfloat16 *)k->scale : nullptr};
}

inline pmha_status check_join(const char *who, const pmha_join_params *p, int64_t rows)
{
    if (!p) {
        set_error("%s: params is NULL", who);
        return PMHA_ERR_INVALID_ARG;
    }
    pmha_status st = check_rows(who, p->dtype, rows, p->width);
    if (st != PMHA_OK) return st;
    if (!(p->eps >= 1e-30f) || !isfinite(p->eps) || !isfinite(p->residual_scale)) {
        set_error("%s: eps %g must be finite and at least 1e-30, residual_scale %g finite", who, (double)p->eps,
                  (double)p->residual_scale);
        return PMHA_ERR_INVALID_ARG;
    }
    if (p->gate ? p->gates < 1 || (rows > 0 && (p->gates > rows || rows % p->gates != 0)) : p->gates != 0) {
        set_error("%s: gates %lld must be 0 without a gate, and a divisor of the %lld rows with one", who,
                  (long long)p->gates, (long long)rows);
        return PMHA_ERR_INVALID_ARG;
    }
    if (!aligned(p->post, 16) || !aligned(p->gate, 16) || !aligned(p->pre, 16)) {
        set_error("%s: post, gate or pre is not 16-byte aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    return PMHA_OK;
}


}  // namespace
}  // namespace pmha
