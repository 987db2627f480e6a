// The gated block for a few tokens (single-token decoding, small graphs): the
// weights are read once, by every SM, and multiplied on the CUDA cores. A warp
// takes one hidden column (its gate and up rows, 16 bytes a lane), then one
// output column, for 16 tokens, which lie in shared memory; the hidden rows go
// through L2 in float32. What bounds it is latency: two launches, of which the
// second comes up and loads its weights while the first one runs.
#include <cuda_fp8.h>

#include <type_traits>

#include "ffn_internal.h"
#include "ffn_math.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

// Type of the tokens and of the gate and up weights (E4M3 ones have scales); the rest of a block is float32 or bf16.
enum Kind { kBf16, kE4m3, kF32 };
template <int KIND>
constexpr int kBytesOf = KIND == kF32 ? 4 : KIND == kE4m3 ? 1 : 2;

struct SmallArgs {
    const void *x, *wg, *wu;
    const float *xs, *gs, *us;
    const void *wd, *bg, *bu, *bd, *res;  // float32 or bf16
    float *h;
    void *out;
    int M, E, F;
};
constexpr int kTokens = 16;  // of a block; blockIdx.y counts the blocks of tokens

// This block's tokens of the arguments; `bytes` of a token's value, es of a result's.
__device__ __forceinline__ SmallArgs tokens_of(SmallArgs a, int bytes, int es)
{
    const int m0 = blockIdx.y * kTokens;
    a.x = (const uint8_t *)a.x + (size_t)m0 * a.E * bytes;
    if (a.xs) a.xs += m0;
    if (a.res) a.res = (const uint8_t *)a.res + (size_t)m0 * a.E * es;
    a.h += (size_t)m0 * a.F;
    a.out = (uint8_t *)a.out + (size_t)m0 * a.E * es;
    a.M = min(kTokens, a.M - m0);
    return a;
}
__device__ __forceinline__ float value_at(const void *p, size_t i, bool f32)
{
    return f32 ? ((const float *)p)[i] : __bfloat162float(((const __nv_bfloat16 *)p)[i]);
}

// V consecutive values as float: 16 bytes of float32 (V = 4), bf16 (8) or E4M3 (16), or one value
template <int KIND, int V>
__device__ __forceinline__ void widen(const void *p, float (&f)[V])
{
    if constexpr (V == 1) {
        f[0] = value_at(p, 0, KIND == kF32);
    } else {
        const uint4 raw = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (KIND == kF32) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (KIND == kE4m3) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * k)), __NV_E4M3);
                    const float2 e = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                    f[4 * i + 2 * k] = e.x;
                    f[4 * i + 2 * k + 1] = e.y;
                }
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

template <int KIND, int V, int MB, int ACT>
__global__ void __launch_bounds__(kThreads) k_small_up(SmallArgs all)
{
    constexpr int kBytes = kBytesOf<KIND>;
    constexpr bool kIsF32 = KIND == kF32;
    const SmallArgs a = tokens_of(all, kBytes, kIsF32 ? 4 : 2);
    extern __shared__ __align__(16) uint8_t x_s[];  // M rows
    tcu::grid_dependents_may_start();
    const int lane = threadIdx.x & 31, f = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if constexpr (V > 1) {
        for (int i = threadIdx.x * 16; i < a.M * a.E * kBytes; i += kThreads * 16)
            *reinterpret_cast<uint4 *>(x_s + i) = *reinterpret_cast<const uint4 *>((const uint8_t *)a.x + i);
    } else {
        using Word = std::conditional_t<kIsF32, uint32_t, uint16_t>;
        for (int i = threadIdx.x; i < a.M * a.E; i += kThreads) ((Word *)x_s)[i] = ((const Word *)a.x)[i];
    }
    __syncthreads();
    if (f >= a.F) return;
    const uint8_t *wg = (const uint8_t *)a.wg + (size_t)f * a.E * kBytes, *wu = (const uint8_t *)a.wu + (size_t)f * a.E * kBytes;
    float g[MB], u[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) g[m] = u[m] = 0.f;
#pragma unroll 2
    for (int c = lane * V; c < a.E; c += 32 * V) {
        float eg[V], eu[V], ex[V];
        widen<KIND, V>(wg + (size_t)c * kBytes, eg);
        widen<KIND, V>(wu + (size_t)c * kBytes, eu);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m >= a.M) break;
            widen<KIND, V>(x_s + ((size_t)m * a.E + c) * kBytes, ex);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                g[m] = fmaf(eg[i], ex[i], g[m]);
                u[m] = fmaf(eu[i], ex[i], u[m]);
            }
        }
    }
    float mg = 0.f, mu = 0.f;  // of token `lane`
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const float sg = warp_sum(g[m]), su = warp_sum(u[m]);
        if (lane == m) mg = sg, mu = su;
    }
    if (lane >= a.M) return;
    if constexpr (KIND == kE4m3) {
        const float xs = a.xs[lane];
        mg *= xs * a.gs[f];
        mu *= xs * a.us[f];
    }
    if (a.bg) mg += value_at(a.bg, f, kIsF32);
    if (a.bu) mu += value_at(a.bu, f, kIsF32);
    a.h[(size_t)lane * a.F + f] =
        kIsF32 ? Act<ACT>::exact(mg) * mu : Act<ACT>::hidden(mg * Act<ACT>::kGate, mu * Act<ACT>::kUp);
}

template <bool F32, int V, int MB>
__global__ void __launch_bounds__(kThreads) k_small_down(SmallArgs all)
{
    constexpr int KIND = F32 ? kF32 : kBf16, kBytes = F32 ? 4 : 2;
    const SmallArgs a = tokens_of(all, kBytes, kBytes);
    constexpr int kAhead = 4;  // weight pieces loaded before the hidden rows are there
    const int lane = threadIdx.x & 31, e = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const uint8_t *wd = (const uint8_t *)a.wd + (size_t)min(e, a.E - 1) * a.F * kBytes;
    float w[kAhead][V];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const int c = (j * 32 + lane) * V;
        if (c < a.F) widen<KIND, V>(wd + (size_t)c * kBytes, w[j]);
    }
    tcu::grid_wait();  // the weights come from before the launch that this one overlaps
    if (e >= a.E) return;
    float y[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) y[m] = 0.f;
    auto add = [&](const float (&wv)[V], int c) {
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m >= a.M) break;
            const float *h = a.h + (size_t)m * a.F + c;
            float hv[V];
            if constexpr (V == 1) {
                hv[0] = h[0];
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    *reinterpret_cast<float4 *>(hv + i) = *reinterpret_cast<const float4 *>(h + i);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) y[m] = fmaf(wv[i], hv[i], y[m]);
        }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const int c = (j * 32 + lane) * V;
        if (c < a.F) add(w[j], c);
    }
    for (int c = (kAhead * 32 + lane) * V; c < a.F; c += 32 * V) {
        widen<KIND, V>(wd + (size_t)c * kBytes, w[0]);
        add(w[0], c);
    }
    float mine = 0.f;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const float s = warp_sum(y[m]);
        if (lane == m) mine = s;
    }
    if (lane >= a.M) return;
    const size_t at = (size_t)lane * a.E + e;
    if (a.bd) mine += value_at(a.bd, e, F32);
    if (a.res) mine += value_at(a.res, at, F32);
    if constexpr (F32) ((float *)a.out)[at] = mine;
    else ((__nv_bfloat16 *)a.out)[at] = __float2bfloat16_rn(mine);
}

template <int KIND, int V, int MB>
pmha_status launch_up(pmha_act act, const SmallArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)((a.F + kWarps - 1) / kWarps), (unsigned)((a.M + kTokens - 1) / kTokens));
    const size_t smem = (size_t)std::min(a.M, kTokens) * a.E * kBytesOf<KIND>;
    StageTimer timer(KIND == kE4m3 ? "ffn_up_quantized" : "ffn_up", s);
    if (act == PMHA_ACT_SILU) k_small_up<KIND, V, MB, PMHA_ACT_SILU><<<grid, kThreads, smem, s>>>(a);
    else k_small_up<KIND, V, MB, PMHA_ACT_GELU><<<grid, kThreads, smem, s>>>(a);
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

template <int MB>
pmha_status launch(pmha_act act, const SmallArgs &a, bool f32, cudaStream_t s)
{
    pmha_status st;
    if (a.xs) st = launch_up<kE4m3, 16, MB>(act, a, s);
    else if (f32) st = a.E % 4 == 0 ? launch_up<kF32, 4, MB>(act, a, s) : launch_up<kF32, 1, MB>(act, a, s);
    else st = a.E % 8 == 0 ? launch_up<kBf16, 8, MB>(act, a, s) : launch_up<kBf16, 1, MB>(act, a, s);
    if (st != PMHA_OK) return st;
    StageTimer timer("ffn_down", s);
    const dim3 grid((unsigned)((a.E + kWarps - 1) / kWarps), (unsigned)((a.M + kTokens - 1) / kTokens));
    if (f32)
        return a.F % 4 == 0 ? tcu::launch_overlapping(k_small_down<true, 4, MB>, grid, kThreads, 0, s, a)
                            : tcu::launch_overlapping(k_small_down<true, 1, MB>, grid, kThreads, 0, s, a);
    return a.F % 8 == 0 ? tcu::launch_overlapping(k_small_down<false, 8, MB>, grid, kThreads, 0, s, a)
                        : tcu::launch_overlapping(k_small_down<false, 1, MB>, grid, kThreads, 0, s, a);
}

}  // namespace

// Up to 4 tokens, of float32 8, and up to 64 where all their values are 2,048 at
// most (whose hidden rows better stay float32). Against the other kernels, whose
// tiles hold 64 or 256 tokens (us): bf16, 256 x 1,024, 1 token 4.2 / 13.2, 4 tokens
// 7.7 / 13.2, 8 tokens 13.4 / 13.2; 512 x 2,048, 4 tokens 12 / 19, 8 tokens 24 / 19;
// 64 x 256, 32 tokens 8.9 / 6.7. Float32, 1,024 x 4,096, 1 token 9.9 / 164, 8 tokens
// 82 / 162, 16 tokens 159 / 159. 16 rows have to fit in 48 KB of shared memory.
bool ffn_small_supported(int64_t E, int64_t M, int token_bytes)
{
    if (std::min<int64_t>(M, kTokens) * E * token_bytes > 48 * 1024) return false;
    return M <= (token_bytes == 4 ? 8 : 4) || (token_bytes < 4 && M <= 64 && M * E <= 2048);
}

pmha_status ffn_small_forward(const FfnTc &f, bool f32, const FfnUpArgs &u, const void *wd, const void *residual,
                              void *out, cudaStream_t s)
{
    SmallArgs a = {};
    a.x = u.x, a.wg = u.wg, a.wu = u.wu, a.xs = u.x_scale, a.gs = u.wg_scale, a.us = u.wu_scale;
    a.wd = wd, a.res = residual, a.bg = f.bg, a.bu = f.bu, a.bd = f.bd;
    a.h = (float *)u.h, a.out = out;
    a.M = (int)u.M, a.E = (int)f.E, a.F = (int)f.F;
    if (a.M == 1) return launch<1>(f.act, a, f32, s);
    return a.M <= 4 ? launch<4>(f.act, a, f32, s) : launch<16>(f.act, a, f32, s);
}

}  // namespace pmha
