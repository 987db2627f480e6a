// The gated block for a few tokens (single-token decoding, small graphs): the
// weights are read once, by every SM, and multiplied on the CUDA cores. A warp
// takes one hidden column (its gate and up rows, 16 bytes a lane), then one
// output column, for 16 tokens, which lie in shared memory; the hidden rows go
// through L2 in float32. What bounds it is latency: two launches, of which the
// second comes up and loads its weights while the first one runs.
#include <cuda_fp8.h>

#include "ffn_internal.h"
#include "ffn_math.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

struct SmallArgs {
    const void *x, *wg, *wu;
    const float *xs, *gs, *us;
    const __nv_bfloat16 *wd, *bg, *bu, *bd, *res;
    float *h;
    __nv_bfloat16 *out;
    int M, E, F;
};
constexpr int kTokens = 16;  // of a block; blockIdx.y counts the blocks of tokens

// This block's tokens of the arguments.
__device__ __forceinline__ SmallArgs tokens_of(SmallArgs a, int bytes)
{
    const int m0 = blockIdx.y * kTokens;
    a.x = (const uint8_t *)a.x + (size_t)m0 * a.E * bytes;
    if (a.xs) a.xs += m0;
    if (a.res) a.res += (size_t)m0 * a.E;
    a.h += (size_t)m0 * a.F;
    a.out += (size_t)m0 * a.E;
    a.M = min(kTokens, a.M - m0);
    return a;
}

// V consecutive values as float: 16 bytes of bf16 (V = 8) or E4M3 (V = 16), or one value
template <bool Q8, int V>
__device__ __forceinline__ void widen(const void *p, float (&f)[V])
{
    if constexpr (V == 1) {
        f[0] = __bfloat162float(*(const __nv_bfloat16 *)p);
    } else {
        const uint4 raw = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Q8) {
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

template <bool Q8, int V, int MB, int ACT>
__global__ void __launch_bounds__(kThreads) k_small_up(SmallArgs all)
{
    constexpr int kBytes = Q8 ? 1 : 2;
    const SmallArgs a = tokens_of(all, kBytes);
    extern __shared__ __align__(16) uint8_t x_s[];  // M rows
    tcu::grid_dependents_may_start();
    const int lane = threadIdx.x & 31, f = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if constexpr (V > 1) {
        for (int i = threadIdx.x * 16; i < a.M * a.E * kBytes; i += kThreads * 16)
            *reinterpret_cast<uint4 *>(x_s + i) = *reinterpret_cast<const uint4 *>((const uint8_t *)a.x + i);
    } else {
        for (int i = threadIdx.x; i < a.M * a.E; i += kThreads) ((uint16_t *)x_s)[i] = ((const uint16_t *)a.x)[i];
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
        widen<Q8, V>(wg + (size_t)c * kBytes, eg);
        widen<Q8, V>(wu + (size_t)c * kBytes, eu);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m >= a.M) break;
            widen<Q8, V>(x_s + ((size_t)m * a.E + c) * kBytes, ex);
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
    if constexpr (Q8) {
        const float xs = a.xs[lane];
        mg *= xs * a.gs[f];
        mu *= xs * a.us[f];
    }
    if (a.bg) mg += __bfloat162float(a.bg[f]);
    if (a.bu) mu += __bfloat162float(a.bu[f]);
    a.h[(size_t)lane * a.F + f] = Act<ACT>::hidden(mg * Act<ACT>::kGate, mu * Act<ACT>::kUp);
}

template <int V, int MB>
__global__ void __launch_bounds__(kThreads) k_small_down(SmallArgs all)
{
    const SmallArgs a = tokens_of(all, 2);
    constexpr int kAhead = 4;  // weight pieces loaded before the hidden rows are there
    const int lane = threadIdx.x & 31, e = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const __nv_bfloat16 *wd = a.wd + (size_t)min(e, a.E - 1) * a.F;
    float w[kAhead][V];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const int c = (j * 32 + lane) * V;
        if (c < a.F) widen<false, V>(wd + c, w[j]);
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
            if constexpr (V == 8) {
                *reinterpret_cast<float4 *>(hv) = *reinterpret_cast<const float4 *>(h);
                *reinterpret_cast<float4 *>(hv + 4) = *reinterpret_cast<const float4 *>(h + 4);
            } else {
                hv[0] = h[0];
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
        widen<false, V>(wd + c, w[0]);
        add(w[0], c);
    }
    float mine = 0.f;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const float s = warp_sum(y[m]);
        if (lane == m) mine = s;
    }
    if (lane >= a.M) return;
    if (a.bd) mine += __bfloat162float(a.bd[e]);
    if (a.res) mine += __bfloat162float(a.res[(size_t)lane * a.E + e]);
    a.out[(size_t)lane * a.E + e] = __float2bfloat16_rn(mine);
}

template <bool Q8, int V, int MB>
pmha_status launch_up(pmha_act act, const SmallArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)((a.F + kWarps - 1) / kWarps), (unsigned)((a.M + kTokens - 1) / kTokens));
    const size_t smem = (size_t)std::min(a.M, kTokens) * a.E * (Q8 ? 1 : 2);
    StageTimer timer(Q8 ? "ffn_up_quantized" : "ffn_up", s);
    if (act == PMHA_ACT_SILU) k_small_up<Q8, V, MB, PMHA_ACT_SILU><<<grid, kThreads, smem, s>>>(a);
    else k_small_up<Q8, V, MB, PMHA_ACT_GELU><<<grid, kThreads, smem, s>>>(a);
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

template <int MB>
pmha_status launch(pmha_act act, const SmallArgs &a, cudaStream_t s)
{
    pmha_status st;
    if (a.xs) st = launch_up<true, 16, MB>(act, a, s);
    else if (a.E % 8 == 0) st = launch_up<false, 8, MB>(act, a, s);
    else st = launch_up<false, 1, MB>(act, a, s);
    if (st != PMHA_OK) return st;
    StageTimer timer("ffn_down", s);
    const dim3 grid((unsigned)((a.E + kWarps - 1) / kWarps), (unsigned)((a.M + kTokens - 1) / kTokens));
    return a.F % 8 == 0 ? tcu::launch_overlapping(k_small_down<8, MB>, grid, kThreads, 0, s, a)
                        : tcu::launch_overlapping(k_small_down<1, MB>, grid, kThreads, 0, s, a);
}

}  // namespace

// Up to 64 tokens, 16 of whose rows fit in 48 KB of shared memory. One token
// through width 256, hidden 1,024: 6.2 us against 17 of the tensor-core kernels,
// whose tiles hold 256 tokens.
bool ffn_small_supported(int64_t E, int64_t M, bool q8)
{
    return M <= kSmallRows && std::min<int64_t>(M, kTokens) * E * (q8 ? 1 : 2) <= 48 * 1024;
}

pmha_status ffn_small_forward(const FfnTc &f, const FfnUpArgs &u, const void *wd, const void *residual, void *out,
                              cudaStream_t s)
{
    SmallArgs a = {};
    a.x = u.x, a.wg = u.wg, a.wu = u.wu, a.xs = u.x_scale, a.gs = u.wg_scale, a.us = u.wu_scale;
    a.wd = (const __nv_bfloat16 *)wd, a.res = (const __nv_bfloat16 *)residual;
    a.bg = (const __nv_bfloat16 *)f.bg, a.bu = (const __nv_bfloat16 *)f.bu, a.bd = (const __nv_bfloat16 *)f.bd;
    a.h = (float *)u.h, a.out = (__nv_bfloat16 *)out;
    a.M = (int)u.M, a.E = (int)f.E, a.F = (int)f.F;
    if (a.M == 1) return launch<1>(f.act, a, s);
    return a.M <= 4 ? launch<4>(f.act, a, s) : launch<16>(f.act, a, s);
}

}  // namespace pmha
