// Microscaled 4-bit floating point (mx.cuh): quantisation, products for a few
// tokens, argument checks and the order of launches of the linear product and the gated block.
//
//   linear  y = x W^T + bias + residual
//   block   h = act(x Wg^T + bg) * (x Wu^T + bu), rounded to 4 bits;  y = h Wd^T + bd + residual
//
// Sums are float32 (products of two E2M1 values are exact in any of the forms), outputs bf16.
#include <math.h>

#include <algorithm>

#include "ffn_math.cuh"
#include "mx.cuh"
#include "pair.cuh"
#include "rows.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {

// ---------------------------------------------------------------- quantisation
// A block of threads takes a scale tile, 128 rows by 128 columns: a lane VEC values, 32 / VEC lanes a block of 32, two
// 16-byte loads a lane where the width allows (one: 320,000 x 128 bf16 20 us, bound by instructions). Some rows' values are
// loaded before the first of them is used; the scales are gathered in shared memory and written as one piece, zeros for
// blocks and rows that are not there. Where rows do not lie on 16-byte boundaries a lane's values go one by one, but stay
// next to one another: one value a lane made every lane do a whole block's sums (100,000 x 171 62 us for 16).
// Bound by memory: 1,280,000 x 256 bf16 in 122 us, the copy rate; 320,000 x 128 in 19.0 us over tensors in turn, 80 % of it
// (15.3 us repeated on one tensor, which L2 then holds in part).
template <typename T, int VEC, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_mx_quantize(const T *x, long long rows, int width, int tiles, uint8_t *codes,
                                                          uint8_t *scale)
{
    constexpr int kLanes = 32 / VEC, kRow = 4 * kLanes, kRows = kThreads / kRow;  // lanes of a row, rows of a pass
    constexpr int kAhead = 128 / kRows < 8 ? 128 / kRows : ALIGNED ? 8 : 4;
    __shared__ __align__(16) uint8_t bytes[512];
    tcu::grid_dependents_may_start();
    const long long row0 = (long long)(blockIdx.x / (unsigned)tiles) * 128;
    const int tile = (int)(blockIdx.x % (unsigned)tiles), l = threadIdx.x % kLanes, k = threadIdx.x % kRow / kLanes;
    const int blocks = (width + 31) / 32, c = tile * 128 + k * 32 + l * VEC;
    const bool block = tile * 4 + k < blocks;
    const T *x_first = x + row0 * width + c;
    uint8_t *codes_first = codes + (row0 * blocks + tile * 4 + k) * 16 + l * (VEC / 2);
    for (int i = threadIdx.x; i < 128; i += kThreads) ((uint32_t *)bytes)[i] = 0;
    __syncthreads();
    const int r_end = (int)min(128ll, rows - row0), r_first = (int)threadIdx.x / kRow;
    const int r_warp = (int)(threadIdx.x / 32 * 32) / kRow;  // whole warps walk
    for (int p0 = 0; p0 + r_warp < r_end; p0 += kAhead * kRows) {
        Vals<T, VEC> v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = p0 + i * kRows + r_first;
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i].v[e] = from_f<T>(0.f);
            if (r < r_end && c < width)
                load_some<T, VEC, ALIGNED>(x_first + (size_t)(unsigned)r * (unsigned)width, width - c, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = p0 + i * kRows + r_first;
            uint32_t most = most_bits<T, VEC>(v[i]);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
            const uint32_t byte = mx_scale_byte(most);
            const float inv = mx_inverse(byte);
            if (!(block && r < r_end)) continue;
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; e += 2)
                mul2(Pair(to_f<T>(v[i].v[e]), to_f<T>(v[i].v[e + 1])), Pair(inv, inv)).get(f[e], f[e + 1]);
            uint8_t *dst = codes_first + (size_t)(unsigned)r * (unsigned)(blocks * 16);
            if constexpr (VEC == 16) *reinterpret_cast<uint2 *>(dst) = make_uint2(mx_word(f), mx_word(f + 8));
            else if constexpr (VEC == 8) *reinterpret_cast<uint32_t *>(dst) = mx_word(f);
            else *reinterpret_cast<uint16_t *>(dst) = (uint16_t)(mx_byte(f[0], f[1]) | mx_byte(f[2], f[3]) << 8);
            if (l == 0) bytes[(r & 31) * 16 + (r >> 5) * 4 + k] = (uint8_t)byte;
        }
    }
    __syncthreads();
    if (threadIdx.x < 32)
        *reinterpret_cast<uint4 *>(scale + (size_t)blockIdx.x * 512 + threadIdx.x * 16) =
            *reinterpret_cast<const uint4 *>(bytes + threadIdx.x * 16);
}

// ---------------------------------------------------------------- a few tokens
// The weights are read once, by every SM, and multiplied on the CUDA cores. A lane takes a block of 32 weights (16
// bytes), LPR lanes an output column. The tokens lie in shared memory as the E2M1 values themselves in fp16, 80 bytes a
// block with its scale behind them (a stride that spreads eight lanes' 16-byte reads over all banks). Eight products of
// E2M1 values are at most 288 and multiples of 1/4: their sums are exact in fp16. What bounds it is latency.
constexpr int kCell = 80;

struct MxSmallArgs {
    const uint8_t *x, *xs;   // tokens in 4 bits, or null
    const float *h;          // tokens in float32, rounded to 4 bits here
    const uint8_t *w0, *s0, *w1, *s1;
    const __nv_bfloat16 *b0, *b1, *res;
    float *h_out;            // gated
    __nv_bfloat16 *out;
    int M, N, K;
};

__device__ __forceinline__ size_t scale_at(long long row, int k, int tiles)
{
    return (size_t)((row >> 7) * tiles + (k >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (k & 3);
}
__device__ __forceinline__ __half2 two_of(uint32_t byte)
{
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1);
    return *reinterpret_cast<const __half2 *>(&h);
}
__device__ __forceinline__ void widen16(uint4 raw, __half2 (&v)[16])
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = two_of((w[i >> 2] >> (8 * (i & 3))) & 0xffu);
}
// 32 products of a block, without the scales
__device__ __forceinline__ float block_dot(const __half2 (&w)[16], const uint8_t *cell)
{
    float s = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __half2 acc = __float2half2_rn(0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 raw = *reinterpret_cast<const uint4 *>(cell + 32 * half + 16 * j);
            const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = __hfma2(w[8 * half + 4 * j + i], *reinterpret_cast<const __half2 *>(&x[i]), acc);
        }
        const float2 f = __half22float2(acc);
        s += f.x + f.y;
    }
    return s;
}

// y + dot s t for scales s and t: times the smaller one first, which is exact (dot is 0 or 1/4 to 1152, s and t powers of two
// from 2^-127 on), so that neither far scales that cancel nor two large ones beside a small dot or 0 leave float32 between
__device__ __forceinline__ float plus_scaled(float y, float dot, float s, float t)
{
    float lo, hi;  // NaN where either is
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(s), "f"(t));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(hi) : "f"(s), "f"(t));
    return fmaf(dot * lo, hi, y);
}

template <bool GATED, int ACT, int MB, int LPR, int AHEAD>
__global__ void __launch_bounds__(kThreads) k_mx_small(MxSmallArgs a)
{
    extern __shared__ __align__(16) uint8_t cells[];  // [M][blocks]
    const int blocks = (a.K + 31) / 32, tiles = (blocks + 3) / 4;
    const int l = threadIdx.x % LPR, n = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const bool live = n < a.N;
    const size_t wrow = (size_t)min(n, a.N - 1) * blocks * 16;
    // The launch before this one may be what writes the weights, but for the block's down product: the up product is
    // before that, and lets it start only when all that came before itself is done.
    uint4 first = make_uint4(0, 0, 0, 0);
    if (a.h && l < blocks) first = *reinterpret_cast<const uint4 *>(a.w0 + wrow + l * 16);
    tcu::grid_wait();
    tcu::grid_dependents_may_start();
    if (a.x) {
        for (int i = threadIdx.x; i < a.M * blocks; i += kThreads) {
            const int m = i / blocks, k = i - m * blocks;
            __half2 v[16];
            widen16(*reinterpret_cast<const uint4 *>(a.x + (size_t)i * 16), v);
            uint8_t *cell = cells + i * kCell;
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(cell + 16 * j) = *reinterpret_cast<uint4 *>(&v[4 * j]);
            *reinterpret_cast<float *>(cell + 64) = mx_scale_value(a.xs[scale_at(m, k, tiles)]);
        }
    } else {
        // eight lanes a block, four values a lane; whole warps walk, with kAhead blocks' values under way
        constexpr int kAhead = 4, kStep = kThreads / 8;
        const int all = a.M * blocks, q = threadIdx.x % 8;
        const bool whole = a.K % 32 == 0;  // rows are whole blocks, one after the other
        for (int i0 = threadIdx.x / 32 * 4; i0 < all; i0 += kAhead * kStep) {
            float4 f[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int i = i0 + e * kStep + (threadIdx.x & 31) / 8;
                f[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i >= all) continue;
                if (whole) {
                    f[e] = *reinterpret_cast<const float4 *>(a.h + (size_t)i * 32 + q * 4);
                } else {
                    const int m = i / blocks, c = (i - m * blocks) * 32 + q * 4;
                    const float *h = a.h + (size_t)m * a.K + c;
                    if (c < a.K) f[e].x = h[0];
                    if (c + 1 < a.K) f[e].y = h[1];
                    if (c + 2 < a.K) f[e].z = h[2];
                    if (c + 3 < a.K) f[e].w = h[3];
                }
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int i = i0 + e * kStep + (threadIdx.x & 31) / 8;
                uint32_t most = max(max(abs_bits(f[e].x), abs_bits(f[e].y)), max(abs_bits(f[e].z), abs_bits(f[e].w)));
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
                if (i >= all) continue;
                const uint32_t byte = mx_scale_byte(most);
                const float inv = mx_inverse(byte);
                __half2 v[2] = {two_of(mx_byte(f[e].x * inv, f[e].y * inv)), two_of(mx_byte(f[e].z * inv, f[e].w * inv))};
                uint8_t *cell = cells + i * kCell;
                *reinterpret_cast<uint2 *>(cell + 8 * q) = *reinterpret_cast<uint2 *>(v);
                if (q == 0) *reinterpret_cast<float *>(cell + 64) = mx_scale_value(byte);
            }
        }
    }
    __syncthreads();
    float y0[MB], y1[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) y0[m] = y1[m] = 0.f;
    // AHEAD blocks' weights under way
    for (int k0 = l; k0 < blocks; k0 += AHEAD * LPR) {
        uint4 r0[AHEAD], r1[AHEAD];
        uint32_t b0[AHEAD], b1[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const int k = k0 + e * LPR;
            r0[e] = r1[e] = make_uint4(0, 0, 0, 0);
            b0[e] = b1[e] = 0;
            if (k >= blocks) continue;
            const size_t at = scale_at(min(n, a.N - 1), k, tiles);
            r0[e] = e == 0 && k0 == l && a.h ? first : *reinterpret_cast<const uint4 *>(a.w0 + wrow + k * 16);
            b0[e] = a.s0[at];
            if constexpr (GATED) {
                r1[e] = *reinterpret_cast<const uint4 *>(a.w1 + wrow + k * 16);
                b1[e] = a.s1[at];
            }
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const int k = k0 + e * LPR;
            if (k >= blocks) break;
            __half2 w0[16], w1[16];
            widen16(r0[e], w0);
            if constexpr (GATED) widen16(r1[e], w1);
            const float s0 = mx_scale_value(b0[e]), s1 = mx_scale_value(b1[e]);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (m >= a.M) break;
                const uint8_t *cell = cells + (m * blocks + k) * kCell;
                const float sx = *reinterpret_cast<const float *>(cell + 64);
                y0[m] = plus_scaled(y0[m], block_dot(w0, cell), s0, sx);
                if constexpr (GATED) y1[m] = plus_scaled(y1[m], block_dot(w1, cell), s1, sx);
            }
        }
    }
    float m0 = 0.f, m1 = 0.f;  // of token l
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            y0[m] += __shfl_xor_sync(kFull, y0[m], o);
            if constexpr (GATED) y1[m] += __shfl_xor_sync(kFull, y1[m], o);
        }
        if (l == m) m0 = y0[m], m1 = y1[m];
    }
    if (!live || l >= a.M) return;
    if (a.b0) m0 += __bfloat162float(a.b0[n]);
    const size_t at = (size_t)l * a.N + n;
    if constexpr (GATED) {
        if (a.b1) m1 += __bfloat162float(a.b1[n]);
        a.h_out[at] = Act<ACT>::hidden(m0 * Act<ACT>::kGate, m1 * Act<ACT>::kUp);
    } else {
        if (a.res) m0 += __bfloat162float(a.res[at]);
        a.out[at] = __float2bfloat16_rn(m0);
    }
}

// Up to 8 tokens whose cells fill at most 48 KB. Against the tensor cores, whose tiles hold 256 tokens (us, here / there):
// linear 512 -> 2,048, 1 token 1.7 / 3.6, 8 tokens 2.6 / 3.7; 2,048 -> 512, 8 tokens 3.8 / 4.9; 4,096 -> 1,024, 4 tokens 3.8 /
// 6.9. The CUDA cores' time grows with tokens x outputs, the tensor cores' with the width alone: 1,024 -> 4,096, 4 tokens 3.7
// / 4.8, 6 tokens 4.8 / 4.7, 8 tokens 5.5 / 4.7.
constexpr int kFewTokens = 8;
constexpr size_t kFewBytes = 48 * 1024;
bool few(int64_t M, int64_t K) { return M <= kFewTokens && (size_t)(M * mx_blocks(K)) * kCell <= kFewBytes; }
bool few_linear(int64_t M, int64_t N, int64_t K) { return few(M, K) && M * N * K <= (1 << 24) + 8192 * K; }
// A block's, where the hidden values are 12,288 at most: every thread block of the down product rounds all of them. 256 x
// 1,024, 8 tokens 6.9 / 7.5; 512 x 2,048, 4 tokens 6.3 / 8.8, 6 tokens 8.8 / 8.9; 1,024 x 4,096, 2 tokens 9.2 / 12.0.
bool few_block(int64_t M, int64_t E, int64_t F) { return few(M, E) && few(M, F) && M * F <= 12288; }

template <bool GATED, int ACT, int MB, int LPR, int AHEAD>
pmha_status launch_small(const MxSmallArgs &a, cudaStream_t s)
{
    const int per = kThreads / LPR;
    return tcu::launch_overlapping(k_mx_small<GATED, ACT, MB, LPR, AHEAD>, dim3((unsigned)((a.N + per - 1) / per)), kThreads,
                                   (int)((size_t)a.M * mx_blocks(a.K) * kCell), s, a);
}
// As many lanes an output as blocks, up to a warp; longer rows have several blocks' weights under way (4,096 -> 1,024, 1
// token 2.4 us, one at a time 3.1; rows of one block a lane lose by it: 1,024 -> 4,096, 4 tokens 4.6 for 3.7).
template <bool GATED, int ACT, int MB>
pmha_status by_lanes(const MxSmallArgs &a, cudaStream_t s)
{
    const int64_t blocks = mx_blocks(a.K);
    if (blocks <= 8) return launch_small<GATED, ACT, MB, 8, 1>(a, s);
    if (blocks <= 16) return launch_small<GATED, ACT, MB, 16, 1>(a, s);
    if (blocks <= 32) return launch_small<GATED, ACT, MB, 32, 1>(a, s);
    return launch_small<GATED, ACT, MB, 32, GATED ? 2 : 4>(a, s);
}
template <bool GATED, int ACT>
pmha_status small(const MxSmallArgs &a, const char *stage, cudaStream_t s)
{
    StageTimer timer(stage, s);
    if (a.M == 1) return by_lanes<GATED, ACT, 1>(a, s);
    return a.M <= 4 ? by_lanes<GATED, ACT, 4>(a, s) : by_lanes<GATED, ACT, kFewTokens>(a, s);
}

// ---------------------------------------------------------------- checks
pmha_status check_mx(const char *who, const char *name, const pmha_mx *m)
{
    if (m && m->codes && m->scale && aligned(m->codes, 16) && aligned(m->scale, 16)) return PMHA_OK;
    set_error("%s: %s lacks its codes or scales, or they are not 16-byte aligned", who, name);
    return PMHA_ERR_INVALID_ARG;
}
pmha_status check_sizes(const char *who, int64_t rows, int64_t width, int64_t outputs)
{
    if (rows < 0 || rows > ((int64_t)1 << 31) - 1 || width < 1 || width > ((int64_t)1 << 20) || outputs < 1 ||
        outputs > ((int64_t)1 << 20) || width * outputs > (int64_t)1 << 34 ||
        rows * std::max(width, outputs) > (int64_t)1 << 40) {
        set_error("%s: rows %lld must be 0 .. 2^31 - 1, widths %lld and %lld 1 .. 2^20, their product at most 2^34, rows "
                  "times the wider at most 2^40",
                  who, (long long)rows, (long long)width, (long long)outputs);
        return PMHA_ERR_INVALID_ARG;
    }
    return PMHA_OK;
}
Mx mx_of(const pmha_mx &m) { return Mx{(const uint8_t *)m.codes, (const uint8_t *)m.scale}; }
pmha_status linear(const MxLinear &a, const char *stage, cudaStream_t s)
{
    if (!few_linear(a.M, a.N, a.K)) return mx_tc_linear(a, stage, s);
    MxSmallArgs q = {};
    q.x = a.x.codes, q.xs = a.x.scale, q.w0 = a.w.codes, q.s0 = a.w.scale;
    q.b0 = (const __nv_bfloat16 *)a.bias, q.res = (const __nv_bfloat16 *)a.residual, q.out = (__nv_bfloat16 *)a.out;
    q.M = (int)a.M, q.N = (int)a.N, q.K = (int)a.K;
    return small<false, 0>(q, stage, s);
}

pmha_status check_ffn_mx(const char *who, const pmha_ffn_params *p, int64_t rows)
{
    if (!p || p->dtype != PMHA_BF16 || (p->act != PMHA_ACT_SILU && p->act != PMHA_ACT_GELU)) {
        set_error("%s: params is NULL, its dtype is not PMHA_BF16 or its act is unknown", who);
        return PMHA_ERR_INVALID_ARG;
    }
    return check_sizes(who, rows, p->embed_dim, p->hidden_dim);
}
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
// Hidden rows in 4 bits, or those of a few tokens in float32
size_t hidden_bytes(const pmha_ffn_params *p, int64_t rows)
{
    const size_t small = (size_t)std::min<int64_t>(rows, kFewTokens) * (size_t)p->hidden_dim * 4;
    if (few_block(rows, p->embed_dim, p->hidden_dim)) return round256(small);
    return std::max(round256(small),
                    round256(mx_code_bytes(rows, p->hidden_dim)) + round256(mx_scale_bytes(rows, p->hidden_dim)));
}

}  // namespace
}  // namespace pmha

using namespace pmha;

extern "C" {

size_t pmha_mx_code_bytes(int64_t rows, int64_t width)
{
    return check_sizes("pmha_mx_code_bytes", rows, width, 1) == PMHA_OK ? mx_code_bytes(rows, width) : SIZE_MAX;
}
size_t pmha_mx_scale_bytes(int64_t rows, int64_t width)
{
    return check_sizes("pmha_mx_scale_bytes", rows, width, 1) == PMHA_OK ? mx_scale_bytes(rows, width) : SIZE_MAX;
}

pmha_status pmha_mx_quantize(pmha_dtype dtype, int64_t rows, int64_t width, const void *x, const pmha_mx *out,
                             pmha_stream stream)
{
    const char *who = "pmha_mx_quantize";
    pmha_status st = check_rows(who, dtype, rows, width);
    if (st == PMHA_OK) st = check_sizes(who, rows, width, 1);
    if (st != PMHA_OK || rows == 0) return st;
    if ((st = check_mx(who, "out", out)) != PMHA_OK) return st;
    if (!x || !aligned(x, 16)) {
        set_error("%s: x is NULL or not 16-byte aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t nb = (size_t)(rows * width) * bytes_of(dtype), cb = mx_code_bytes(rows, width), sb = mx_scale_bytes(rows, width);
    const Span ins[] = {{x, nb}}, outs[] = {{out->codes, cb}, {out->scale, sb}};
    if (any_overlap(ins, outs)) {
        set_error("%s: an output overlaps an input or another output", who);
        return PMHA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = (cudaStream_t)stream;
    {
        StageTimer timer("mx_quantize", cs);
        const int64_t tiles = (mx_blocks(width) + 3) / 4;
        const unsigned grid = (unsigned)((rows + 127) / 128 * tiles);
        auto launch = [&](auto kern, auto *p) {
            kern<<<grid, kThreads, 0, cs>>>(p, rows, (int)width, (int)tiles, (uint8_t *)out->codes, (uint8_t *)out->scale);
        };
        using B = __nv_bfloat16;
        if (dtype == PMHA_BF16) {
            if (width % 16 == 0) launch(k_mx_quantize<B, 16, true>, (const B *)x);
            else launch(width % 8 == 0 ? k_mx_quantize<B, 8, true> : k_mx_quantize<B, 8, false>, (const B *)x);
        } else {
            if (width % 8 == 0) launch(k_mx_quantize<float, 8, true>, (const float *)x);
            else launch(width % 4 == 0 ? k_mx_quantize<float, 4, true> : k_mx_quantize<float, 4, false>, (const float *)x);
        }
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

pmha_status pmha_mx_linear(int64_t rows, int64_t width, int64_t outputs, const pmha_mx *x, const pmha_mx *weight,
                           const void *bias, const void *residual, void *out, pmha_stream stream)
{
    const char *who = "pmha_mx_linear";
    pmha_status st = check_sizes(who, rows, width, outputs);
    if (st != PMHA_OK || rows == 0) return st;
    if ((st = check_mx(who, "x", x)) != PMHA_OK || (st = check_mx(who, "weight", weight)) != PMHA_OK) return st;
    if (!out || !aligned(out, 16) || !aligned(residual, 16) || !aligned(bias, 2)) {
        set_error("%s: out is NULL, out or residual is not 16-byte aligned, or bias not to its elements", who);
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t ob = (size_t)(rows * outputs) * 2;
    const Span ins[] = {{x->codes, mx_code_bytes(rows, width)}, {x->scale, mx_scale_bytes(rows, width)},
                        {weight->codes, mx_code_bytes(outputs, width)}, {weight->scale, mx_scale_bytes(outputs, width)},
                        {bias, (size_t)outputs * 2}, {residual, ob}};
    const Span outs[] = {{out, ob}};
    if (any_overlap(ins, outs)) {
        set_error("%s: an output overlaps an input or another output", who);
        return PMHA_ERR_INVALID_ARG;
    }
    return linear(MxLinear{mx_of(*x), mx_of(*weight), bias, residual, out, rows, outputs, width}, "mx_linear",
                  (cudaStream_t)stream);
}

size_t pmha_ffn_forward_mx_workspace_size(const pmha_ffn_params *params, int64_t rows)
{
    if (check_ffn_mx("pmha_ffn_forward_mx", params, rows) != PMHA_OK) return SIZE_MAX;
    return rows ? hidden_bytes(params, rows) : 0;
}

pmha_status pmha_ffn_forward_mx(const pmha_ffn_params *params, const pmha_ffn_mx *weights, const pmha_mx *x,
                                const void *residual, int64_t rows, void *out, void *workspace, size_t workspace_bytes,
                                pmha_stream stream)
{
    const char *who = "pmha_ffn_forward_mx";
    pmha_status st = check_ffn_mx(who, params, rows);
    if (st != PMHA_OK || rows == 0) return st;
    const int64_t E = params->embed_dim, F = params->hidden_dim;
    if (!weights) {
        set_error("%s: weights is NULL", who);
        return PMHA_ERR_INVALID_ARG;
    }
    if ((st = check_mx(who, "x", x)) != PMHA_OK || (st = check_mx(who, "wg", &weights->wg)) != PMHA_OK ||
        (st = check_mx(who, "wu", &weights->wu)) != PMHA_OK || (st = check_mx(who, "wd", &weights->wd)) != PMHA_OK)
        return st;
    if (!out || !aligned(out, 16) || !aligned(residual, 16) || !aligned(params->bg, 2) || !aligned(params->bu, 2) ||
        !aligned(params->bd, 2)) {
        set_error("%s: out is NULL, out or residual is not 16-byte aligned, or a bias not to its elements", who);
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t ob = (size_t)(rows * E) * 2, need = hidden_bytes(params, rows);
    const size_t wc = mx_code_bytes(F, E), wsc = mx_scale_bytes(F, E);
    const Span ins[] = {{x->codes, mx_code_bytes(rows, E)}, {x->scale, mx_scale_bytes(rows, E)},
                        {weights->wg.codes, wc}, {weights->wg.scale, wsc}, {weights->wu.codes, wc}, {weights->wu.scale, wsc},
                        {weights->wd.codes, mx_code_bytes(E, F)}, {weights->wd.scale, mx_scale_bytes(E, F)},
                        {params->bg, (size_t)F * 2}, {params->bu, (size_t)F * 2}, {params->bd, (size_t)E * 2}, {residual, ob},
                        {workspace, need}};
    const Span outs[] = {{out, ob}};
    if (any_overlap(ins, outs)) {
        set_error("%s: an output overlaps an input or the workspace", who);
        return PMHA_ERR_INVALID_ARG;
    }
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)) {
        set_error("%s: workspace needs %zu bytes, 256-byte aligned (got %zu at %p)", who, need, workspace_bytes, workspace);
        return PMHA_ERR_WORKSPACE;
    }
    cudaStream_t s = (cudaStream_t)stream;
    if (few_block(rows, E, F)) {
        MxSmallArgs a = {};
        a.x = (const uint8_t *)x->codes, a.xs = (const uint8_t *)x->scale;
        a.w0 = (const uint8_t *)weights->wg.codes, a.s0 = (const uint8_t *)weights->wg.scale;
        a.w1 = (const uint8_t *)weights->wu.codes, a.s1 = (const uint8_t *)weights->wu.scale;
        a.b0 = (const __nv_bfloat16 *)params->bg, a.b1 = (const __nv_bfloat16 *)params->bu;
        a.h_out = (float *)workspace;
        a.M = (int)rows, a.N = (int)F, a.K = (int)E;
        st = params->act == PMHA_ACT_SILU ? small<true, PMHA_ACT_SILU>(a, "ffn_up_mx", s)
                                          : small<true, PMHA_ACT_GELU>(a, "ffn_up_mx", s);
        if (st != PMHA_OK) return st;
        MxSmallArgs d = {};
        d.h = (const float *)workspace;
        d.w0 = (const uint8_t *)weights->wd.codes, d.s0 = (const uint8_t *)weights->wd.scale;
        d.b0 = (const __nv_bfloat16 *)params->bd, d.res = (const __nv_bfloat16 *)residual, d.out = (__nv_bfloat16 *)out;
        d.M = (int)rows, d.N = (int)E, d.K = (int)F;
        return small<false, 0>(d, "ffn_down_mx", s);
    }
    uint8_t *hc = (uint8_t *)workspace, *hs = hc + round256(mx_code_bytes(rows, F));
    st = mx_tc_gated(MxGated{mx_of(*x), mx_of(weights->wg), mx_of(weights->wu), params->bg, params->bu, hc, hs, rows, F, E,
                             params->act},
                     s);
    if (st != PMHA_OK) return st;
    return mx_tc_linear(MxLinear{Mx{hc, hs}, mx_of(weights->wd), params->bd, residual, out, rows, E, F}, "ffn_down_mx", s);
}

}  // extern "C"
