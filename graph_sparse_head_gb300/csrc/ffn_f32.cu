// The float32 block's products on the CUDA cores (the tensor cores would round
// the operands): 128 x 64 or 128 x 128 outputs a block of 256 threads, 8 x 4 or
// 8 x 8 a thread, 16 values of K at a time through two shared-memory buffers,
// the next ones' loads under way while these are multiplied. Sums run in
// ascending K with fused multiply-adds. The gate and up products share their
// tokens' tile, and the epilogues apply the activation, the residual or the
// gradients' arithmetic.
#include "ffn_internal.h"
#include "ffn_math.cuh"

namespace pmha {
namespace {

constexpr int kM = 128, kK = 16, kThreads = 256;

// An operand's element (row, k) lies at row * ld + k (KC: K contiguous) or k * ld + row.
struct Operand {
    const float *p;
    int64_t ld, rows;
};

// acc[b][i][j] += sum over k in [k0, k1) of A[m0 + mrow(i), k] B_b[n0 + ncol(j), k]
template <int NB, int TN, bool AK, bool BK>
struct Tile {
    static constexpr int kN = 16 * TN;
    float as[2][kK][kM + 4];
    float bs[2][NB][kK][kN + 4];

    static __device__ __forceinline__ int mrow(int i) { return (threadIdx.x / 16) * 4 + (i & 3) + (i >> 2) * 64; }
    static __device__ __forceinline__ int ncol(int j) { return (threadIdx.x % 16) * 4 + (j & 3) + (j >> 2) * 64; }

    // R rows x 16 k of an operand: R / 64 float4 a thread, along its contiguous axis
    template <int R, bool KC>
    static __device__ __forceinline__ void fetch(float4 (&v)[R / 64], const Operand &o, int64_t r0, int64_t k0, int64_t k1,
                                                 bool vec)
    {
#pragma unroll
        for (int q = 0; q < R / 64; ++q) {
            const int idx = threadIdx.x + q * kThreads;
            const int64_t r = r0 + (KC ? idx / 4 : (idx % (R / 4)) * 4), k = k0 + (KC ? (idx % 4) * 4 : idx / (R / 4));
            const float *p = o.p + (KC ? r * o.ld + k : k * o.ld + r);
            float e[4] = {0.f, 0.f, 0.f, 0.f};
            if (vec && (KC ? r < o.rows && k + 4 <= k1 : k < k1 && r + 4 <= o.rows)) {
                const float4 f = *reinterpret_cast<const float4 *>(p);
                e[0] = f.x, e[1] = f.y, e[2] = f.z, e[3] = f.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (KC ? r < o.rows && k + i < k1 : k < k1 && r + i < o.rows) e[i] = p[i];
            }
            v[q] = make_float4(e[0], e[1], e[2], e[3]);
        }
    }
    template <int R, bool KC, int P>
    static __device__ __forceinline__ void put(float (&s)[kK][P], const float4 (&v)[R / 64])
    {
#pragma unroll
        for (int q = 0; q < R / 64; ++q) {
            const int idx = threadIdx.x + q * kThreads;
            if constexpr (KC) {
                const int r = idx / 4, k = (idx % 4) * 4;
                s[k][r] = v[q].x, s[k + 1][r] = v[q].y, s[k + 2][r] = v[q].z, s[k + 3][r] = v[q].w;
            } else {
                *reinterpret_cast<float4 *>(&s[idx / (R / 4)][(idx % (R / 4)) * 4]) = v[q];
            }
        }
    }
    static __device__ __forceinline__ bool vectors(const Operand &o)
    {
        return ((uintptr_t)o.p & 15) == 0 && o.ld % 4 == 0;
    }

    __device__ void run(const Operand &A, const Operand (&B)[NB], int64_t m0, int64_t n0, int64_t k0, int64_t k1,
                        float (&acc)[NB][8][TN])
    {
        const bool va = vectors(A) && k0 % 4 == 0;
        bool vb[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) vb[b] = vectors(B[b]) && k0 % 4 == 0;
        float4 ra[kM / 64], rb[NB][kN / 64];
        auto load = [&](int64_t k) {
            fetch<kM, AK>(ra, A, m0, k, k1, va);
#pragma unroll
            for (int b = 0; b < NB; ++b) fetch<kN, BK>(rb[b], B[b], n0, k, k1, vb[b]);
        };
        auto store = [&](int t) {
            put<kM, AK>(as[t], ra);
#pragma unroll
            for (int b = 0; b < NB; ++b) put<kN, BK>(bs[t][b], rb[b]);
        };
        __syncthreads();  // an earlier product's tiles have been read
        load(k0);
        store(0);
        __syncthreads();
        int t = 0;
        for (int64_t k = k0; k < k1; k += kK, t ^= 1) {
            if (k + kK < k1) load(k + kK);
#pragma unroll
            for (int kk = 0; kk < kK; ++kk) {
                float a[8];
                *reinterpret_cast<float4 *>(a) = *reinterpret_cast<const float4 *>(&as[t][kk][(threadIdx.x / 16) * 4]);
                *reinterpret_cast<float4 *>(a + 4) =
                    *reinterpret_cast<const float4 *>(&as[t][kk][64 + (threadIdx.x / 16) * 4]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float e[TN];
#pragma unroll
                    for (int j = 0; j < TN; j += 4)
                        *reinterpret_cast<float4 *>(e + j) =
                            *reinterpret_cast<const float4 *>(&bs[t][b][kk][(threadIdx.x % 16) * 4 + j * 16]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[b][i][j] = __fmaf_rn(a[i], e[j], acc[b][i][j]);
                }
            }
            if (k + kK < k1) {
                store(t ^ 1);
                __syncthreads();
            }
        }
    }
};

#define PMHA_TILE_ORIGIN(T) const int64_t m0 = (int64_t)blockIdx.x * kM, n0 = (int64_t)blockIdx.y * T::kN

// h, or h, dg and du
template <int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads) k_hidden(FfnF32Args a)
{
    using T = Tile<2, 4, true, true>;
    using TD = Tile<1, 4, true, false>;
    __shared__ union U {
        T t;
        TD d;
        __device__ U() {}
    } sh;
    PMHA_TILE_ORIGIN(T);
    float c[2][8][4] = {}, d[1][8][4] = {};
    const Operand B[2] = {{a.wg, a.E, a.F}, {a.wu, a.E, a.F}};
    sh.t.run({a.x, a.E, a.M}, B, m0, n0, 0, a.E, c);
    if constexpr (BWD) {
        const Operand D[1] = {{a.wd, a.F, a.F}};
        sh.d.run({a.dy, a.E, a.M}, D, m0, n0, 0, a.E, d);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m >= a.M || n >= a.F) continue;
            const float g = c[0][i][j] + (a.bg ? a.bg[n] : 0.f), u = c[1][i][j] + (a.bu ? a.bu[n] : 0.f);
            const int64_t at = m * a.F + n;
            if constexpr (BWD) {
                float slope;
                const float act = Act<ACT>::exact(g, &slope);
                a.h[at] = act * u;
                a.du[at] = d[0][i][j] * act;
                a.dg[at] = d[0][i][j] * u * slope;
            } else {
                a.h[at] = Act<ACT>::exact(g) * u;
            }
        }
}

// out = h Wd^T + bd + residual
template <int TN>
__global__ void __launch_bounds__(kThreads) k_down(FfnF32Args a)
{
    using T = Tile<1, TN, true, true>;
    __shared__ T sh;
    PMHA_TILE_ORIGIN(T);
    float c[1][8][TN] = {};
    const Operand B[1] = {{a.wd, a.F, a.E}};
    sh.run({a.h, a.F, a.M}, B, m0, n0, 0, a.F, c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m >= a.M || n >= a.E) continue;
            float v = c[0][i][j] + (a.bd ? a.bd[n] : 0.f);
            if (a.res) v += a.res[m * a.E + n];
            a.out[m * a.E + n] = v;
        }
}

// dx = dg Wg + du Wu
template <int TN>
__global__ void __launch_bounds__(kThreads) k_dx(FfnF32Args a)
{
    using T = Tile<1, TN, true, false>;
    __shared__ T sh;
    PMHA_TILE_ORIGIN(T);
    float c[1][8][TN] = {};
    const Operand G[1] = {{a.wg, a.E, a.E}}, U[1] = {{a.wu, a.E, a.E}};
    sh.run({a.dg, a.F, a.M}, G, m0, n0, 0, a.F, c);
    sh.run({a.du, a.F, a.M}, U, m0, n0, 0, a.F, c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m < a.M && n < a.E) a.out[m * a.E + n] = c[0][i][j];
        }
}

// part[split][what] (+)= {dg, du, h}^T {x, x, dy} over the split's rows; blockIdx.z = split * 3 + what
template <int TN>
__global__ void __launch_bounds__(kThreads) k_dw(FfnF32Args a, float *part, int splits, bool accumulate)
{
    using T = Tile<1, TN, false, false>;
    __shared__ T sh;
    PMHA_TILE_ORIGIN(T);
    const int what = blockIdx.z % 3, split = blockIdx.z / 3;
    const int64_t per = ((a.M + splits - 1) / splits + 3) / 4 * 4, k0 = min(a.M, split * per), k1 = min(a.M, k0 + per);
    float c[1][8][TN] = {};
    const Operand B[1] = {{what == 2 ? a.dy : a.x, a.E, a.E}};
    if (k0 < k1) sh.run({what == 0 ? a.dg : what == 1 ? a.du : a.h, a.F, a.F}, B, m0, n0, k0, k1, c);
    float *dst = part + (int64_t)blockIdx.z * a.F * a.E;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m < a.F && n < a.E) dst[m * a.E + n] = accumulate ? dst[m * a.E + n] + c[0][i][j] : c[0][i][j];
        }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// 128 columns a block where that leaves no SM idle
bool wide(int64_t M, int64_t N, int64_t z = 1) { return N > 64 && ceil_div(M, kM) * ceil_div(N, 128) * z >= num_sms(); }
dim3 grid_of(int64_t M, int64_t N, int bn, int64_t z = 1)
{
    return dim3((unsigned)ceil_div(M, kM), (unsigned)ceil_div(N, bn), (unsigned)z);
}
pmha_status launched()
{
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

}  // namespace

pmha_status ffn_f32_hidden(pmha_act act, const FfnF32Args &a, bool backward, cudaStream_t s)
{
    StageTimer timer(backward ? "ffn_hidden" : "ffn_up", s);
    const dim3 g = grid_of(a.M, a.F, 64);
    if (act == PMHA_ACT_SILU) {
        if (backward) k_hidden<PMHA_ACT_SILU, true><<<g, kThreads, 0, s>>>(a);
        else k_hidden<PMHA_ACT_SILU, false><<<g, kThreads, 0, s>>>(a);
    } else {
        if (backward) k_hidden<PMHA_ACT_GELU, true><<<g, kThreads, 0, s>>>(a);
        else k_hidden<PMHA_ACT_GELU, false><<<g, kThreads, 0, s>>>(a);
    }
    return launched();
}

pmha_status ffn_f32_down(const FfnF32Args &a, cudaStream_t s)
{
    StageTimer timer("ffn_down", s);
    if (wide(a.M, a.E)) k_down<8><<<grid_of(a.M, a.E, 128), kThreads, 0, s>>>(a);
    else k_down<4><<<grid_of(a.M, a.E, 64), kThreads, 0, s>>>(a);
    return launched();
}

pmha_status ffn_f32_dx(const FfnF32Args &a, cudaStream_t s)
{
    StageTimer timer("ffn_dx", s);
    if (wide(a.M, a.E)) k_dx<8><<<grid_of(a.M, a.E, 128), kThreads, 0, s>>>(a);
    else k_dx<4><<<grid_of(a.M, a.E, 64), kThreads, 0, s>>>(a);
    return launched();
}

int ffn_f32_splits(int64_t E, int64_t F, int64_t rows)
{
    const int64_t tiles = 3 * ceil_div(F, kM) * ceil_div(E, 64);
    return (int)std::max<int64_t>(1, std::min<int64_t>({ceil_div((int64_t)num_sms() * 2, tiles), ceil_div(rows, 64), 64}));
}

pmha_status ffn_f32_dw(const FfnF32Args &a, float *part, int splits, bool accumulate, cudaStream_t s)
{
    StageTimer timer("ffn_dw", s);
    if (wide(a.F, a.E, 3 * splits)) k_dw<8><<<grid_of(a.F, a.E, 128, 3 * splits), kThreads, 0, s>>>(a, part, splits, accumulate);
    else k_dw<4><<<grid_of(a.F, a.E, 64, 3 * splits), kThreads, 0, s>>>(a, part, splits, accumulate);
    return launched();
}

}  // namespace pmha
