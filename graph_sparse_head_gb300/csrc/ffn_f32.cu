// The float32 block's products on the CUDA cores (the tensor cores would round
// the operands): 64 x 32 to 128 x 128 outputs a block of 256 threads (the
// largest tiles that leave no SM idle), 16 values of K at a time through two shared-memory buffers,
// the next ones' loads under way while these are multiplied. Sums run in
// ascending K with fused multiply-adds, by pieces of 256 where registers allow. The gate and up products share their
// tokens' tile, and the epilogues apply the activation, the residual or the
// gradients' arithmetic. 4,001 x 64 x 171: 22.7 us for both launches, whose 3 to
// 6 steps of K wait for their loads; 5,000 x 256 x 1,024: 276 us (28 TFLOP/s).
#include "ffn_internal.h"
#include "ffn_math.cuh"

namespace pmha {
namespace {

constexpr int kThreads = 256;

// An operand's element (row, k) lies at row * ld + k (KC: K contiguous) or k * ld + row.
struct Operand {
    const float *p;
    int64_t ld, rows;
};

// acc[b][i][j] += sum over k in [k0, k1) of A[m0 + mrow(i), k] B_b[n0 + ncol(j), k]
// TM x TN outputs a thread and operand.
template <int NB, int TM, int TN, bool AK, bool BK>
struct Tile {
    static constexpr int kM = 16 * TM, kN = 16 * TN, kK = TM == 4 ? 32 : 16;  // small tiles wait for loads, not for sums
    float as[2][kK][kM + 4];
    float bs[2][NB][kK][kN + 4];

    static __device__ __forceinline__ int mrow(int i) { return (threadIdx.x / 16) * 4 + (i & 3) + (i >> 2) * 64; }
    static __device__ __forceinline__ int ncol(int j)
    {
        return TN == 2 ? (threadIdx.x % 16) * 2 + j : (threadIdx.x % 16) * 4 + (j & 3) + (j >> 2) * 64;
    }

    // R rows x kK of an operand, float4 by float4 along its contiguous axis
    template <int R>
    static constexpr int kPieces = R * kK / 4 / kThreads;
    template <int R, bool KC>
    static __device__ __forceinline__ void fetch(float4 (&v)[kPieces<R>], const Operand &o, int64_t r0, int64_t k0, int64_t k1,
                                                 bool vec)
    {
#pragma unroll
        for (int q = 0; q < kPieces<R>; ++q) {
            const int idx = threadIdx.x + q * kThreads;
            const int64_t r = r0 + (KC ? idx / (kK / 4) : (idx % (R / 4)) * 4), k = k0 + (KC ? (idx % (kK / 4)) * 4 : idx / (R / 4));
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
    static __device__ __forceinline__ void put(float (&s)[kK][P], const float4 (&v)[kPieces<R>])
    {
#pragma unroll
        for (int q = 0; q < kPieces<R>; ++q) {
            const int idx = threadIdx.x + q * kThreads;
            if constexpr (KC) {
                const int r = idx / (kK / 4), k = (idx % (kK / 4)) * 4;
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

    template <typename S>
    static __device__ __forceinline__ float (&sums_of(S &folded, float (&acc)[NB][TM][TN]))[NB][TM][TN]
    {
        if constexpr (kFolds) return folded;
        else return acc;
    }
    // A sum in ascending order is off by some sqrt(K) roundings of its running value: where there are registers for
    // a second set of sums, `c` takes kFold values of K and is folded into `acc`. The larger tiles take K at once.
    static constexpr bool kFolds = NB == 1 ? TM * TN < 64 : TN == 2;
    static constexpr int64_t kFold = 256;
    __device__ void run(const Operand &A, const Operand (&B)[NB], int64_t m0, int64_t n0, int64_t k0, int64_t k1,
                        float (&acc)[NB][TM][TN])
    {
        float folded[kFolds ? NB : 1][kFolds ? TM : 1][kFolds ? TN : 1];
        float(&c)[NB][TM][TN] = sums_of(folded, acc);
        auto clear = [&]() {
#pragma unroll
            for (auto &operand : folded)
#pragma unroll
                for (auto &row : operand)
#pragma unroll
                    for (float &v : row) v = 0.f;
        };
        auto fold = [&]() {
            if constexpr (kFolds) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[b][i][j] += folded[b][i][j];
                clear();
            }
        };
        clear();
        const bool va = vectors(A) && k0 % 4 == 0;
        bool vb[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) vb[b] = vectors(B[b]) && k0 % 4 == 0;
        float4 ra[kPieces<kM>], rb[NB][kPieces<kN>];
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
                float a[TM];
#pragma unroll
                for (int i = 0; i < TM; i += 4)
                    *reinterpret_cast<float4 *>(a + i) =
                        *reinterpret_cast<const float4 *>(&as[t][kk][(threadIdx.x / 16) * 4 + i * 16]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float e[TN];
                    if constexpr (TN == 2) {
                        *reinterpret_cast<float2 *>(e) =
                            *reinterpret_cast<const float2 *>(&bs[t][b][kk][(threadIdx.x % 16) * 2]);
                    } else {
#pragma unroll
                        for (int j = 0; j < TN; j += 4)
                            *reinterpret_cast<float4 *>(e + j) =
                                *reinterpret_cast<const float4 *>(&bs[t][b][kk][(threadIdx.x % 16) * 4 + j * 16]);
                    }
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) c[b][i][j] = __fmaf_rn(a[i], e[j], c[b][i][j]);
                }
            }
            if (k + kK < k1) {
                store(t ^ 1);
                __syncthreads();
            }
            if ((k - k0) % kFold == kFold - kK) fold();
        }
        fold();
    }
};

#define PMHA_TILE_ORIGIN(T) const int64_t m0 = (int64_t)blockIdx.x * T::kM, n0 = (int64_t)blockIdx.y * T::kN

// h, or h, dg and du
template <int TM, int TN, int ACT, bool BWD>
__global__ void __launch_bounds__(kThreads) k_hidden(FfnF32Args a)
{
    using T = Tile<2, TM, TN, true, true>;
    using TD = Tile<1, TM, TN, true, false>;
    __shared__ union U {
        T t;
        TD d;
        __device__ U() {}
    } sh;
    PMHA_TILE_ORIGIN(T);
    float c[2][TM][TN] = {}, d[1][TM][TN] = {};
    const Operand B[2] = {{a.wg, a.E, a.F}, {a.wu, a.E, a.F}};
    sh.t.run({a.x, a.E, a.M}, B, m0, n0, 0, a.E, c);
    if constexpr (BWD) {
        const Operand D[1] = {{a.wd, a.F, a.F}};
        sh.d.run({a.dy, a.E, a.M}, D, m0, n0, 0, a.E, d);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
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
template <int TM, int TN>
__global__ void __launch_bounds__(kThreads) k_down(FfnF32Args a)
{
    using T = Tile<1, TM, TN, true, true>;
    __shared__ T sh;
    PMHA_TILE_ORIGIN(T);
    float c[1][TM][TN] = {};
    const Operand B[1] = {{a.wd, a.F, a.E}};
    sh.run({a.h, a.F, a.M}, B, m0, n0, 0, a.F, c);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m >= a.M || n >= a.E) continue;
            float v = c[0][i][j] + (a.bd ? a.bd[n] : 0.f);
            if (a.res) v += a.res[m * a.E + n];
            a.out[m * a.E + n] = v;
        }
}

// dx = dg Wg + du Wu, over the hidden columns of part blockIdx.z of `parts`
template <int TM, int TN>
__global__ void __launch_bounds__(kThreads) k_dx(FfnF32Args a, int parts)
{
    using T = Tile<1, TM, TN, true, false>;
    __shared__ T sh;
    PMHA_TILE_ORIGIN(T);
    float c[1][TM][TN] = {};
    const Operand G[1] = {{a.wg, a.E, a.E}}, U[1] = {{a.wu, a.E, a.E}};
    const int64_t per = ((a.F + parts - 1) / parts + 3) / 4 * 4, k0 = min(a.F, blockIdx.z * per), k1 = min(a.F, k0 + per);
    if (k0 < k1) {
        sh.run({a.dg, a.F, a.M}, G, m0, n0, k0, k1, c);
        sh.run({a.du, a.F, a.M}, U, m0, n0, k0, k1, c);
    }
    float *out = a.out + blockIdx.z * a.M * a.E;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m < a.M && n < a.E) out[m * a.E + n] = c[0][i][j];
        }
}

// part[split][what] (+)= {dg, du, h}^T {x, x, dy} over the split's rows; blockIdx.z = split * 3 + what
template <int TM, int TN>
__global__ void __launch_bounds__(kThreads) k_dw(FfnF32Args a, float *part, int splits, bool accumulate)
{
    using T = Tile<1, TM, TN, false, false>;
    __shared__ T sh;
    PMHA_TILE_ORIGIN(T);
    const int what = blockIdx.z % 3, split = blockIdx.z / 3;
    const int64_t per = ((a.M + splits - 1) / splits + 3) / 4 * 4, k0 = min(a.M, split * per), k1 = min(a.M, k0 + per);
    float c[1][TM][TN] = {};
    const Operand B[1] = {{what == 2 ? a.dy : a.x, a.E, a.E}};
    if (k0 < k1) sh.run({what == 0 ? a.dg : what == 1 ? a.du : a.h, a.F, a.F}, B, m0, n0, k0, k1, c);
    float *dst = part + (int64_t)blockIdx.z * a.F * a.E;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t m = m0 + T::mrow(i), n = n0 + T::ncol(j);
            if (m < a.F && n < a.E) dst[m * a.E + n] = accumulate ? dst[m * a.E + n] + c[0][i][j] : c[0][i][j];
        }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// f(TM, TN tag, grid): the largest tile with a block for every SM, at most `most` columns; else the smallest
template <int TM_, int TN_>
struct Shape {
    static constexpr int TM = TM_, TN = TN_;
};
template <int MOST, typename L>
void with_tile(int64_t M, int64_t N, int64_t z, L f)
{
    auto grid = [&](int tm, int tn) { return dim3((unsigned)ceil_div(M, 16 * tm), (unsigned)ceil_div(N, 16 * tn), (unsigned)z); };
    auto enough = [&](int tm, int tn) { return ceil_div(M, 16 * tm) * ceil_div(N, 16 * tn) * z >= num_sms() && N > 8 * tn; };
    if constexpr (MOST >= 8)
        if (enough(8, 8)) return f(Shape<8, 8>(), grid(8, 8));
    if (enough(8, 4)) return f(Shape<8, 4>(), grid(8, 4));
    if (enough(4, 4)) return f(Shape<4, 4>(), grid(4, 4));
    f(Shape<4, 2>(), grid(4, 2));
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
    with_tile<4>(a.M, a.F, 1, [&](auto t, dim3 g) {
        using S = decltype(t);
        if (act == PMHA_ACT_SILU) {
            if (backward) k_hidden<S::TM, S::TN, PMHA_ACT_SILU, true><<<g, kThreads, 0, s>>>(a);
            else k_hidden<S::TM, S::TN, PMHA_ACT_SILU, false><<<g, kThreads, 0, s>>>(a);
        } else {
            if (backward) k_hidden<S::TM, S::TN, PMHA_ACT_GELU, true><<<g, kThreads, 0, s>>>(a);
            else k_hidden<S::TM, S::TN, PMHA_ACT_GELU, false><<<g, kThreads, 0, s>>>(a);
        }
    });
    return launched();
}

pmha_status ffn_f32_down(const FfnF32Args &a, cudaStream_t s)
{
    StageTimer timer("ffn_down", s);
    with_tile<8>(a.M, a.E, 1, [&](auto t, dim3 g) {
        using S = decltype(t);
        k_down<S::TM, S::TN><<<g, kThreads, 0, s>>>(a);
    });
    return launched();
}

int ffn_f32_dx_parts(int64_t E, int64_t F, int64_t rows)
{
    // pieces of 64 hidden columns or more, until every SM has a tile of 64 x 32 (512 x 1,024, 2 rows: 73 -> 14 us)
    return (int)std::max<int64_t>(1, std::min(ceil_div(F, 64), num_sms() / (ceil_div(rows, 64) * ceil_div(E, 32))));
}

pmha_status ffn_f32_dx(const FfnF32Args &a, int parts, cudaStream_t s)
{
    StageTimer timer("ffn_dx", s);
    with_tile<8>(a.M, a.E, parts, [&](auto t, dim3 g) {
        using S = decltype(t);
        k_dx<S::TM, S::TN><<<g, kThreads, 0, s>>>(a, parts);
    });
    return launched();
}

int ffn_f32_splits(int64_t E, int64_t F, int64_t rows)
{
    const int64_t tiles = 3 * ceil_div(F, 128) * ceil_div(E, 64);
    return (int)std::max<int64_t>(1, std::min<int64_t>({ceil_div((int64_t)num_sms() * 2, tiles), ceil_div(rows, 64), 64}));
}

pmha_status ffn_f32_dw(const FfnF32Args &a, float *part, int splits, bool accumulate, cudaStream_t s)
{
    StageTimer timer("ffn_dw", s);
    with_tile<8>(a.F, a.E, 3 * splits, [&](auto t, dim3 g) {
        using S = decltype(t);
        k_dw<S::TM, S::TN><<<g, kThreads, 0, s>>>(a, part, splits, accumulate);
    });
    return launched();
}

}  // namespace pmha
