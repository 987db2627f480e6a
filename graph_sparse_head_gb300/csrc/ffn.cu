// Gated feed-forward block: argument checks, workspace, the order of launches,
// and the small kernels around the products (copies to padded widths,
// transposes, sums).
//
//   h = act(x Wg^T + bg) * (x Wu^T + bu),    y = h Wd^T + bd (+ residual)
//   backward, from dy:  dh = dy Wd,  du = dh act(g),  dg = dh u act'(g),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h, biases column sums.
//
// Rows are taken in blocks of at most kBlock bytes of hidden values, so that
// the workspace stops growing with the rows. Smaller blocks, which stay in L2,
// were measured slower: every launch has its start and drain, and at embed_dim
// 128, 512 hidden, 320,000 rows the backward pass took 638 us with blocks of
// 60 MB, 575 with 120, 532 with 240, 497 with 480 and 456 with one of 980 MB.
#include <math.h>

#include <algorithm>

#include "ffn_internal.h"
#include "ffn_math.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {

constexpr int64_t kBlock = (int64_t)2 << 30;   // bytes of hidden values (h, or h, dg and du) of a block of rows
// Rows from which the forward pass runs as one kernel, whose pairs of SMs take
// 256 rows each through the whole hidden width, while the two products deal
// tiles of that width out too. Measured (us, one kernel / two): 64 x 256 at 100
// rows 6.9 / 8.6, 128 x 512 at 2,000 rows 11.0 / 10.3 and at 10,000 11.4 / 13.4,
// 128 x 1,024 at 4,096 16.3 / 13.1 and at 10,000 16.9 / 17.5, 256 x 1,024 at
// 10,000 22.8 / 21.2 and at 19,000 23.9 / 27.0, 256 x 2,048 at 10,000 37.3 / 31.4 and
// at 19,000 38.7 / 47.9.
int64_t fused_rows(int64_t E, int64_t F)
{
    if (E * F <= 1 << 14) return 1;
    return std::min<int64_t>(16384, F * (E > 128 ? 12 : 8));
}
// rows * E * F up to which a bf16 block's backward pass runs on float32 copies
// and the CUDA cores, without the rounding of the hidden gradients to bf16,
// which few values do not average out. Both wait for launches there: 64 x 128 at
// 1,000 rows 62 us against 55 of the tensor cores, 16 x 16 at 8,192 rows 67
// against 56, and at 32,000 rows 99 against 58. Alone on the device, in a graph: 64 x 128 at 256 rows 27 us
// against 19, 16 x 16 at 8,192 rows 45 against 25.
constexpr int64_t kFewWork = (int64_t)1 << 21;
// The same up to so many values of dx, the array on which the rounding shows most: 128 x 512 at 16 rows costs the
// same (29 us against 31 in a graph), 512 x 1,024 at 2 rows 66 against 41, 1,024 x 4,096 at 2 rows 216 against 128,
// and 2,048 x 2,048 at one row, the worst of those measured, 283 against 111.
constexpr int64_t kFewOut = 2048;

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---------------------------------------------------------------- small kernels

// rows x cols bf16 of pitch `cols` -> pitch out_cols (padding zero, or cut)
__global__ void __launch_bounds__(256) k_repitch(const uint16_t *in, int64_t rows, int cols, int64_t out_rows,
                                                 int out_cols, uint16_t *out)
{
    const int64_t n = out_rows * out_cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / out_cols;
        const int c = (int)(i - r * out_cols);
        out[i] = r < rows && c < cols ? in[r * cols + c] : (uint16_t)0;
    }
}

// Up to seven bf16 arrays as float32
struct Widen {
    const __nv_bfloat16 *in[7];
    float *out[7];
    int64_t n[7];
};
__global__ void __launch_bounds__(256) k_widen(Widen w)
{
    for (int a = 0; a < 7; ++a)
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < w.n[a]; i += (int64_t)gridDim.x * 256)
            w.out[a][i] = __bfloat162float(w.in[a][i]);
}
// out = the sum of `parts` float32 arrays, n apart
template <typename T>
__global__ void __launch_bounds__(256) k_narrow(const float *in, int64_t n, int parts, T *out)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v = 0.f;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) v += in[k * n + i];
        out[i] = from_f<T>(v);
    }
}

struct Transposes {
    const uint16_t *in[3];
    uint16_t *out[3];
    int rows[3], cols[3];
};
// out[z] = in[z] transposed (bf16; rows and columns multiples of 8), 64 x 64
// tiles, 16 bytes a load and store. Three 4,096 x 1,024 weights: 21 us
// (115 with 32 x 32 tiles and 2-byte accesses).
__global__ void __launch_bounds__(256) k_transpose(Transposes t)
{
    __shared__ uint32_t sh[64][33];
    const int z = blockIdx.y, rows = t.rows[z], cols = t.cols[z], across = (cols + 63) / 64;
    const int r0 = blockIdx.x / across * 64, c0 = blockIdx.x % across * 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int idx = threadIdx.x + i * 256, r = idx / 8, u = idx % 8;
        if (r0 + r < rows && c0 + 8 * u < cols) {
            const uint4 v = *reinterpret_cast<const uint4 *>(t.in[z] + (int64_t)(r0 + r) * cols + c0 + 8 * u);
            sh[r][4 * u] = v.x, sh[r][4 * u + 1] = v.y, sh[r][4 * u + 2] = v.z, sh[r][4 * u + 3] = v.w;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int idx = threadIdx.x + i * 256, c = idx / 8, u = idx % 8;
        if (c0 + c < cols && r0 + 8 * u < rows) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = __byte_perm(sh[8 * u + 2 * k][c / 2], sh[8 * u + 2 * k + 1][c / 2], c & 1 ? 0x7632 : 0x5410);
            *reinterpret_cast<uint4 *>(t.out[z] + (int64_t)(c0 + c) * rows + r0 + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Column sums of a float32 block's dg, du and dy over this block of rows, by gridDim.y
// row ranges: out[range][2 F + E] (+)=
struct Sums {
    const float *in[3];
    float *out;
    int cols[3], at[3], width;
    int64_t rows;
    bool accumulate;
};
__global__ void __launch_bounds__(256) k_colsum(Sums s)
{
    __shared__ float sh[8][33];
    const int z = blockIdx.z, cols = s.cols[z], c = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
    if (!s.in[z] || blockIdx.x * 32 >= cols) return;
    const int64_t per = (s.rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per, r1 = min(s.rows, r0 + per);
    const float *in = s.in[z];
    float v = 0.f, w[8] = {};  // eight chains of additions, each an eighth as long
    if (c < cols)
        for (int64_t r = r0 + y; r < r1; r += 64)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r + 8 * i < r1) w[i] += in[(r + 8 * i) * cols + c];
#pragma unroll
    for (int i = 0; i < 8; ++i) v += w[i];
    sh[y][threadIdx.x % 32] = v;
    __syncthreads();
    if (y == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += sh[i][threadIdx.x];
        float *o = s.out + (int64_t)blockIdx.y * s.width + s.at[z] + c;
        *o = s.accumulate ? *o + v : v;
    }
}

struct Finish {
    const float *part;  // [splits][3][F2][E2]
    void *w[3];         // (F, E), (F, E), (E, F) or null
    struct {
        const float *p;  // n rows of partial column sums, ld apart
        int n, ld;
    } sums[3];
    void *b[3];         // (F), (F), (E) or null
    int splits;
    int vec;            // four consecutive gate or up gradients are one aligned piece
    int E, F, E2, F2;   // widths of the gradients and of the products
};
// Parameter gradients from the partial sums, each added in a fixed order.
// 64 x 64 tiles of (F, E), four columns a load; the down weight's is written transposed.
template <typename T>
__global__ void __launch_bounds__(256) k_finish(Finish p)
{
    __shared__ float sh[64][65];
    const int z = blockIdx.z;
    if (z >= 3) {  // biases: 8 columns at a time, 32 threads a column in a fixed order
        const int nf = (p.F + 7) / 8, ne = (p.E + 7) / 8, c8 = threadIdx.x % 8, row = threadIdx.x / 8;
        const int blocks = gridDim.x * gridDim.y;
        for (int t = (z - 3) * blocks + blockIdx.y * gridDim.x + blockIdx.x; t < 2 * nf + ne; t += (gridDim.z - 3) * blocks) {
            const int i = t < nf ? 0 : t < 2 * nf ? 1 : 2, col = (t - i * nf) * 8 + c8;
            const bool in = p.b[i] && col < (i == 2 ? p.E : p.F);
            float v = 0.f;
            if (in)
#pragma unroll 8
                for (int k = row; k < p.sums[i].n; k += 32) v += p.sums[i].p[(int64_t)k * p.sums[i].ld + col];
            sh[row][c8] = v;
            __syncthreads();
            if (row == 0 && in) {
                for (int k = 1; k < 32; ++k) v += sh[k][c8];
                ((T *)p.b[i])[col] = from_f<T>(v);
            }
            __syncthreads();
        }
        return;
    }
    if (!p.w[z]) return;
    const int f0 = blockIdx.y * 64, e0 = blockIdx.x * 64, x = threadIdx.x % 16 * 4, y = threadIdx.x / 16, e = e0 + x;
    const int64_t step = (int64_t)3 * p.F2 * p.E2;
    const float *src = p.part + ((int64_t)z * p.F2 + f0 + y) * p.E2 + e;
    float v[4][4] = {};  // rows y, y + 16, y + 32, y + 48 of the tile
    if (p.E2 % 4 == 0) {
#pragma unroll 4
        for (int k = 0; k < p.splits; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (f0 + y + 16 * i < p.F && e < p.E) {
                    const float4 a = *reinterpret_cast<const float4 *>(src + k * step + (int64_t)(16 * i) * p.E2);
                    v[i][0] += a.x, v[i][1] += a.y, v[i][2] += a.z, v[i][3] += a.w;
                }
    } else {
        for (int k = 0; k < p.splits; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (f0 + y + 16 * i < p.F && e + j < p.E) v[i][j] += src[k * step + (int64_t)(16 * i) * p.E2 + j];
    }
    if (z < 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = f0 + y + 16 * i;
            if (f >= p.F) break;
            T *o = (T *)p.w[z] + (int64_t)f * p.E + e;
            if (p.vec && e < p.E) {
                if constexpr (sizeof(T) == 2)
                    *reinterpret_cast<uint2 *>(o) = make_uint2(tcu::pack_bf16(v[i][0], v[i][1]), tcu::pack_bf16(v[i][2], v[i][3]));
                else
                    *reinterpret_cast<float4 *>(o) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < p.E) o[j] = from_f<T>(v[i][j]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sh[y + 16 * i][x + j] = v[i][j];
    __syncthreads();
    const int f = threadIdx.x % 64;
    for (int i = threadIdx.x / 64; i < 64; i += 4)
        if (e0 + i < p.E && f0 + f < p.F) ((T *)p.w[2])[(int64_t)(e0 + i) * p.F + f0 + f] = from_f<T>(sh[f][i]);
}

// ---------------------------------------------------------------- host side
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round8(int64_t n) { return (n + 7) & ~(int64_t)7; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    if (!a || !b || !an || !bn) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + bn && y < x + an;
}

pmha_status check_ffn(const char *who, const pmha_ffn_params *p, int64_t rows, bool quantized)
{
    if (!p) {
        set_error("%s: params is NULL", who);
        return PMHA_ERR_INVALID_ARG;
    }
    if (p->dtype != PMHA_F32 && p->dtype != PMHA_BF16) {
        set_error("%s: dtype %d is neither PMHA_F32 nor PMHA_BF16", who, (int)p->dtype);
        return PMHA_ERR_INVALID_ARG;
    }
    if (p->act != PMHA_ACT_SILU && p->act != PMHA_ACT_GELU) {
        set_error("%s: act %d is neither PMHA_ACT_SILU nor PMHA_ACT_GELU", who, (int)p->act);
        return PMHA_ERR_INVALID_ARG;
    }
    const int64_t most = 1 << 20;
    if (p->embed_dim < 1 || p->hidden_dim < 1 || p->embed_dim > most || p->hidden_dim > most ||
        p->embed_dim * p->hidden_dim > (int64_t)1 << 31) {
        set_error("%s: embed_dim %lld and hidden_dim %lld must be 1 .. 2^20, their product at most 2^31", who,
                  (long long)p->embed_dim, (long long)p->hidden_dim);
        return PMHA_ERR_INVALID_ARG;
    }
    if (rows < 0 || rows > ((int64_t)1 << 31) - 512 || rows * p->embed_dim > (int64_t)1 << 42) {
        set_error("%s: rows %lld must be 0 .. 2^31 - 512, and rows * embed_dim at most 2^42", who, (long long)rows);
        return PMHA_ERR_INVALID_ARG;
    }
    if (quantized) {
        if (p->dtype != PMHA_BF16) {
            set_error("%s: the parameters must be PMHA_BF16", who);
            return PMHA_ERR_INVALID_ARG;
        }
        if (p->embed_dim % 16 || p->hidden_dim % 8) {
            set_error("%s: embed_dim %lld must be a multiple of 16 and hidden_dim %lld of 8", who,
                      (long long)p->embed_dim, (long long)p->hidden_dim);
            return PMHA_ERR_UNSUPPORTED;
        }
    }
    return PMHA_OK;
}

pmha_status check_weights(const char *who, const pmha_ffn_params *p, bool quantized)
{
    const size_t es = p->dtype == PMHA_BF16 ? 2 : 4;
    if ((!quantized && (!p->wg || !p->wu || !aligned(p->wg, 16) || !aligned(p->wu, 16))) || !p->wd ||
        !aligned(p->wd, 16)) {
        set_error("%s: a weight is NULL or not 16-byte aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    if (!aligned(p->bg, es) || !aligned(p->bu, es) || !aligned(p->bd, es)) {
        set_error("%s: a bias is not aligned to its elements", who);
        return PMHA_ERR_INVALID_ARG;
    }
    return PMHA_OK;
}

pmha_status check_workspace(const char *who, const void *ws, size_t got, size_t need)
{
    if (need && (!ws || got < need || !aligned(ws, 256))) {
        set_error("%s: workspace needs %zu bytes, 256-byte aligned (got %zu at %p)", who, need, got, ws);
        return PMHA_ERR_WORKSPACE;
    }
    return PMHA_OK;
}

// Offsets in the workspace and the block of rows, for widths E2, F2 of the
// products (multiples of 8 for bf16; copies are made where that differs).
struct Plan {
    int64_t E2, F2, R;
    bool padded, fused, small;
    size_t wg, wu, wd, bg, bu, bd;  // padded copies
    size_t x, dy, out;              // padded rows of a block (dy: dy or the residual)
    size_t wgt, wut, wdt;           // transposed weights (backward)
    size_t h, dg, du, part, sums, dy_sums;
    int splits;
    int64_t sum_rows;
    int sum_parts;                  // row ranges of a float32 block's column sums
    bool few;                       // a bf16 block's backward pass in float32: see kFewWork
    int dx_parts;
    size_t f_x, f_dy, f_w[3], f_b[2], f_dx;  // its float32 copies
    size_t total;
};

Plan plan_of(const pmha_ffn_params *p, int64_t rows, bool backward, bool q8)
{
    Plan l = {};
    l.few = p->dtype == PMHA_BF16 && backward &&
            (rows * p->embed_dim <= kFewWork / p->hidden_dim || rows * p->embed_dim <= kFewOut);
    const bool bf16 = p->dtype == PMHA_BF16 && !l.few;  // products on the tensor cores
    const size_t es = bf16 ? 2 : 4;
    l.E2 = bf16 ? round8(p->embed_dim) : p->embed_dim;
    l.F2 = bf16 ? round8(p->hidden_dim) : p->hidden_dim;
    l.small = !backward && ffn_small_supported(p->embed_dim, rows, q8 ? 1 : (int)es);
    if (l.small) l.E2 = p->embed_dim, l.F2 = p->hidden_dim;
    l.padded = l.E2 != p->embed_dim || l.F2 != p->hidden_dim;
    l.fused = bf16 && !l.small && ffn_fused_supported(l.E2, l.F2) && (backward || rows >= fused_rows(l.E2, l.F2));
    const int64_t per_row = l.F2 * (int64_t)es * (backward ? 3 : 1);
    // a whole number of times 256 rows for each pair of SMs, where there are that many
    const int64_t wave = 256 * (int64_t)(num_sms() / 2);
    l.R = std::max<int64_t>(256, kBlock / per_row / 256 * 256);
    if (l.R >= wave) l.R = l.R / wave * wave;
    if (l.fused && !backward && !l.padded) l.R = rows;
    l.R = std::min(l.R, ceil_div(std::max<int64_t>(rows, 1), 256) * 256);
    size_t o = 0;
    auto take = [&](int64_t n) {
        const size_t at = o;
        o += align256((size_t)n * es);
        return at;
    };
    if (l.padded) {
        l.wg = take(l.E2 * l.F2), l.wu = take(l.E2 * l.F2), l.wd = take(l.E2 * l.F2);
        l.bg = take(l.F2), l.bu = take(l.F2), l.bd = take(l.E2);
        l.x = take(l.R * l.E2), l.dy = take(l.R * l.E2), l.out = take(l.R * l.E2);
    }
    if (backward || !l.fused) l.h = take(l.R * l.F2 * (l.small && bf16 ? 2 : 1));  // float32 for a few tokens
    if (backward) {
        l.dg = take(l.R * l.F2), l.du = take(l.R * l.F2);
        if (bf16) l.wgt = take(l.E2 * l.F2), l.wut = take(l.E2 * l.F2), l.wdt = take(l.E2 * l.F2);
        const int64_t block = std::min(l.R, std::max<int64_t>(rows, 1));
        l.splits = bf16 ? ffn_dw_splits(l.E2, l.F2, block) : ffn_f32_splits(l.E2, l.F2, block);
        l.part = o;
        o += align256((size_t)l.splits * 3 * (size_t)(l.E2 * l.F2) * 4);
        // blocks of 32 columns and some 256 rows or more, enough for every SM
        l.sum_parts = (int)std::max<int64_t>(
            1, std::min(ceil_div(block, 256), ceil_div((int64_t)num_sms() * 4, ceil_div(2 * l.F2 + l.E2, 32))));
        // column sums: of a float32 block sum_parts rows of [2 F + E]; of a bf16 block a row of [E] a split, and the
        // hidden kernel's rows of [2][F]
        l.dy_sums = o;
        o += align256((bf16 ? (size_t)l.splits * (size_t)l.E2 : (size_t)l.sum_parts * (size_t)(2 * l.F2 + l.E2)) * 4);
        l.sums = o;
        l.sum_rows = bf16 ? ffn_hidden_parts(block, l.F2) : 0;
        o += align256((size_t)l.sum_rows * (size_t)(2 * l.F2) * 4);
        l.dx_parts = 1;
        if (!bf16) {  // dx in parts, of at most a tile of 64 x 32 for each SM
            l.dx_parts = ffn_f32_dx_parts(l.E2, l.F2, block);
            l.f_dx = take(std::max<int64_t>(l.few ? l.R * l.E2 : 0, (int64_t)num_sms() * 64 * 32));
        }
        if (l.few) {
            l.f_x = take(l.R * l.E2), l.f_dy = take(l.R * l.E2);
            for (size_t &w : l.f_w) w = take(l.E2 * l.F2);
            for (size_t &w : l.f_b) w = take(l.F2);
        }
    }
    l.total = o;
    return l;
}

// Workspace of the most expensive number of rows up to `rows`: a program that
// sizes its workspace once can run every smaller batch in it. The paths for
// fewer rows may take more than the one for many (float32 hidden rows of a few
// tokens, the float32 backward pass of small problems, hidden rows in memory
// below fused_rows()); within a path the size grows with the rows.
size_t most_of(const pmha_ffn_params *p, int64_t rows, bool backward, bool q8)
{
    if (!rows) return 0;
    const int64_t few = std::max(kFewWork / p->hidden_dim, kFewOut) / p->embed_dim;
    size_t n = 0;
    const int64_t tiled = fused_rows(round8(p->embed_dim), round8(p->hidden_dim)) - 1;
    for (const int64_t r : {rows, backward ? few : 1, tiled})
        if (r > 0 && r <= rows) n = std::max(n, plan_of(p, r, backward, q8).total);
    return n;
}

unsigned grid_of(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(ceil_div(n, 256), (int64_t)num_sms() * 16)); }

pmha_status repitch(const void *in, int64_t rows, int64_t cols, int64_t out_rows, int64_t out_cols, void *out,
                    cudaStream_t s)
{
    StageTimer timer("ffn_pad", s);
    k_repitch<<<grid_of(out_rows * out_cols), 256, 0, s>>>((const uint16_t *)in, rows, (int)cols, out_rows,
                                                            (int)out_cols, (uint16_t *)out);
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

#define PMHA_TRY(expr)                             \
    do {                                           \
        const pmha_status _s = (expr);             \
        if (_s != PMHA_OK) return _s;              \
    } while (0)

// Weights and biases in the widths of the products.
pmha_status pad_params(const pmha_ffn_params *p, const Plan &l, char *ws, pmha_ffn_params *q, cudaStream_t s)
{
    *q = *p;
    if (!l.padded) return PMHA_OK;
    const int64_t E = p->embed_dim, F = p->hidden_dim;
    q->embed_dim = l.E2, q->hidden_dim = l.F2;
    PMHA_TRY(repitch(p->wg, F, E, l.F2, l.E2, ws + l.wg, s));
    PMHA_TRY(repitch(p->wu, F, E, l.F2, l.E2, ws + l.wu, s));
    PMHA_TRY(repitch(p->wd, E, F, l.E2, l.F2, ws + l.wd, s));
    q->wg = ws + l.wg, q->wu = ws + l.wu, q->wd = ws + l.wd;
    if (p->bg) {
        PMHA_TRY(repitch(p->bg, 1, F, 1, l.F2, ws + l.bg, s));
        q->bg = ws + l.bg;
    }
    if (p->bu) {
        PMHA_TRY(repitch(p->bu, 1, F, 1, l.F2, ws + l.bu, s));
        q->bu = ws + l.bu;
    }
    if (p->bd) {
        PMHA_TRY(repitch(p->bd, 1, E, 1, l.E2, ws + l.bd, s));
        q->bd = ws + l.bd;
    }
    return PMHA_OK;
}

pmha_status launched()
{
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

// The forward pass, for tokens in the layer type or (q8) in E4M3.
pmha_status forward(const char *who, const pmha_ffn_params *p, const pmha_ffn_quantized *q8, const void *x,
                    const float *x_scale, const void *residual, int64_t rows, void *out, void *workspace,
                    size_t ws_bytes, cudaStream_t s)
{
    const size_t es = p->dtype == PMHA_BF16 ? 2 : 4;
    const int64_t E = p->embed_dim, F = p->hidden_dim;
    if (rows == 0) return PMHA_OK;
    PMHA_TRY(check_weights(who, p, q8 != nullptr));
    if (!x || !out || !aligned(x, 16) || !aligned(out, 16) || !aligned(residual, 16)) {
        set_error("%s: x or out is NULL, or a pointer is not 16-byte aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t ob = (size_t)(rows * E) * es, wb = (size_t)(E * F) * es;
    bool bad = overlap(out, ob, x, q8 ? (size_t)(rows * E) : ob) || overlap(out, ob, residual, ob) ||
               overlap(out, ob, p->wd, wb) || overlap(out, ob, p->bg, (size_t)F * es) ||
               overlap(out, ob, p->bu, (size_t)F * es) || overlap(out, ob, p->bd, (size_t)E * es);
    if (!q8) bad = bad || overlap(out, ob, p->wg, wb) || overlap(out, ob, p->wu, wb);
    else
        bad = bad || overlap(out, ob, q8->wg, wb / 2) || overlap(out, ob, q8->wu, wb / 2) ||
              overlap(out, ob, q8->wg_scale, (size_t)F * 4) || overlap(out, ob, q8->wu_scale, (size_t)F * 4) ||
              overlap(out, ob, x_scale, (size_t)rows * 4);
    if (bad) {
        set_error("%s: out overlaps an input", who);
        return PMHA_ERR_INVALID_ARG;
    }
    const Plan l = plan_of(p, rows, false, q8 != nullptr);
    PMHA_TRY(check_workspace(who, workspace, ws_bytes, most_of(p, rows, false, q8 != nullptr)));
    char *ws = (char *)workspace;
    pmha_ffn_params q;
    PMHA_TRY(pad_params(p, l, ws, &q, s));
    const FfnTc tc{l.E2, l.F2, q.act, q.bg, q.bu, q.bd};
    for (int64_t r = 0; r < rows; r += l.R) {
        const int64_t M = std::min(l.R, rows - r);
        const char *xr = (const char *)x + (size_t)(r * E) * (q8 ? 1 : es);
        const char *rr = residual ? (const char *)residual + (size_t)(r * E) * es : nullptr;
        char *yr = (char *)out + (size_t)(r * E) * es;
        if (p->dtype == PMHA_F32 && !l.small) {
            FfnF32Args a = {};
            a.x = (const float *)xr, a.wg = (const float *)p->wg, a.wu = (const float *)p->wu;
            a.wd = (const float *)p->wd, a.bg = (const float *)p->bg, a.bu = (const float *)p->bu;
            a.bd = (const float *)p->bd, a.res = (const float *)rr, a.h = (float *)(ws + l.h), a.out = (float *)yr;
            a.M = M, a.E = E, a.F = F;
            PMHA_TRY(ffn_f32_hidden(p->act, a, false, s));
            PMHA_TRY(ffn_f32_down(a, s));
            continue;
        }
        const void *xp = xr, *rp = rr;
        void *yp = yr;
        if (l.padded) {
            PMHA_TRY(repitch(xr, M, E, M, l.E2, ws + l.x, s));
            xp = ws + l.x;
            if (rr) {
                PMHA_TRY(repitch(rr, M, E, M, l.E2, ws + l.dy, s));
                rp = ws + l.dy;
            }
            yp = ws + l.out;
        }
        FfnUpArgs up = {};
        up.x = xp, up.wg = q8 ? q8->wg : q.wg, up.wu = q8 ? q8->wu : q.wu;
        if (q8) up.x_scale = x_scale + r, up.wg_scale = q8->wg_scale, up.wu_scale = q8->wu_scale;
        up.M = M;
        up.h = ws + l.h;
        if (l.small) {
            PMHA_TRY(ffn_small_forward(tc, p->dtype == PMHA_F32, up, q.wd, rp, yp, s));
        } else if (l.fused) {
            PMHA_TRY(ffn_fused_forward(tc, up, q.wd, rp, yp, s));
        } else {
            PMHA_TRY(ffn_tc_up(tc, up, s));
            PMHA_TRY(ffn_tc_down(tc, ws + l.h, q.wd, rp, M, yp, s));
        }
        if (l.padded) PMHA_TRY(repitch(ws + l.out, M, l.E2, M, E, yr, s));
    }
    return PMHA_OK;
}

}  // namespace
}  // namespace pmha

using namespace pmha;

extern "C" {

size_t pmha_ffn_forward_workspace_size(const pmha_ffn_params *params, int64_t rows)
{
    if (check_ffn("pmha_ffn_forward", params, rows, false) != PMHA_OK) return SIZE_MAX;
    return most_of(params, rows, false, false);
}

pmha_status pmha_ffn_forward(const pmha_ffn_params *params, const void *x, const void *residual, int64_t rows,
                             void *out, void *workspace, size_t workspace_bytes, pmha_stream stream)
{
    PMHA_TRY(check_ffn("pmha_ffn_forward", params, rows, false));
    return forward("pmha_ffn_forward", params, nullptr, x, nullptr, residual, rows, out, workspace, workspace_bytes,
                   (cudaStream_t)stream);
}

size_t pmha_ffn_forward_quantized_workspace_size(const pmha_ffn_params *params, int64_t rows)
{
    if (check_ffn("pmha_ffn_forward_quantized", params, rows, true) != PMHA_OK) return SIZE_MAX;
    return most_of(params, rows, false, true);
}

pmha_status pmha_ffn_forward_quantized(const pmha_ffn_params *params, const pmha_ffn_quantized *quantized,
                                       const void *x, const float *x_scale, const void *residual, int64_t rows,
                                       void *out, void *workspace, size_t workspace_bytes, pmha_stream stream)
{
    const char *who = "pmha_ffn_forward_quantized";
    PMHA_TRY(check_ffn(who, params, rows, true));
    if (!quantized || !quantized->wg || !quantized->wu || !quantized->wg_scale || !quantized->wu_scale ||
        !aligned(quantized->wg, 16) || !aligned(quantized->wu, 16) || !aligned(quantized->wg_scale, 4) ||
        !aligned(quantized->wu_scale, 4)) {
        set_error("%s: a quantized weight or scale is NULL or not aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    if (rows && (!x_scale || !aligned(x_scale, 4))) {
        set_error("%s: x_scale is NULL or not aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    return forward(who, params, quantized, x, x_scale, residual, rows, out, workspace, workspace_bytes,
                   (cudaStream_t)stream);
}

size_t pmha_ffn_backward_workspace_size(const pmha_ffn_params *params, int64_t rows)
{
    if (check_ffn("pmha_ffn_backward", params, rows, false) != PMHA_OK) return SIZE_MAX;
    return most_of(params, rows, true, false);
}

pmha_status pmha_ffn_backward(const pmha_ffn_params *params, const void *x, const void *dout, int64_t rows, void *dx,
                              const pmha_ffn_grads *grads, void *workspace, size_t workspace_bytes,
                              pmha_stream stream)
{
    const char *who = "pmha_ffn_backward";
    PMHA_TRY(check_ffn(who, params, rows, false));
    const pmha_ffn_params *p = params;
    const size_t es = p->dtype == PMHA_BF16 ? 2 : 4;
    const int64_t E = p->embed_dim, F = p->hidden_dim;
    cudaStream_t s = (cudaStream_t)stream;
    void *gw[3] = {nullptr, nullptr, nullptr}, *gb[3] = {nullptr, nullptr, nullptr};
    if (grads) {
        gw[0] = grads->wg, gw[1] = grads->wu, gw[2] = grads->wd;
        gb[0] = grads->bg, gb[1] = grads->bu, gb[2] = grads->bd;
    }
    const size_t nb[3] = {(size_t)F * es, (size_t)F * es, (size_t)E * es}, wb = (size_t)(E * F) * es,
                 xb = (size_t)(rows * E) * es;
    for (int i = 0; i < 3; ++i)
        if (!aligned(gw[i], es) || !aligned(gb[i], es)) {
            set_error("%s: a gradient is not aligned to its elements", who);
            return PMHA_ERR_INVALID_ARG;
        }
    if (rows == 0) {
        for (int i = 0; i < 3; ++i) {
            if (gw[i]) PMHA_CUDA_TRY(cudaMemsetAsync(gw[i], 0, wb, s));
            if (gb[i]) PMHA_CUDA_TRY(cudaMemsetAsync(gb[i], 0, nb[i], s));
        }
        return PMHA_OK;
    }
    PMHA_TRY(check_weights(who, p, false));
    if (!x || !dout || !aligned(x, 16) || !aligned(dout, 16) || !aligned(dx, 16)) {
        set_error("%s: x or dout is NULL, or a pointer is not 16-byte aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    {
        const void *in[8] = {x, dout, p->wg, p->wu, p->wd, p->bg, p->bu, p->bd};
        const size_t in_n[8] = {xb, xb, wb, wb, wb, nb[0], nb[1], nb[2]};
        const void *o[7] = {dx, gw[0], gw[1], gw[2], gb[0], gb[1], gb[2]};
        const size_t o_n[7] = {xb, wb, wb, wb, nb[0], nb[1], nb[2]};
        bool bad = false;
        for (int i = 0; i < 7; ++i) {
            for (int j = 0; j < 8; ++j) bad = bad || overlap(o[i], o_n[i], in[j], in_n[j]);
            for (int j = 0; j < i; ++j) bad = bad || overlap(o[i], o_n[i], o[j], o_n[j]);
        }
        if (bad) {
            set_error("%s: an output overlaps an input or another output", who);
            return PMHA_ERR_INVALID_ARG;
        }
    }
    const Plan l = plan_of(p, rows, true, false);
    PMHA_TRY(check_workspace(who, workspace, workspace_bytes, most_of(p, rows, true, false)));
    char *ws = (char *)workspace;
    const bool bf16 = p->dtype == PMHA_BF16 && !l.few;
    const bool any_w = gw[0] || gw[1] || gw[2], any_b = gb[0] || gb[1] || gb[2];
    if (!dx && !any_w && !any_b) return PMHA_OK;
    pmha_ffn_params q;
    PMHA_TRY(pad_params(p, l, ws, &q, s));
    const FfnTc tc{l.E2, l.F2, q.act, q.bg, q.bu, q.bd};
    if (bf16) {
        Transposes t = {};
        const int E2 = (int)l.E2, F2 = (int)l.F2;
        t.in[0] = (const uint16_t *)q.wg, t.out[0] = (uint16_t *)(ws + l.wgt), t.rows[0] = F2, t.cols[0] = E2;
        t.in[1] = (const uint16_t *)q.wu, t.out[1] = (uint16_t *)(ws + l.wut), t.rows[1] = F2, t.cols[1] = E2;
        t.in[2] = (const uint16_t *)q.wd, t.out[2] = (uint16_t *)(ws + l.wdt), t.rows[2] = E2, t.cols[2] = F2;
        const unsigned tiles = (unsigned)(ceil_div(E2, 64) * ceil_div(F2, 64));
        StageTimer timer("ffn_transpose", s);
        k_transpose<<<dim3(tiles, 3), 256, 0, s>>>(t);
        PMHA_TRY(launched());
    }
    float *part = (float *)(ws + l.part), *sums = (float *)(ws + l.sums), *dy_sums = (float *)(ws + l.dy_sums);
    if (l.few) {
        q.wg = ws + l.f_w[0], q.wu = ws + l.f_w[1], q.wd = ws + l.f_w[2];
        if (q.bg) q.bg = ws + l.f_b[0];
        if (q.bu) q.bu = ws + l.f_b[1];
    }
    const bool hidden_sums = bf16 && (gb[0] || gb[1]);
    if (hidden_sums)
        PMHA_CUDA_TRY(cudaMemsetAsync(sums, 0, (size_t)l.sum_rows * 2 * (size_t)l.F2 * 4, s));
    bool first = true;
    for (int64_t r = 0; r < rows; r += l.R, first = false) {
        const int64_t M = std::min(l.R, rows - r);
        const void *xr = (const char *)x + (size_t)(r * E) * es, *dyr = (const char *)dout + (size_t)(r * E) * es;
        void *dxr = dx ? (char *)dx + (size_t)(r * E) * es : nullptr, *const dx_out = dxr;
        if (l.few) {  // float32 copies of the rows, and once of the weights
            const void *in[7] = {xr, dyr, p->wg, p->wu, p->wd, p->bg, p->bu};
            const size_t at[7] = {l.f_x, l.f_dy, l.f_w[0], l.f_w[1], l.f_w[2], l.f_b[0], l.f_b[1]};
            const int64_t n[7] = {M * E, M * E, E * F, E * F, E * F, F, F};
            Widen w = {};
            for (int i = 0; i < (first ? 7 : 2); ++i)
                if (in[i]) w.in[i] = (const __nv_bfloat16 *)in[i], w.out[i] = (float *)(ws + at[i]), w.n[i] = n[i];
            xr = ws + l.f_x, dyr = ws + l.f_dy;
            StageTimer timer("ffn_widen", s);
            k_widen<<<grid_of(std::max(E * F, M * E)), 256, 0, s>>>(w);
            PMHA_TRY(launched());
        }
        if (bf16) {
            const void *xp = xr, *dyp = dyr;
            if (l.padded) {
                PMHA_TRY(repitch(xr, M, E, M, l.E2, ws + l.x, s));
                PMHA_TRY(repitch(dyr, M, E, M, l.E2, ws + l.dy, s));
                xp = ws + l.x, dyp = ws + l.dy;
            }
            FfnHiddenArgs hid = {xp, dyp, q.wg, q.wu, ws + l.wdt, M, ws + l.h, ws + l.dg, ws + l.du,
                                 hidden_sums ? sums : nullptr};
            void *dxp = !dx ? nullptr : l.padded ? ws + l.out : dxr;
            if (l.fused) PMHA_TRY(ffn_fused_backward(tc, hid, ws + l.wgt, ws + l.wut, dxp, s));
            else PMHA_TRY(ffn_tc_hidden(tc, hid, s));
            if (dx) {
                if (!l.fused || !ffn_fused_dx(l.E2))
                    PMHA_TRY(ffn_tc_dx(tc, ws + l.dg, ws + l.du, ws + l.wgt, ws + l.wut, M, dxp, s));
                if (l.padded) PMHA_TRY(repitch(ws + l.out, M, l.E2, M, E, dxr, s));
            }
            if (any_w || gb[2]) {
                FfnDwArgs d = {ws + l.dg, ws + l.du, ws + l.h, xp, dyp, M, part, gb[2] ? dy_sums : nullptr,
                               gw[0] || gw[1], gw[2] || gb[2], !first, l.splits};
                PMHA_TRY(ffn_tc_dw(tc, d, s));
            }
        } else {
            const bool sum_dx = dx && (l.few || l.dx_parts > 1);
            if (sum_dx) dxr = ws + l.f_dx;
            FfnF32Args a = {};
            a.x = (const float *)xr, a.dy = (const float *)dyr, a.wg = (const float *)q.wg;
            a.wu = (const float *)q.wu, a.wd = (const float *)q.wd, a.bg = (const float *)q.bg;
            a.bu = (const float *)q.bu, a.h = (float *)(ws + l.h), a.dg = (float *)(ws + l.dg);
            a.du = (float *)(ws + l.du), a.out = (float *)dxr, a.M = M, a.E = E, a.F = F;
            PMHA_TRY(ffn_f32_hidden(p->act, a, true, s));
            if (dx) PMHA_TRY(ffn_f32_dx(a, l.dx_parts, s));
            if (any_w) PMHA_TRY(ffn_f32_dw(a, part, l.splits, !first, s));
            if (any_b) {
                Sums c = {};
                c.in[0] = a.dg, c.in[1] = a.du, c.in[2] = a.dy;
                c.out = dy_sums;
                c.cols[0] = c.cols[1] = (int)F, c.cols[2] = (int)E;
                c.at[1] = (int)F, c.at[2] = (int)(2 * F), c.width = (int)(2 * F + E);
                c.rows = M, c.accumulate = !first;
                StageTimer timer("ffn_bias_sums", s);
                k_colsum<<<dim3((unsigned)ceil_div(std::max(E, F), 32), (unsigned)l.sum_parts, 3), 256, 0, s>>>(c);
                PMHA_TRY(launched());
            }
            if (sum_dx) {
                StageTimer timer("ffn_dx_sum", s);
                const float *in = (const float *)dxr;
                if (l.few) k_narrow<<<grid_of(M * E), 256, 0, s>>>(in, M * E, l.dx_parts, (__nv_bfloat16 *)dx_out);
                else k_narrow<<<grid_of(M * E), 256, 0, s>>>(in, M * E, l.dx_parts, (float *)dx_out);
                PMHA_TRY(launched());
            }
        }
    }
    if (any_w || any_b) {
        Finish f = {};
        f.part = part, f.splits = l.splits;
        for (int i = 0; i < 3; ++i) {
            const bool hidden = bf16 && i < 2;
            f.sums[i].p = hidden ? sums + i * l.F2 : bf16 ? dy_sums : dy_sums + i * l.F2;
            f.sums[i].n = hidden ? (int)l.sum_rows : bf16 ? l.splits : l.sum_parts;
            f.sums[i].ld = (int)(hidden ? 2 * l.F2 : bf16 ? l.E2 : 2 * l.F2 + l.E2);
        }
        f.E = (int)E, f.F = (int)F, f.E2 = (int)l.E2, f.F2 = (int)l.F2;
        for (int i = 0; i < 3; ++i) f.w[i] = gw[i], f.b[i] = gb[i];
        f.vec = E % 4 == 0 && aligned(gw[0], 4 * es) && aligned(gw[1], 4 * es);
        const int64_t tiles = ceil_div(E, 64) * ceil_div(F, 64), columns8 = 2 * ceil_div(F, 8) + ceil_div(E, 8);
        const dim3 grid((unsigned)ceil_div(E, 64), (unsigned)ceil_div(F, 64),
                        3 + (unsigned)std::min<int64_t>(ceil_div(columns8, tiles), 64));
        StageTimer timer("ffn_grads", s);
        if (p->dtype == PMHA_BF16) k_finish<__nv_bfloat16><<<grid, 256, 0, s>>>(f);
        else k_finish<float><<<grid, 256, 0, s>>>(f);
        PMHA_TRY(launched());
    }
    return PMHA_OK;
}

}  // extern "C"
