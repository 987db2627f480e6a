// Clipping of many gradient tensors by their global norm:
//   norm = sqrt(sum of g^2 over all tensors),  out = g * min(1, max_norm / (norm + 1e-6)).
//
// Two passes, bound by memory: each block sums the squares of its run of chunks
// (64 KB each) and leaves one partial sum; the scaling pass has every block add
// the partial sums (a few KB from L2) in the same order, so all blocks hold the
// same norm without a launch in between, and walks its run backwards, because
// the last chunks read are the ones still in L2. The table of
// tensors travels in the kernel's parameters, so that nothing is copied, no
// host array has to outlive the call, and a captured graph holds its own. 384
// tensors, 252 MB: 137 us in a graph; launched alone the squares take 58 (4.3 TB/s) and
// the scaling, which reads and writes, 90.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "pmha_internal.h"

namespace pmha {
namespace {

constexpr int kThreads = 512;
constexpr int kBatch = 512;       // tensors of one launch: a table of 12 KB of parameters
constexpr int kChunkBytes = 65536;  // what a block takes at a time
// After so many chunks a thread's sums, of up to 128 squares, go on in double: equal values, whose additions
// are all off to the same side, leave the norm within 2^-19. (One chain over the run was off by 3e-5 at 4,000.)
constexpr uint32_t kFoldChunks = 2;
constexpr int kBlocksPerSm = 3;   // all resident at 40 registers a thread (32 bytes of it spilled)
constexpr int kMaxBlocks = 1024;  // partial sums of one launch
constexpr unsigned kFull = 0xffffffffu;

// Squares of float32 values span twice its exponents. Each value goes, by its
// size, into one of three sums: as it is, scaled up by 2^80, or down by 2^-80
// (powers of two: exact), each of which neither overflows nor loses small
// squares; the three meet in double.
constexpr float kSmall = 9.094947e-13f, kBig = 1.0995116e12f;  // 2^-40, 2^40
constexpr float kUp = 1.2089258e24f, kDown = 8.2718061e-25f;   // 2^80, 2^-80

template <int N>
struct TableOf {
    const void *g[N];
    void *out[N];
    uint32_t first[N + 1];  // first chunk of each tensor
    uint32_t last_n[N];     // values of its last chunk; top bit: bf16
    int n;
};
using Table = TableOf<kBatch>;
// Tensors of a short table, whose launches carry 0.8 KB of parameters instead of
// 12: 16 tensors 18.5 -> 16.7 us.
constexpr int kShort = 32;

struct Sums {
    float mid, big, small;
};

__device__ __forceinline__ bool is_mid(float g)
{
    const float t = fabsf(g);
    return (t >= kSmall || t == 0.f) && t <= kBig;
}
__device__ __forceinline__ void add_square(Sums &s, float g)
{
    const float t = fabsf(g);
    if (t >= kSmall && t <= kBig) s.mid = fmaf(g, g, s.mid);
    else if (t < kSmall) s.small = fmaf(g * kUp, g * kUp, s.small);
    else s.big = fmaf(g * kDown, g * kDown, s.big);  // infinities and NaN too
}

// chunk -> tensor: the last i with first[i] <= c
template <int N>
__device__ __forceinline__ int tensor_of(const TableOf<N> &t, uint32_t c)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (t.first[m] <= c) lo = m;
        else hi = m;
    }
    return lo;
}

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

constexpr int kInFlight = 4;  // 16-byte loads of a thread before their values are used

template <typename T>
__device__ __forceinline__ void sum_run(const T *g, int n, Sums &s)
{
    constexpr int V = 16 / sizeof(T), kStep = kThreads * V;
    int i0 = 0;
    if (((uintptr_t)g & 15) == 0) {
        i0 = n / V * V;
        for (int i = threadIdx.x * V; i < i0; i += kInFlight * kStep) {
            uint4 raw[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                raw[u] = i + u * kStep < i0 ? *reinterpret_cast<const uint4 *>(g + i + u * kStep) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                T v[V];
                *reinterpret_cast<uint4 *>(v) = raw[u];
                bool mid = true;
#pragma unroll
                for (int k = 0; k < V; ++k) mid &= is_mid(to_f<T>(v[k]));
                if (mid) {  // the usual case, without a branch a value
#pragma unroll
                    for (int k = 0; k < V; ++k) s.mid = fmaf(to_f<T>(v[k]), to_f<T>(v[k]), s.mid);
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k) add_square(s, to_f<T>(v[k]));
                }
            }
        }
    }
    for (int i = i0 + threadIdx.x; i < n; i += kThreads) add_square(s, to_f<T>(g[i]));
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T *g, T *out, int n, float c)
{
    constexpr int V = 16 / sizeof(T), kStep = kThreads * V;
    int i0 = 0;
    if ((((uintptr_t)g | (uintptr_t)out) & 15) == 0) {
        i0 = n / V * V;
        for (int i = threadIdx.x * V; i < i0; i += kInFlight * kStep) {
            uint4 raw[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (i + u * kStep < i0) raw[u] = *reinterpret_cast<const uint4 *>(g + i + u * kStep);
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (i + u * kStep >= i0) break;
                T v[V];
                *reinterpret_cast<uint4 *>(v) = raw[u];
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = from_f<T>(to_f<T>(v[k]) * c);
                *reinterpret_cast<uint4 *>(out + i + u * kStep) = *reinterpret_cast<uint4 *>(v);
            }
        }
    }
    for (int i = i0 + threadIdx.x; i < n; i += kThreads) out[i] = from_f<T>(to_f<T>(g[i]) * c);
}

// Sum over the block of a double, the same in every thread and in every block.
__device__ __forceinline__ double block_sum(double v, double *sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sh[i];
    return v;
}

// This block's run of chunks: [first, last) of `chunks`, in equal parts.
__device__ __forceinline__ uint32_t run_start(uint32_t chunks, uint32_t block)
{
    return (uint32_t)((uint64_t)chunks * block / gridDim.x);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_grad_squares(const __grid_constant__ TableOf<N> t, double *part)
{
    __shared__ double sh[kThreads / 32];
    const uint32_t chunks = t.first[t.n], last = run_start(chunks, blockIdx.x + 1);
    uint32_t c = run_start(chunks, blockIdx.x);
    double v = 0.0;
    if (c < last)
        for (int i = tensor_of(t, c); c < last;) {
            const uint32_t first = t.first[i], end = min(min(last, t.first[i + 1]), c + kFoldChunks);
            const bool bf16 = t.last_n[i] >> 31, whole = end < t.first[i + 1];  // its last chunk is not in this piece
            const int es = bf16 ? 2 : 4, per = kChunkBytes / es;
            const int n = (int)(end - c - 1) * per + (whole ? per : (int)(t.last_n[i] & 0x7fffffffu));
            const char *g = (const char *)t.g[i] + (size_t)(c - first) * kChunkBytes;
            Sums s = {0.f, 0.f, 0.f};
            if (bf16) sum_run((const __nv_bfloat16 *)g, n, s);
            else sum_run((const float *)g, n, s);
            v += (double)s.mid;
            if (s.small != 0.f) v += (double)s.small / ((double)kUp * (double)kUp);
            if (s.big != 0.f) v += (double)s.big / ((double)kDown * (double)kDown);
            c = end;
            i += !whole;
        }
    const double sum = block_sum(v, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    k_grad_scale(const __grid_constant__ TableOf<N> t, const double *__restrict__ part, int n_part, float max_norm,
                 float *norm_out)
{
    __shared__ double sh[kThreads / 32];
    double v = 0.0;
    for (int i = threadIdx.x; i < n_part; i += kThreads) v += part[i];
    const double norm = sqrt(block_sum(v, sh));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    const double ratio = (double)max_norm / (norm + 1e-6);
    const float c = ratio > 1.0 ? 1.f : (float)ratio;  // a NaN stays
    const uint32_t chunks = t.first[t.n], first = run_start(chunks, blockIdx.x);
    uint32_t end = run_start(chunks, blockIdx.x + 1);
    if (first < end)
        for (int i = tensor_of(t, end - 1); end > first; --i) {
            // chunks [from, end) of tensor i, from the last one down
            const uint32_t from = max(first, t.first[i]);
            if (!(c == 1.f && t.out[i] == t.g[i])) {  // else in place and nothing to scale
                const bool bf16 = t.last_n[i] >> 31;
                const int per = kChunkBytes / (bf16 ? 2 : 4);
                for (uint32_t ch = end; ch-- > from;) {
                    const size_t at = (size_t)(ch - t.first[i]) * kChunkBytes;
                    const int n = ch + 1 < t.first[i + 1] ? per : (int)(t.last_n[i] & 0x7fffffffu);
                    const char *g = (const char *)t.g[i] + at;
                    char *o = (char *)t.out[i] + at;
                    if (bf16) scale_chunk((const __nv_bfloat16 *)g, (__nv_bfloat16 *)o, n, c);
                    else scale_chunk((const float *)g, (float *)o, n, c);
                }
            }
            end = from;
        }
}

size_t part_bytes(int64_t n_tensors)
{
    // batches are cut by tensors and by chunks (32-bit), so a call may take a few more than n / kBatch
    return (size_t)((n_tensors + kBatch - 1) / kBatch + 1) * kMaxBlocks * sizeof(double);
}

TableOf<kShort> shortened(const Table &t)
{
    TableOf<kShort> s = {};
    s.n = t.n;
    std::copy_n(t.g, t.n, s.g);
    std::copy_n(t.out, t.n, s.out);
    std::copy_n(t.first, t.n + 1, s.first);
    std::copy_n(t.last_n, t.n, s.last_n);
    return s;
}

struct Range {
    uintptr_t at;
    size_t n;
};

}  // namespace
}  // namespace pmha

using namespace pmha;

extern "C" {

size_t pmha_clip_grad_norm_workspace_size(int64_t n_tensors)
{
    if (n_tensors < 0 || n_tensors > (int64_t)1 << 24) return 0;
    return part_bytes(n_tensors);
}

pmha_status pmha_clip_grad_norm(int64_t n_tensors, const void *const *grads, void *const *out, const int64_t *numel,
                                const pmha_dtype *dtype, float max_norm, float *norm, void *workspace,
                                size_t workspace_bytes, pmha_stream stream)
{
    if (n_tensors < 0 || n_tensors > (int64_t)1 << 24 || (n_tensors && (!grads || !numel || !dtype))) {
        set_error("pmha_clip_grad_norm: %lld tensors, or a NULL table", (long long)n_tensors);
        return PMHA_ERR_INVALID_ARG;
    }
    if (!isfinite(max_norm) || max_norm < 0.f) {
        set_error("pmha_clip_grad_norm: max_norm %g must be finite and at least 0", (double)max_norm);
        return PMHA_ERR_INVALID_ARG;
    }
    if (!norm || ((uintptr_t)norm & 3u)) {
        set_error("pmha_clip_grad_norm: norm is NULL or not aligned");
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t need = part_bytes(n_tensors);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)) {
        set_error("pmha_clip_grad_norm: workspace needs %zu bytes, 256-byte aligned (got %zu at %p)", need,
                  workspace_bytes, workspace);
        return PMHA_ERR_WORKSPACE;
    }
    cudaStream_t cs = (cudaStream_t)stream;
    try {
        std::vector<Range> ranges;
        std::vector<Range> outs;
        ranges.reserve((size_t)n_tensors * 2 + 1);
        if (out) outs.reserve((size_t)n_tensors + 1);
        outs.push_back({(uintptr_t)norm, 4});
        int64_t total = 0;
        for (int64_t i = 0; i < n_tensors; ++i) {
            if (dtype[i] != PMHA_F32 && dtype[i] != PMHA_BF16) {
                set_error("pmha_clip_grad_norm: tensor %lld: dtype %d is neither PMHA_F32 nor PMHA_BF16",
                          (long long)i, (int)dtype[i]);
                return PMHA_ERR_INVALID_ARG;
            }
            if (numel[i] < 0 || numel[i] > (int64_t)1 << 40 || (total += numel[i]) > (int64_t)1 << 44) {
                set_error("pmha_clip_grad_norm: tensor %lld: %lld values", (long long)i, (long long)numel[i]);
                return PMHA_ERR_INVALID_ARG;
            }
            if (numel[i] == 0) continue;
            const size_t es = dtype[i] == PMHA_BF16 ? 2 : 4;
            const void *o = out ? out[i] : grads[i];
            if (!grads[i] || !o || ((uintptr_t)grads[i] % es) || ((uintptr_t)o % es)) {
                set_error("pmha_clip_grad_norm: tensor %lld is NULL or not aligned to its values", (long long)i);
                return PMHA_ERR_INVALID_ARG;
            }
            ranges.push_back({(uintptr_t)grads[i], (size_t)numel[i] * es});
            if (o != grads[i]) outs.push_back({(uintptr_t)o, (size_t)numel[i] * es});
        }
        // gradients counted twice are refused like outputs that touch anything
        const auto before = [](const Range &a, const Range &b) { return a.at < b.at; };
        for (std::vector<Range> *v : {&ranges, &outs})  // usually in order already: each laid out in one buffer
            if (!std::is_sorted(v->begin(), v->end(), before)) std::sort(v->begin(), v->end(), before);
        const auto middle = ranges.insert(ranges.end(), outs.begin(), outs.end());
        std::inplace_merge(ranges.begin(), middle, ranges.end(), before);
        uintptr_t end = 0;
        for (const Range &r : ranges) {
            if (r.at < end) {
                set_error("pmha_clip_grad_norm: two of the tensors, outputs and norm overlap, or one is given twice");
                return PMHA_ERR_INVALID_ARG;
            }
            end = r.at + r.n;
        }
        // launches of up to kBatch tensors and 2^31 chunks each
        const int max_grid = std::min(num_sms() * kBlocksPerSm, kMaxBlocks);
        auto fill = [&](Table &t, int64_t first) {
            int64_t chunks = 0, i = first;
            t.n = 0;
            for (; i < n_tensors && t.n < kBatch; ++i) {
                if (numel[i] == 0) continue;
                const int64_t per = kChunkBytes / (dtype[i] == PMHA_BF16 ? 2 : 4), c = (numel[i] + per - 1) / per;
                if (chunks + c > (int64_t)0x7fffffff) break;
                t.g[t.n] = grads[i];
                t.out[t.n] = out ? out[i] : const_cast<void *>(grads[i]);
                t.first[t.n] = (uint32_t)chunks;
                t.last_n[t.n] = (uint32_t)(numel[i] - (c - 1) * per) | (dtype[i] == PMHA_BF16 ? 1u << 31 : 0u);
                chunks += c;
                ++t.n;
            }
            t.first[t.n] = (uint32_t)chunks;
            return i;
        };
        Table t;
        int n_part = 0, launches = 0;
        double *part = (double *)workspace;
        int64_t i = 0;
        do {  // at least once: the norm of nothing is 0
            i = fill(t, i);
            const int grid = std::max(1, std::min<int>((int)t.first[t.n], max_grid));
            if ((size_t)(n_part + grid) * sizeof(double) > need) {
                set_error("pmha_clip_grad_norm: too many values for one call");
                return PMHA_ERR_INVALID_ARG;
            }
            StageTimer timer("grad_squares", cs);
            if (t.n <= kShort) k_grad_squares<<<grid, kThreads, 0, cs>>>(shortened(t), part + n_part);
            else k_grad_squares<<<grid, kThreads, 0, cs>>>(t, part + n_part);
            count_launch();
            PMHA_CUDA_TRY(cudaGetLastError());
            n_part += grid;
            ++launches;
        } while (i < n_tensors);
        i = 0;
        bool first = true;
        do {
            if (launches > 1) i = fill(t, i);
            else i = n_tensors;  // the only table is still here
            const int grid = std::max(1, std::min<int>((int)t.first[t.n], max_grid));
            StageTimer timer("grad_scale", cs);
            float *const norm_out = first ? norm : nullptr;
            if (t.n <= kShort) k_grad_scale<<<grid, kThreads, 0, cs>>>(shortened(t), part, n_part, max_norm, norm_out);
            else k_grad_scale<<<grid, kThreads, 0, cs>>>(t, part, n_part, max_norm, norm_out);
            count_launch();
            PMHA_CUDA_TRY(cudaGetLastError());
            first = false;
        } while (i < n_tensors);
    } catch (const std::bad_alloc &) {
        set_error("pmha_clip_grad_norm: out of host memory");
        return PMHA_ERR_INVALID_ARG;
    }
    return PMHA_OK;
}

}  // extern "C"
