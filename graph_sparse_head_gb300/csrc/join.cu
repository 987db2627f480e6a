// The join of a block's output with the residual stream, norms on both sides:
//
//   z = branch (mean(branch^2) + eps)^(-1/2) post       (without post: z = branch)
//   s = round(alpha residual + gate z)                  (kept in the layer type; the norm below is of the kept sum)
//   n = s (mean(s^2) + eps)^(-1/2) pre
//
// with gate one row for all rows, or one for each run of rows (the tokens of a sample); and its backward pass, with
// D = dsum + (gradient of the norm of s for dn pre):
//
//   dresidual = alpha D,  dbranch = gradient of the norm of branch for gate D post
//   dpre = sum dn s r,    dgate_g = post P_g,  dpost = sum_g gate_g P_g,  P_g = sum over the rows of g of D branch r_b
//
// and the tensors kept in 8 bits between the two (kept.cuh): the forward pass
// stores its inputs in 8 bits while it holds them, the backward pass (and a
// forward pass that forms s and n again) reads them from there. All of it is bound by
// memory; rows lie in registers as in norm.cu.
#include "join.cuh"

namespace pmha {
namespace {

struct JoinArgs {
    Source branch, res;
    const void *post, *gate, *pre;
    void *sum, *out;
    KeptOut keep_branch, keep_res;
    long long rows, per_gate;  // rows that share a gate
    int width;
    float alpha, eps;
};

// LPR threads share a row; thread l of them holds pieces l, l + LPR, ... of VEC values, NV of them.
template <typename T, int VEC, int NV, int LPR, bool KEPT>
__global__ void __launch_bounds__(kThreads) k_join(JoinArgs a)
{
    __shared__ TeamSums sh;
    int turn = 0;
    const int l = threadIdx.x % LPR;
    const long long row = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const bool live = row < a.rows;
    const long long base = row * a.width;
    float b[NV * VEC], x[NV * VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + l) * VEC;
        float (&bj)[VEC] = *reinterpret_cast<float (*)[VEC]>(b + j * VEC);
        float (&xj)[VEC] = *reinterpret_cast<float (*)[VEC]>(x + j * VEC);
#pragma unroll
        for (int i = 0; i < VEC; ++i) bj[i] = xj[i] = 0.f;
        if (live && c < a.width) {
            if constexpr (KEPT) {
                if (a.branch.any()) load_source<T, VEC>(a.branch, row, c, a.width, bj);
                load_source<T, VEC>(a.res, row, c, a.width, xj);
            } else {
                if (a.branch.p) load_row<T, VEC>(a.branch.p, base + c, bj);
                load_row<T, VEC>(a.res.p, base + c, xj);
            }
        }
    }
    if constexpr (KEPT) {
        auto keep_row = [&](const KeptOut &k, float *f) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * LPR + l) * VEC;
                T v[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = from_f<T>(f[j * VEC + i]);  // exact: values of the type
                keep<T, VEC>(k, row, c, a.width, live && c < a.width, v);
            }
        };
        if (a.keep_branch.codes) keep_row(a.keep_branch, b);
        if (a.keep_res.codes) keep_row(a.keep_res, x);
    }
    float rb = 1.f;
    if (a.post) {
        float sc;
        rb = row_root<NV * VEC, LPR>(b, a.width, a.eps, &sc, sh, turn);  // of b sc, which is what b holds now
    }
    const long long gate_at = a.gate && live ? row / a.per_gate * a.width : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + l) * VEC;
        const bool in = live && c < a.width;
        Vals<T, VEC> s;
        if (a.post && in) {
            float w[VEC];
            load_row<T, VEC>(a.post, c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) b[j * VEC + i] *= rb * w[i];
        }
        if (a.gate && in) {
            float w[VEC];
            load_row<T, VEC>(a.gate, gate_at + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) b[j * VEC + i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            s.v[i] = from_f<T>(fmaf(a.alpha, x[j * VEC + i], b[j * VEC + i]));
            x[j * VEC + i] = to_f<T>(s.v[i]);
        }
        if (in) store<T, VEC>((T *)a.sum + base + c, s.v);
    }
    if (!a.out) return;
    float sc;
    const float r = row_root<NV * VEC, LPR>(x, a.width, a.eps, &sc, sh, turn);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR + l) * VEC;
        if (!(live && c < a.width)) continue;
        float w[VEC];
        load_row<T, VEC>(a.pre, c, w);
        Vals<T, VEC> y;
#pragma unroll
        for (int i = 0; i < VEC; ++i) y.v[i] = from_f<T>(x[j * VEC + i] * r * w[i]);
        store<T, VEC>((T *)a.out + base + c, y.v);
    }
}

// Rows of more than 2048 values: one block a row, which reads its inputs again from L1 / L2 for each step.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_join_wide(JoinArgs a)
{
    __shared__ float sh[kThreads / 32];
    const long long row = blockIdx.x, base = row * a.width;
    const int lane = threadIdx.x & 31;
    const int first = (int)threadIdx.x * VEC, stride = kThreads * VEC;
    // whole warps walk here: a group's values lie in neighbouring lanes
    auto keep_row = [&](const KeptOut &k, const void *p) {
        for (int c0 = first - lane * VEC; c0 < a.width; c0 += stride) {
            const int c = c0 + lane * VEC;
            Vals<T, VEC> v;
#pragma unroll
            for (int i = 0; i < VEC; ++i) v.v[i] = from_f<T>(0.f);
            if (c < a.width) load<T, VEC>((const T *)p + base + c, v.v);
            keep<T, VEC>(k, row, c, a.width, c < a.width, v.v);
        }
    };
    if (a.keep_branch.codes) keep_row(a.keep_branch, a.branch.p);
    if (a.keep_res.codes) keep_row(a.keep_res, a.res.p);
    float rb = 1.f, scb = 1.f;
    if (a.post)
        rb = block_root(sh, a.width, a.eps, &scb,
                        [&](float sc) {
                            float ss = 0.f;
                            for (int c = first; c < a.width; c += stride) {
                                float v[VEC];
                                load_source<T, VEC>(a.branch, row, c, a.width, v);
#pragma unroll
                                for (int i = 0; i < VEC; ++i) ss = fmaf(v[i] * sc, v[i] * sc, ss);
                            }
                            return ss;
                        },
                        [&]() {
                            float m = 0.f;
                            for (int c = first; c < a.width; c += stride) {
                                float v[VEC];
                                load_source<T, VEC>(a.branch, row, c, a.width, v);
#pragma unroll
                                for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(v[i]));
                            }
                            return m;
                        });
    const long long gate_at = a.gate ? row / a.per_gate * a.width : 0;
    float ss = 0.f, most = 0.f;
    for (int c = first; c < a.width; c += stride) {
        float b[VEC], x[VEC], w[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[i] = 0.f;
        if (a.branch.any()) load_source<T, VEC>(a.branch, row, c, a.width, b);
        load_source<T, VEC>(a.res, row, c, a.width, x);
        if (a.post) {
            load_row<T, VEC>(a.post, c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) b[i] = b[i] * scb * (rb * w[i]);
        }
        if (a.gate) {
            load_row<T, VEC>(a.gate, gate_at + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) b[i] *= w[i];
        }
        Vals<T, VEC> s;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            s.v[i] = from_f<T>(fmaf(a.alpha, x[i], b[i]));
            const float f = to_f<T>(s.v[i]);
            ss = fmaf(f, f, ss);
            most = fmaxf(most, fabsf(f));
        }
        store<T, VEC>((T *)a.sum + base + c, s.v);
    }
    if (!a.out) return;
    float sc;
    const float r = block_root(sh, a.width, a.eps, &sc,
                               [&](float k) {
                                   if (k == 1.f) return ss;
                                   float t = 0.f;
                                   for (int c = first; c < a.width; c += stride) {
                                       float v[VEC];
                                       load_row<T, VEC>(a.sum, base + c, v);  // this thread's own values
#pragma unroll
                                       for (int i = 0; i < VEC; ++i) t = fmaf(v[i] * k, v[i] * k, t);
                                   }
                                   return t;
                               },
                               [&]() { return most; });
    for (int c = first; c < a.width; c += stride) {
        float v[VEC], w[VEC];
        load_row<T, VEC>(a.sum, base + c, v);
        load_row<T, VEC>(a.pre, c, w);
        Vals<T, VEC> y;
#pragma unroll
        for (int i = 0; i < VEC; ++i) y.v[i] = from_f<T>(v[i] * sc * r * w[i]);
        store<T, VEC>((T *)a.out + base + c, y.v);
    }
}

// ---------------------------------------------------------------- 8-bit tensors on their own
// A lane takes VEC values of a group; a warp 32 / (32 / VEC) groups at a time.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_keep(const T *x, long long rows, int width, KeptOut k)
{
    constexpr int kLanes = kGroup / VEC;
    const int groups = (width + kGroup - 1) / kGroup;
    const long long n = rows * groups, step = (long long)gridDim.x * kThreads / kLanes;
    const int l = threadIdx.x % kLanes;
    // whole warps walk: a warp's groups are consecutive
    const long long lead = ((long long)blockIdx.x * kThreads + threadIdx.x / 32 * 32) / kLanes;
    for (long long g0 = lead; g0 < n; g0 += step) {
        const long long g = g0 + (threadIdx.x % 32) / kLanes;
        const long long row = g / groups;
        const int c = (int)(g - row * groups) * kGroup + l * VEC;
        const bool in = g < n && c < width;
        Vals<T, VEC> v;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.v[i] = from_f<T>(0.f);
        if (in) load<T, VEC>(x + row * width + c, v.v);
        keep<T, VEC>(k, row, c, width, in, v.v);
    }
}
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_unkeep(Kept k, long long rows, int width, T *out)
{
    constexpr int kLanes = kGroup / VEC;
    const int groups = (width + kGroup - 1) / kGroup;
    const long long n = rows * groups, step = (long long)gridDim.x * kThreads / kLanes;
    for (long long g = ((long long)blockIdx.x * kThreads + threadIdx.x) / kLanes; g < n; g += step) {
        const long long row = g / groups;
        const int c = (int)(g - row * groups) * kGroup + (int)(threadIdx.x % kLanes) * VEC;
        if (c >= width) continue;
        float f[VEC];
        load_kept<VEC>(k, row, c, width, f);
        Vals<T, VEC> v;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.v[i] = from_f<T>(f[i]);
        store<T, VEC>(out + row * width + c, v.v);
    }
}

}  // namespace
}  // namespace pmha

using namespace pmha;

extern "C" {

pmha_status pmha_join(const pmha_join_params *params, int64_t rows, const void *branch, const pmha_kept *branch_kept,
                      const void *residual, const pmha_kept *residual_kept, void *sum, void *out,
                      const pmha_kept *keep_branch, const pmha_kept *keep_residual, pmha_stream stream)
{
    pmha_status st = check_join("pmha_join", params, rows);
    if (st != PMHA_OK || rows == 0) return st;
    const pmha_join_params &p = *params;
    const bool has_branch = branch || branch_kept;
    if ((branch && branch_kept) || !(residual || residual_kept) || (residual && residual_kept) ||
        (!has_branch && (p.post || p.gate)) || !sum || (out != nullptr) != (p.pre != nullptr) ||
        (keep_branch && !branch) || (keep_residual && !residual)) {
        set_error("pmha_join: needs sum, one form of the residual and at most one of the branch (none only without post and "
                  "gate), out just if pre is set, and keeps a branch or residual only of those given in dtype");
        return PMHA_ERR_INVALID_ARG;
    }
    if (!aligned(branch, 16) || !aligned(residual, 16) || !aligned(sum, 16) || !aligned(out, 16) || !whole(branch_kept) ||
        !whole(residual_kept) || !whole(keep_branch) || !whole(keep_residual)) {
        set_error("pmha_join: a pointer is not 16-byte aligned, or a kept tensor lacks its codes or scales");
        return PMHA_ERR_INVALID_ARG;
    }
    const int64_t w = p.width;
    const size_t nb = (size_t)(rows * w) * bytes_of(p.dtype), wb = (size_t)w * bytes_of(p.dtype);
    const Span ins[] = {{branch, nb}, {residual, nb}, codes_of(branch_kept, rows, w), scales_of(branch_kept, rows, w),
                        codes_of(residual_kept, rows, w), scales_of(residual_kept, rows, w), {p.post, wb}, {p.pre, wb},
                        {p.gate, wb * (size_t)p.gates}};
    const Span outs[] = {{sum, nb}, {out, nb}, codes_of(keep_branch, rows, w), scales_of(keep_branch, rows, w),
                         codes_of(keep_residual, rows, w), scales_of(keep_residual, rows, w)};
    if (any_overlap(ins, outs)) {
        set_error("pmha_join: an output overlaps an input or another output");
        return PMHA_ERR_INVALID_ARG;
    }
    JoinArgs a{source(branch, branch_kept), source(residual, residual_kept), p.post, p.gate, p.pre, sum, out,
               kept_out(keep_branch), kept_out(keep_residual), rows, p.gate ? rows / p.gates : rows, (int)w,
               p.residual_scale, p.eps};
    const bool kept = branch_kept || residual_kept || keep_branch || keep_residual;
    const Shape s = join_shape(p.dtype, w);
    cudaStream_t cs = (cudaStream_t)stream;
    {
        StageTimer timer(kept ? "join_kept" : "join", cs);
        if (s.lpr) {
            const int64_t per = kThreads / s.lpr;
            const unsigned grid = (unsigned)((rows + per - 1) / per);
            join_dispatch(p.dtype, s, [&](auto t) {
                using G = decltype(t);
                if (kept) k_join<typename G::type, G::vec, G::nv, G::lpr, true><<<grid, kThreads, 0, cs>>>(a);
                else k_join<typename G::type, G::vec, G::nv, G::lpr, false><<<grid, kThreads, 0, cs>>>(a);
            });
        } else {
            dispatch_wide(p.dtype, s.vec, [&](auto t) {
                using G = decltype(t);
                k_join_wide<typename G::type, G::vec><<<(unsigned)rows, kThreads, 0, cs>>>(a);
            });
        }
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

static pmha_status check_kept(const char *who, pmha_dtype dtype, int64_t rows, int64_t width, const void *x,
                              const pmha_kept *kept)
{
    pmha_status st = check_rows(who, dtype, rows, width);
    if (st != PMHA_OK || rows == 0) return st;
    if (!x || !aligned(x, 16) || !kept || !whole(kept)) {
        set_error("%s: a pointer is NULL or not 16-byte aligned", who);
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t nb = (size_t)(rows * width) * bytes_of(dtype);
    const Span none[] = {{nullptr, 0}}, all[] = {{x, nb}, codes_of(kept, rows, width), scales_of(kept, rows, width)};
    if (any_overlap(none, all)) {
        set_error("%s: an output overlaps an input or another output", who);
        return PMHA_ERR_INVALID_ARG;
    }
    return PMHA_OK;
}

pmha_status pmha_checkpoint(pmha_dtype dtype, int64_t rows, int64_t width, const void *x, const pmha_kept *kept,
                            pmha_stream stream)
{
    pmha_status st = check_kept("pmha_checkpoint", dtype, rows, width, x, kept);
    if (st != PMHA_OK || rows == 0) return st;
    cudaStream_t cs = (cudaStream_t)stream;
    {
        StageTimer timer("checkpoint", cs);
        dispatch_wide(dtype, shape_of(dtype, width).vec, [&](auto t) {
            using G = decltype(t);
            const int64_t lanes = rows * groups_of(width) * (kGroup / G::vec);
            const unsigned grid = (unsigned)std::min<int64_t>((lanes + kThreads - 1) / kThreads, (int64_t)num_sms() * 8);
            k_keep<typename G::type, G::vec>
                <<<grid, kThreads, 0, cs>>>((const typename G::type *)x, rows, (int)width, kept_out(kept));
        });
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

pmha_status pmha_checkpoint_restore(pmha_dtype dtype, int64_t rows, int64_t width, const pmha_kept *kept, void *out,
                                    pmha_stream stream)
{
    pmha_status st = check_kept("pmha_checkpoint_restore", dtype, rows, width, out, kept);
    if (st != PMHA_OK || rows == 0) return st;
    cudaStream_t cs = (cudaStream_t)stream;
    {
        StageTimer timer("checkpoint_restore", cs);
        dispatch_wide(dtype, shape_of(dtype, width).vec, [&](auto t) {
            using G = decltype(t);
            const int64_t lanes = rows * groups_of(width) * (kGroup / G::vec);
            const unsigned grid = (unsigned)std::min<int64_t>((lanes + kThreads - 1) / kThreads, (int64_t)num_sms() * 8);
            k_unkeep<typename G::type, G::vec><<<grid, kThreads, 0, cs>>>(source(nullptr, kept).k, rows, (int)width,
                                                                          (typename G::type *)out);
        });
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

}  // extern "C"
