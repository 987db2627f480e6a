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
    KeptOut keep_branch, keep_res;  // at widths of whole 16-byte pieces only
    long long rows, per_gate;  // rows that share a gate
    int width;
    float alpha, eps;
};

// A block takes a few steps of rows, so that blocks are dealt out as others leave, where memory bounds the call: 320,000 x
// 128 took 50 us with 4 steps, 51 with 16, and 57 with all rows dealt to resident blocks beforehand (SMs do not get at
// memory alike). One step where there are fewer blocks otherwise than are resident. Calls with kept tensors are bound by
// instructions, and a block's start costs some: 62 us with rows dealt out beforehand, 74 with 8 steps.
constexpr int kFewSteps = 4;
constexpr int kResident = 3;  // blocks of an SM
// Rows of 16-byte pieces come through a ring of kRing steps, each thread copying and reading its own pieces (no
// barrier): what is in flight does not take registers. Others are loaded a step ahead.
template <typename T, int VEC, int NV>
constexpr int kRingOf = VEC * sizeof(T) == 16 ? 4 / NV : 0;
constexpr int kSlotBytes = 2 * 16 * kThreads;  // branch and residual of one piece
template <typename T, int VEC, int NV>
constexpr size_t kRingBytes = (size_t)kRingOf<T, VEC, NV> * NV * kSlotBytes;

// Teams of LPR threads (join.cuh) walk rows; thread l of a team holds pieces l, l + LPR, ... of VEC values, NV of them,
// of a row, and of the weights. Instructions count here: with 275 of them for 8 values a lane the 20,000-node graph took
// 57 us and the warps were issuing in three cycles of four, so addresses are one running offset, and copies are skipped
// rather than zero-filled: lanes past the width find zeros in their places, which nothing overwrites, and teams past the
// last row find what was there before, and store nothing.
template <typename T, int VEC, int NV, int LPR, bool KEPT, int kSteps>
__global__ void __launch_bounds__(kThreads, kResident) k_join(JoinArgs a)
{
    extern __shared__ __align__(16) uint8_t ring_s[];
    __shared__ TeamSums sh;
    using Codes = typename Bytes<VEC>::type;
    using V = Vals<T, VEC>;
    constexpr int kRows = kThreads / LPR, N = NV * VEC;  // rows of a block's step, values of a thread
    constexpr int kRing = kRingOf<T, VEC, NV>;
    constexpr int kPiece = LPR * VEC;                    // from one piece of a thread to the next
    int turn = 0;
    const int l = threadIdx.x % LPR;
    // a few steps of consecutive rows, or rows from all over
    const unsigned step = KEPT ? gridDim.x * kRows : kRows;
    const unsigned begin = blockIdx.x * (KEPT ? kRows : kRows * kSteps);
    const unsigned rows = KEPT ? (unsigned)a.rows : min((unsigned)a.rows, begin + kRows * kSteps);
    const long long stride = (long long)step * a.width;
    const float inv_width = 1.f / (float)a.width;
    // a warp's threads walk together: row0 is the first of its rows
    constexpr int kPerWarp = LPR < 32 ? 32 / LPR : 1;
    const unsigned sub = LPR < 32 ? (threadIdx.x & 31) / LPR : 0;
    const unsigned row_first = begin + threadIdx.x / (LPR < 32 ? 32 : LPR) * kPerWarp;
    bool col[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) col[j] = l * VEC + j * kPiece < a.width;
    V wpost[NV], wpre[NV], wgate[NV];  // the gate of the next row, if rows have different ones
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = l * VEC + j * kPiece;
#pragma unroll
        for (int i = 0; i < VEC; ++i) wpost[j].v[i] = wpre[j].v[i] = wgate[j].v[i] = from_f<T>(1.f);
        if (col[j]) {
            if (a.post) load<T, VEC>((const T *)a.post + c, wpost[j].v);
            if (a.out) load<T, VEC>((const T *)a.pre + c, wpre[j].v);
        }
    }
    const bool own_gate = a.gate && a.per_gate < a.rows;
    auto fetch_gate = [&](unsigned row) {
        if (row >= rows) return;
        const long long at = own_gate ? (long long)(row / (unsigned)a.per_gate) * a.width : 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (col[j]) load<T, VEC>((const T *)a.gate + at + l * VEC + j * kPiece, wgate[j].v);
    };
    float wz[N];  // post times gate of the row at hand: exact in bf16
    auto times_gate = [&]() {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float g[VEC];
            widen<T, VEC>(wpost[j], wz + j * VEC);
            widen<T, VEC>(wgate[j], g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) wz[j * VEC + i] *= g[i];
        }
    };
    // kept values' scales, of the next row, as they were loaded: widened there they would be waited for there
    const int groups = (a.width + kGroup - 1) / kGroup;
    __nv_bfloat16 sb[NV] = {}, sx[NV] = {};
    auto fetch_scales = [&](unsigned row, long long at) {
        if constexpr (KEPT) {
            if (row >= rows) return;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!col[j]) continue;
                const long long s = at + j * (kPiece / kGroup);
                if (a.branch.k.codes) sb[j] = a.branch.k.scale[s];
                if (a.res.k.codes) sx[j] = a.res.k.scale[s];
            }
        }
    };
    // the row's offset, and its scales'; those of the row to fetch lie ahead by a fixed distance
    long long at = (long long)(row_first + sub) * a.width + l * VEC;
    long long sat = (long long)(row_first + sub) * groups + l * VEC / kGroup;
    V nb[kRing ? 1 : NV] = {}, nx[kRing ? 1 : NV] = {};  // the next row's, without a ring
    Codes cb[kRing ? 1 : NV] = {}, cx[kRing ? 1 : NV] = {};
    uint8_t *ring = ring_s + threadIdx.x * 16;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    auto fetch = [&](unsigned row, long long from, int slot) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (row >= rows || !col[j]) continue;
            const long long e = from + j * kPiece;
            if constexpr (kRing > 0) {
                const uint32_t dst = ring_at + (slot * NV + j) * kSlotBytes;
                if (a.branch.p) ring_copy(dst, (const T *)a.branch.p + e);
                else if (KEPT && a.branch.k.codes) ring_codes<VEC>(dst, a.branch.k.codes + e);
                if (!KEPT || a.res.p) ring_copy(dst + 16 * kThreads, (const T *)a.res.p + e);
                else ring_codes<VEC>(dst + 16 * kThreads, a.res.k.codes + e);
            } else {
                if (a.branch.p) load<T, VEC>((const T *)a.branch.p + e, nb[j].v);
                else if (KEPT && a.branch.k.codes) cb[j] = *reinterpret_cast<const Codes *>(a.branch.k.codes + e);
                if (!KEPT || a.res.p) load<T, VEC>((const T *)a.res.p + e, nx[j].v);
                else cx[j] = *reinterpret_cast<const Codes *>(a.res.k.codes + e);
            }
        }
        if constexpr (kRing > 0) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (kRing > 0) {
#pragma unroll
        for (int i = 0; i < kRing * NV; ++i)
            if (!col[i % NV] || row_first + sub >= rows)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *reinterpret_cast<uint4 *>(ring + i * kSlotBytes + k * 16 * kThreads) = make_uint4(0, 0, 0, 0);
        for (int i = 0; i < kRing - 1; ++i) fetch(row_first + sub + i * step, at + i * stride, i);
    } else {
        fetch(row_first + sub, at, 0);
    }
    if (a.gate) fetch_gate(row_first + sub);
    times_gate();
    if (own_gate) fetch_gate(row_first + sub + step);
    fetch_scales(row_first + sub, sat);
    int slot = 0;
    for (unsigned row0 = row_first; row0 < rows; row0 += step, at += stride, sat += (long long)step * groups) {
        const unsigned row = row0 + sub;
        const bool live = row < rows;
        if constexpr (kRing > 0) {
            fetch(row + (kRing - 1) * step, at + (kRing - 1) * stride, slot ? slot - 1 : kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        }
        float b[N], x[N];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint8_t *p = ring + (slot * NV + j) * kSlotBytes;
            auto piece = [&](const V *next, int k) {
                if constexpr (kRing > 0) return *reinterpret_cast<const V *>(p + k * 16 * kThreads);
                else return next[j];
            };
            auto codes = [&](const Codes *next, int k) {
                if constexpr (kRing > 0) return *reinterpret_cast<const Codes *>(p + k * 16 * kThreads);
                else return next[j];
            };
            float (&bj)[VEC] = *reinterpret_cast<float (*)[VEC]>(b + j * VEC);
            float (&xj)[VEC] = *reinterpret_cast<float (*)[VEC]>(x + j * VEC);
            if (a.branch.p) {
                const V v = piece(nb, 0);
                widen<T, VEC>(v, bj);
                if constexpr (KEPT && VEC >= 4)
                    if (a.keep_branch.codes) {
                        const long long e = at + j * kPiece;
                        keep<T, VEC>(KeptOut{a.keep_branch.codes + e, a.keep_branch.scale + sat + j * (kPiece / kGroup)},
                                     l * VEC % kGroup == 0, live && col[j], v);
                    }
            } else if (KEPT && a.branch.k.codes) {
                unkeep<VEC>(codes(cb, 0), __bfloat162float(sb[j]), bj);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) bj[i] = 0.f;
            }
            if (!KEPT || a.res.p) {
                const V v = piece(nx, 1);
                widen<T, VEC>(v, xj);
                if constexpr (KEPT && VEC >= 4)
                    if (a.keep_res.codes) {
                        const long long e = at + j * kPiece;
                        keep<T, VEC>(KeptOut{a.keep_res.codes + e, a.keep_res.scale + sat + j * (kPiece / kGroup)},
                                     l * VEC % kGroup == 0, live && col[j], v);
                    }
            } else {
                unkeep<VEC>(codes(cx, 1), __bfloat162float(sx[j]), xj);
            }
        }
        if constexpr (kRing > 0) slot = slot + 1 == kRing ? 0 : slot + 1;
        else fetch(row + step, at + stride, 0);
        fetch_scales(row + step, sat + (long long)step * groups);
        // sum: of the weights' product first, so that branch, weights and root meet in one more product and the addition:
        // sums rounded to bf16 seldom fall to the other side of what exact arithmetic gives
        float rb = 1.f;
        if (a.post) {
            float sc;
            rb = row_root<N, LPR>(b, inv_width, a.eps, &sc, sh, turn);  // of b sc, which is what b holds now
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float (&xj)[VEC] = *reinterpret_cast<float (*)[VEC]>(x + j * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i) xj[i] = fmaf(b[j * VEC + i] * wz[j * VEC + i], rb, a.alpha * xj[i]);
            const V s = rounded<T, VEC>(xj);
            if (live && col[j]) store<T, VEC>((T *)a.sum + at + j * kPiece, s.v);
        }
        if (own_gate) {
            times_gate();
            fetch_gate(row + 2 * step);
        }
        if (!a.out) continue;
        float sc;
        const float r = row_root<N, LPR>(x, inv_width, a.eps, &sc, sh, turn);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float (&xj)[VEC] = *reinterpret_cast<float (*)[VEC]>(x + j * VEC);
            float w[VEC];
            widen<T, VEC>(wpre[j], w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) xj[i] *= r * w[i];
            const V y = rounded<T, VEC>(xj);
            if (live && col[j]) store<T, VEC>((T *)a.out + at + j * kPiece, y.v);
        }
    }
    // the last copies land before the block's shared memory can go to another
    if constexpr (kRing > 0) asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows of more than 2048 values: one block a row, which reads its inputs again from L1 / L2 for each step.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_join_wide(JoinArgs a)
{
    __shared__ float sh[kThreads / 32];
    const long long row = blockIdx.x, base = row * a.width;
    const int first = (int)threadIdx.x * VEC, stride = kThreads * VEC;
    if constexpr (VEC >= 4) {
        // whole warps walk here: a group's values lie in neighbouring lanes
        auto keep_row = [&](const KeptOut &k, const void *p) {
            const int lane = threadIdx.x & 31;
            for (int c0 = first - lane * VEC; c0 < a.width; c0 += stride) {
                const int c = c0 + lane * VEC;
                Vals<T, VEC> v;
#pragma unroll
                for (int i = 0; i < VEC; ++i) v.v[i] = from_f<T>(0.f);
                if (c < a.width) load<T, VEC>((const T *)p + base + c, v.v);
                keep<T, VEC>(KeptOut{k.codes + base + c, k.scale + row * groups_of(a.width) + c / kGroup}, c % kGroup == 0,
                             c < a.width, v);
            }
        };
        if (a.keep_branch.codes) keep_row(a.keep_branch, a.branch.p);
        if (a.keep_res.codes) keep_row(a.keep_res, a.res.p);
    }
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
        if (a.post) load_row<T, VEC>(a.post, c, w);
        else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = 1.f;
        }
        if (a.gate) {
            float g[VEC];
            load_row<T, VEC>(a.gate, gate_at + c, g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] *= g[i];
        }
        Vals<T, VEC> s;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            s.v[i] = from_f<T>(fmaf(b[i] * scb * w[i], rb, a.alpha * x[i]));
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
// A lane takes VEC values of a group, 32 / VEC lanes a group; each thread has kAhead groups' values loaded before it uses
// the first. Two 16-byte loads a lane where rows hold whole pairs of them: a group's scale, shuffles and addresses are then
// shared by twice the values (320,000 x 128 bf16 22 us, 83 % of the copy rate; one load a lane 29 and 103 instructions for
// eight values). A tensor whose rows are whole groups is one long row here (`groups` 0: no division by a row's groups). Where
// rows do not lie on 16-byte boundaries a lane's values are still next to one another, and go one by one: with one value a
// lane every lane does a whole group's sums, 100,000 x 171 took 52 us.
constexpr int kAhead = 4;
struct Place {
    long long at, group;  // of the values, of the scale
    int left;             // values from there to the end of the row, 0 past the last group
};
template <int VEC>
__device__ __forceinline__ Place place_of(long long g, long long n, unsigned groups, int width)
{
    const int l = (int)(threadIdx.x % (kGroup / VEC)) * VEC;
    if (!groups) return {g * kGroup + l, g, g < n ? VEC : 0};
    const long long row = n >> 32 ? g / groups : (long long)((unsigned)g / groups);
    const int c = (int)(g - row * groups) * kGroup + l;
    return {row * width + c, g, g < n ? max(width - c, 0) : 0};
}
template <typename T, int VEC, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_keep(const T *x, long long n, unsigned groups, int width, KeptOut k)
{
    constexpr int kPer = 32 / (kGroup / VEC);  // groups of a warp
    const long long step = (long long)gridDim.x * (kThreads / 32) * kPer;
    // whole warps walk: a warp's groups are consecutive
    for (long long g0 = ((long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kPer; g0 < n; g0 += kAhead * step) {
        Vals<T, VEC> v[kAhead];
        Place p[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            p[i] = place_of<VEC>(g0 + i * step + (threadIdx.x % 32) / (kGroup / VEC), n, groups, width);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i].v[e] = from_f<T>(0.f);
            if (p[i].left) load_some<T, VEC, ALIGNED>(x + p[i].at, p[i].left, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const bool first = threadIdx.x % (kGroup / VEC) == 0;
            if constexpr (ALIGNED) {
                keep<T, VEC>(KeptOut{k.codes + p[i].at, k.scale + p[i].group}, first, p[i].left > 0, v[i]);
            } else {
                uint32_t w[VEC];
                const float scale = kept_codes<T, VEC>(v[i], w);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (e < p[i].left) k.codes[p[i].at + e] = (int8_t)w[e];
                if (first && p[i].left) k.scale[p[i].group] = __float2bfloat16_rn(scale);
            }
        }
    }
}
// Back to values: 320,000 x 128 bf16 in 20 us, 94 % of the copy rate.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_unkeep(Kept k, long long n, unsigned groups, int width, T *out)
{
    const long long step = (long long)gridDim.x * kThreads / (kGroup / VEC);
    for (long long g0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / (kGroup / VEC); g0 < n; g0 += kAhead * step) {
        typename Bytes<VEC>::type c[kAhead];
        float scale[kAhead];
        Place p[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            p[i] = place_of<VEC>(g0 + i * step, n, groups, width);
            if (!p[i].left) continue;
            c[i] = *reinterpret_cast<const typename Bytes<VEC>::type *>(k.codes + p[i].at);
            scale[i] = __bfloat162float(k.scale[p[i].group]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (!p[i].left) continue;
            float f[VEC];
            unkeep<VEC>(c[i], scale[i], f);
            const Vals<T, VEC> v = rounded<T, VEC>(f);
            store<T, VEC>(out + p[i].at, v.v);
        }
    }
}

// The same where rows do not lie on 16-byte boundaries: codes and values have the same places in tensors that as a whole
// do, so a lane takes VEC neighbours of whatever rows, in whole accesses, and looks up the scale of each (100,000 x 171 bf16
// 19 us; a value a lane, its place found by a division, 33).
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_unkeep_flat(Kept k, long long n, unsigned groups, unsigned width, T *out)
{
    const long long step = (long long)gridDim.x * kThreads * VEC;
    for (long long at = ((long long)blockIdx.x * kThreads + threadIdx.x) * VEC; at < n; at += step) {
        const long long row = n >> 32 ? at / width : (long long)((unsigned)at / width);
        unsigned c = (unsigned)(at - row * width);
        const __nv_bfloat16 *scale = k.scale + row * groups;
        typename Bytes<VEC>::type codes = {};
        const bool whole = at + VEC <= n;
        if (whole) {
            codes = *reinterpret_cast<const typename Bytes<VEC>::type *>(k.codes + at);
        } else {
            for (int i = 0; i < (int)(n - at); ++i) reinterpret_cast<int8_t *>(&codes)[i] = k.codes[at + i];
        }
        __nv_bfloat16 sc[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if (i && c == width) c = 0, scale += groups;
            sc[i] = whole || at + i < n ? scale[c / kGroup] : __float2bfloat16_rn(0.f);
            ++c;
        }
        float f[VEC];
        unkeep<VEC>(codes, 1.f, f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] *= __bfloat162float(sc[i]);
        const Vals<T, VEC> v = rounded<T, VEC>(f);
        if (whole) {
            store<T, VEC>(out + at, v.v);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (at + i < n) out[at + i] = v.v[i];
        }
    }
}

// ---------------------------------------------------------------- host side
unsigned kept_groups(int64_t width) { return width % kGroup ? (unsigned)groups_of(width) : 0u; }
// Every thread its kAhead groups once, or as many blocks as are resident
unsigned kept_grid(int64_t n, int vec)
{
    const int64_t threads = (n * (kGroup / vec) + kAhead - 1) / kAhead;
    return (unsigned)std::min<int64_t>((threads + kThreads - 1) / kThreads, (int64_t)num_sms() * 8);
}
pmha_status launch_keep(pmha_dtype dtype, int64_t rows, int64_t width, const void *x, const KeptOut &k, cudaStream_t cs)
{
    StageTimer timer("checkpoint", cs);
    const int64_t n = rows * groups_of(width);
    auto launch = [&](auto kern, auto *p, int vec) {
        kern<<<kept_grid(n, vec), kThreads, 0, cs>>>(p, n, kept_groups(width), (int)width, k);
    };
    using B = __nv_bfloat16;
    if (dtype == PMHA_BF16) {
        if (width % 16 == 0) launch(k_keep<B, 16, true>, (const B *)x, 16);
        else launch(width % 8 == 0 ? k_keep<B, 8, true> : k_keep<B, 8, false>, (const B *)x, 8);
    } else {
        if (width % 8 == 0) launch(k_keep<float, 8, true>, (const float *)x, 8);
        else launch(width % 4 == 0 ? k_keep<float, 4, true> : k_keep<float, 4, false>, (const float *)x, 4);
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
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
    const Shape s = join_shape(p.dtype, w);
    cudaStream_t cs = (cudaStream_t)stream;
    if (s.vec < 4) {
        // With one or two values a lane the codes cost more on the way than a pass of their own: 100,000 x 171 150 us with
        // the branch's, without them 45 and 21 for the pass. The kernels have no such form.
        if (keep_branch && (st = launch_keep(p.dtype, rows, w, branch, a.keep_branch, cs)) != PMHA_OK) return st;
        if (keep_residual && (st = launch_keep(p.dtype, rows, w, residual, a.keep_res, cs)) != PMHA_OK) return st;
        a.keep_branch = a.keep_res = KeptOut{nullptr, nullptr};
    }
    const bool kept = branch_kept || residual_kept || a.keep_branch.codes || a.keep_res.codes;
    {
        StageTimer timer(kept ? "join_kept" : "join", cs);
        if (s.lpr) {
            const int64_t per = kThreads / s.lpr;
            const int64_t steps = (rows + per - 1) / per, all = (int64_t)num_sms() * kResident;
            const bool few = steps < all * kFewSteps;
            join_dispatch(p.dtype, s, [&](auto t) {
                using G = decltype(t);
                using T = typename G::type;
                constexpr size_t smem = kRingBytes<T, G::vec, G::nv>;
                static_assert(smem <= 48 * 1024, "what a launch may have without asking");
                if (kept) k_join<T, G::vec, G::nv, G::lpr, true, 1><<<(unsigned)std::min(steps, all), kThreads, smem, cs>>>(a);
                else if (few) k_join<T, G::vec, G::nv, G::lpr, false, 1><<<(unsigned)steps, kThreads, smem, cs>>>(a);
                else
                    k_join<T, G::vec, G::nv, G::lpr, false, kFewSteps>
                        <<<(unsigned)((steps + kFewSteps - 1) / kFewSteps), kThreads, smem, cs>>>(a);
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
    return launch_keep(dtype, rows, width, x, kept_out(kept), (cudaStream_t)stream);
}

pmha_status pmha_checkpoint_restore(pmha_dtype dtype, int64_t rows, int64_t width, const pmha_kept *kept, void *out,
                                    pmha_stream stream)
{
    pmha_status st = check_kept("pmha_checkpoint_restore", dtype, rows, width, out, kept);
    if (st != PMHA_OK || rows == 0) return st;
    cudaStream_t cs = (cudaStream_t)stream;
    {
        StageTimer timer("checkpoint_restore", cs);
        const int64_t n = rows * groups_of(width), values = rows * width;
        auto launch = [&](auto *p, auto lane) {
            using T = std::remove_reference_t<decltype(*p)>;
            constexpr int kVec = decltype(lane)::value;
            const Kept k = source(nullptr, kept).k;
            if (width % kVec == 0) {
                k_unkeep<T, kVec><<<kept_grid(n, kVec), kThreads, 0, cs>>>(k, n, kept_groups(width), (int)width, p);
            } else {
                const int64_t blocks = (values + kThreads * kVec - 1) / (kThreads * kVec);
                k_unkeep_flat<T, kVec><<<(unsigned)std::min<int64_t>(blocks, (int64_t)num_sms() * 8), kThreads, 0, cs>>>(
                    k, values, (unsigned)groups_of(width), (unsigned)width, p);
            }
        };
        if (dtype == PMHA_BF16) launch((__nv_bfloat16 *)out, std::integral_constant<int, 8>());
        else launch((float *)out, std::integral_constant<int, 4>());
    }
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    return PMHA_OK;
}

}  // extern "C"
