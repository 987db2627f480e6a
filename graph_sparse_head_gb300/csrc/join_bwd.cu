// Backward pass of the join (join.cu has the formulas).
#include "join.cuh"
#include "pair.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {

// ---------------------------------------------------------------- backward
struct JoinBwdArgs {
    Source branch;
    const void *sum, *dy, *ds;  // dy null: no norm after the join
    const void *post, *gate, *pre;
    void *dbranch, *dres;
    float *part_pre, *part_branch;  // (grid, width) partial sums of dn s r and of D branch r_b, or null
    long long per_gate;             // rows that share a gate (all, without one)
    int blocks_per_gate;            // blocks that share them
    int width;
    float alpha, eps;
};

// Steps of a block: so many rows at most does a team add in float32 one after the other. A block's teams (32 at most) follow in
// float32, by shuffles and then eight in order; blocks' partial rows are added as pairs of floats.
constexpr int kSteps = 128;

// Rows of 16-byte pieces come through a ring as in the forward pass; others are loaded when they are needed.
template <typename T, int VEC, int NV>
constexpr int kRingOf = VEC * sizeof(T) == 16 ? 4 / NV : 0;
constexpr int kSlotBytes = 4 * 16 * kThreads;  // dout, sum, dsum and branch of one piece
template <typename T, int VEC, int NV>
constexpr size_t kRingBytes = (size_t)kRingOf<T, VEC, NV> * NV * kSlotBytes;

// A team (join.cuh) walks rows of one gate and keeps its columns' two sums over rows in
// registers; a block adds its teams' through shared memory and writes one partial row of each. As in the forward pass,
// addresses are one running offset and copies are skipped where there is nothing to copy. Bound by memory where rows are many:
// 1,280,000 x 256 bf16 601 us, 96 % of the copy rate; 320,000 x 128 88 us, 83 of them without the sums over rows; from 8
// bits 80. 114 registers, two blocks an SM: the sums' and the weights' columns stay in them (three blocks an SM with the
// weights in shared memory spilled, 95 us).
template <typename T, int VEC, int NV, int LPR, bool KEPT>
__global__ void __launch_bounds__(kThreads, 2) k_join_bwd(JoinBwdArgs a)
{
    extern __shared__ __align__(16) float shw[];  // the ring, then width values
    __shared__ TeamSums sh;
    using Codes = typename Bytes<VEC>::type;
    using V = Vals<T, VEC>;
    constexpr int kRows = kThreads / LPR, N = NV * VEC;  // rows of a block's step, values of a thread
    constexpr int kPerWarp = LPR < 32 ? 32 / LPR : 1;
    constexpr int kRing = kRingOf<T, VEC, NV>;
    constexpr int kPiece = LPR * VEC;                    // from one piece of a thread to the next
    const int l = threadIdx.x % LPR;
    int turn = 0;
    tcu::grid_dependents_may_start();  // the few blocks of the sums come up and wait
    const unsigned gate = blockIdx.x / (unsigned)a.blocks_per_gate;
    const unsigned end = (gate + 1) * (unsigned)a.per_gate, step = (unsigned)a.blocks_per_gate * kRows;
    const long long stride = (long long)step * a.width;
    const float inv_width = 1.f / (float)a.width;
    const int groups = (a.width + kGroup - 1) / kGroup;
    bool col[NV];
    Values<N> wp, wz, q, pb;  // pre; post times gate; sums of dout sum r and of D branch r_b
    float wf[2][N];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = l * VEC + j * kPiece;
        col[j] = c < a.width;
        V pre, post, gt;
#pragma unroll
        for (int i = 0; i < VEC; ++i) pre.v[i] = post.v[i] = gt.v[i] = from_f<T>(1.f);
        if (col[j]) {
            if (a.pre) load<T, VEC>((const T *)a.pre + c, pre.v);
            if (a.post) load<T, VEC>((const T *)a.post + c, post.v);
            if (a.gate) load<T, VEC>((const T *)a.gate + (long long)gate * a.width + c, gt.v);
        }
        float g[VEC];
        widen<T, VEC>(pre, wf[0] + j * VEC);
        widen<T, VEC>(post, wf[1] + j * VEC);
        widen<T, VEC>(gt, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) wf[1][j * VEC + i] *= g[i];
    }
    wp = Values<N>(wf[0]);
    wz = Values<N>(wf[1]);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) q.p[i] = pb.p[i] = Pair(0.f, 0.f);
    // a warp's threads walk together: row0 is the first of its rows
    const unsigned sub = LPR < 32 ? (threadIdx.x & 31) / LPR : 0;
    const unsigned row_first = gate * (unsigned)a.per_gate + blockIdx.x % (unsigned)a.blocks_per_gate * kRows +
                               threadIdx.x / (LPR < 32 ? 32 : LPR) * kPerWarp;
    long long at = (long long)(row_first + sub) * a.width + l * VEC;
    long long sat = (long long)(row_first + sub) * groups + l * VEC / kGroup;
    uint8_t *ring = (uint8_t *)shw + threadIdx.x * 16;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    // of the kept branch's values, loaded a step ahead, and as they were loaded: widened there they would be waited for there
    __nv_bfloat16 scale[NV] = {};
    auto fetch_scale = [&](unsigned row, long long from) {
        if constexpr (KEPT) {
            if (row >= end) return;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (col[j]) scale[j] = a.branch.k.scale[from + j * (kPiece / kGroup)];
        }
    };
    auto fetch = [&](unsigned row, long long from, int slot) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (row >= end || !col[j]) continue;
            const long long e = from + j * kPiece;
            const uint32_t dst = ring_at + (slot * NV + j) * kSlotBytes;
            if (a.dy) {
                ring_copy(dst, (const T *)a.dy + e);
                ring_copy(dst + 16 * kThreads, (const T *)a.sum + e);
            }
            if (a.ds) ring_copy(dst + 32 * kThreads, (const T *)a.ds + e);
            if constexpr (KEPT && kRing > 0) ring_codes<VEC>(dst + 48 * kThreads, a.branch.k.codes + e);
            else if (a.branch.p) ring_copy(dst + 48 * kThreads, (const T *)a.branch.p + e);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (kRing > 0) {
#pragma unroll
        for (int i = 0; i < kRing * NV; ++i)
            if (!col[i % NV])
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4 *>(ring + i * kSlotBytes + k * 16 * kThreads) = make_uint4(0, 0, 0, 0);
        for (int i = 0; i < kRing - 1; ++i) fetch(row_first + sub + i * step, at + i * stride, i);
    }
    fetch_scale(row_first + sub, sat);
    int slot = 0;
    for (unsigned row0 = row_first; row0 < end; row0 += step, at += stride, sat += (long long)step * groups) {
        const unsigned row = row0 + sub;
        const bool live = row < end;
        float D[N], f[N], b[N], g[N];
        if constexpr (kRing > 0) {
            fetch(row + (kRing - 1) * step, at + (kRing - 1) * stride, slot ? slot - 1 : kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        }
        // without a ring: all loads first
        V raw[kRing ? 1 : 4][kRing ? 1 : NV] = {};
        Codes codes[kRing ? 1 : NV] = {};
        if constexpr (kRing == 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const long long e = at + j * kPiece;
                const bool in = live && col[j];
                if (in && a.dy) load<T, VEC>((const T *)a.dy + e, raw[0][j].v);
                if (in && a.dy) load<T, VEC>((const T *)a.sum + e, raw[1][j].v);
                if (in && a.ds) load<T, VEC>((const T *)a.ds + e, raw[2][j].v);
                if constexpr (KEPT) {
                    if (in) codes[j] = *reinterpret_cast<const Codes *>(a.branch.k.codes + e);
                } else if (in && a.branch.p) {
                    load<T, VEC>((const T *)a.branch.p + e, raw[3][j].v);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint8_t *p = ring + (slot * NV + j) * kSlotBytes;
            float (&bj)[VEC] = *reinterpret_cast<float (*)[VEC]>(b + j * VEC);
            if constexpr (kRing == 0) {
                widen<T, VEC>(raw[0][j], g + j * VEC);
                widen<T, VEC>(raw[1][j], f + j * VEC);
                widen<T, VEC>(raw[2][j], D + j * VEC);
                if constexpr (KEPT) unkeep<VEC>(codes[j], __bfloat162float(scale[j]), bj);
                else widen<T, VEC>(raw[3][j], bj);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) D[j * VEC + i] = f[j * VEC + i] = g[j * VEC + i] = bj[i] = 0.f;
                if (!live) continue;  // zeros for the sums; past the width the ring holds them
                if (a.dy) {
                    widen<T, VEC>(*(const V *)p, g + j * VEC);
                    widen<T, VEC>(*(const V *)(p + 16 * kThreads), f + j * VEC);
                }
                if (a.ds) widen<T, VEC>(*(const V *)(p + 32 * kThreads), D + j * VEC);
                if constexpr (KEPT) unkeep<VEC>(*(const Codes *)(p + 48 * kThreads), __bfloat162float(scale[j]), bj);
                else if (a.branch.p) widen<T, VEC>(*(const V *)(p + 48 * kThreads), bj);
            }
        }
        fetch_scale(row + step, sat + (long long)step * groups);
        if constexpr (kRing > 0) slot = slot + 1 == kRing ? 0 : slot + 1;
        // the squares' sums of sum and branch and the sum of dout pre sum, together
        float sc = 1.f, scb = 1.f;
        float t[3];
        Values<N> vf, vb, vd(D);
        const Values<N> vg(g), va = times(vg, wp);
        auto stats = [&]() {
            vf = Values<N>(f);
            vb = Values<N>(b);
            t[0] = Values<N>::dot(vf, vf);
            t[1] = Values<N>::dot(va, vf);
            t[2] = a.post ? Values<N>::dot(vb, vb) : 0.f;
            team_reduce<LPR, false>(t, sh, turn);
        };
        stats();
        const bool over = t[0] > kMostSquares || !(fabsf(t[1]) <= kMostSquares), overb = t[2] > kMostSquares;
        if (__any_sync(kFull, over || overb)) {  // a team of warps comes here together: they have one row
            sc = scale_row<N, LPR>(f, over, sh, turn);
            scb = scale_row<N, LPR>(b, overb, sh, turn);
            stats();
        }
        if (a.dy) {
            const float r = rsqrtf(fmaf(t[0], inv_width, a.eps * sc * sc));  // of sum sc
            const float k = t[1] * inv_width * r * r, rd = r * sc;
            q = times_plus(vg, times(vf, r), q);
            vd = times_plus(times_plus(vf, -k, va), rd, vd);
        }
        float rb = 1.f;
        if (a.post) {
            rb = rsqrtf(fmaf(t[2], inv_width, a.eps * scb * scb));
            vb = times(vb, rb);
        }
        pb = times_plus(vd, vb, pb);
        Values<N> vz = times(vd, wz);
        if (a.dres) {
            times(vd, a.alpha).get(D);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const V o = rounded<T, VEC>(*reinterpret_cast<float (*)[VEC]>(D + j * VEC));
                if (live && col[j]) store<T, VEC>((T *)a.dres + at + j * kPiece, o.v);
            }
        }
        if (!a.dbranch) continue;
        if (a.post) {
            float bs[1] = {Values<N>::dot(vz, vb)};
            team_reduce<LPR, false>(bs, sh, turn);
            vz = times(times_plus(vb, -bs[0] * inv_width, vz), rb * scb);
        }
        vz.get(D);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const V o = rounded<T, VEC>(*reinterpret_cast<float (*)[VEC]>(D + j * VEC));
            if (live && col[j]) store<T, VEC>((T *)a.dbranch + at + j * kPiece, o.v);
        }
    }
    // the last copies land before the block's shared memory is used for other things
    if constexpr (kRing > 0) asm volatile("cp.async.wait_all;" ::: "memory");
    // a warp's rows, then the warps (or teams of warps) in order, all at once through shared memory
    constexpr int kTeam = LPR < 32 ? 32 : LPR, kTeams = kThreads / kTeam;
    const int team = threadIdx.x / kTeam;
    auto put = [&](const Values<N> &sums, float *part) {
        float v[N];
        sums.get(v);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) v[i] += __shfl_xor_sync(kFull, v[i], o);
        if ((int)threadIdx.x % kTeam < LPR)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (col[j])
#pragma unroll
                    for (int i = 0; i < VEC; ++i) shw[team * a.width + l * VEC + j * kPiece + i] = v[j * VEC + i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.width; c += kThreads) {
            float t = shw[c];
#pragma unroll
            for (int i = 1; i < kTeams; ++i) t += shw[i * a.width + c];
            part[(long long)blockIdx.x * a.width + c] = t;
        }
    };
    if (a.part_pre) put(q, a.part_pre);
    if (a.part_branch) put(pb, a.part_branch);
}

// Wide rows: a block walks the rows of its gate's part; the partial sums live in its rows of part_pre and part_branch
// (each column belongs to one thread).
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_join_bwd_wide(JoinBwdArgs a)
{
    __shared__ float sh[kThreads / 32];
    const int first = (int)threadIdx.x * VEC, stride = kThreads * VEC;
    const long long gate = blockIdx.x / a.blocks_per_gate;
    const long long begin = gate * a.per_gate, end = begin + a.per_gate;
    const long long row_first = begin + blockIdx.x % a.blocks_per_gate;
    const float inv_width = 1.f / (float)a.width;
    float *pq = a.part_pre ? a.part_pre + (long long)blockIdx.x * a.width : nullptr;
    float *pp = a.part_branch ? a.part_branch + (long long)blockIdx.x * a.width : nullptr;
    for (long long row = row_first; row < end; row += a.blocks_per_gate) {
        const long long base = row * a.width;
        auto square_sum = [&](const Source &s) {
            return [&, s](float sc) {
                float ss = 0.f;
                for (int c = first; c < a.width; c += stride) {
                    float v[VEC];
                    load_source<T, VEC>(s, row, c, a.width, v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) ss = fmaf(v[i] * sc, v[i] * sc, ss);
                }
                return ss;
            };
        };
        auto largest = [&](const Source &s) {
            return [&, s]() {
                float m = 0.f;
                for (int c = first; c < a.width; c += stride) {
                    float v[VEC];
                    load_source<T, VEC>(s, row, c, a.width, v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(v[i]));
                }
                return m;
            };
        };
        float r = 0.f, sc = 1.f, k = 0.f, rb = 1.f, scb = 1.f;
        if (a.dy) {
            const Source s = {a.sum, {nullptr, nullptr}};
            r = block_root(sh, a.width, a.eps, &sc, square_sum(s), largest(s));
            float as = 0.f;
            for (int c = first; c < a.width; c += stride) {
                float f[VEC], g[VEC], w[VEC];
                load_row<T, VEC>(a.sum, base + c, f);
                load_row<T, VEC>(a.dy, base + c, g);
                load_row<T, VEC>(a.pre, c, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) as = fmaf(g[i] * w[i], f[i] * sc * r, as);
            }
            k = block_sum(as, sh) * inv_width;
        }
        if (a.post) rb = block_root(sh, a.width, a.eps, &scb, square_sum(a.branch), largest(a.branch));
        // the columns at c: D, and the branch times its 1 / rms
        auto columns = [&](int c, float (&D)[VEC], float (&b)[VEC], float (&gu)[VEC]) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) D[i] = b[i] = gu[i] = 0.f;
            if (a.ds) load_row<T, VEC>(a.ds, base + c, D);
            if (a.dy) {
                float f[VEC], g[VEC], w[VEC];
                load_row<T, VEC>(a.sum, base + c, f);
                load_row<T, VEC>(a.dy, base + c, g);
                load_row<T, VEC>(a.pre, c, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float u = f[i] * sc * r;
                    gu[i] = g[i] * u;
                    D[i] = fmaf(r * sc, fmaf(-u, k, g[i] * w[i]), D[i]);
                }
            }
            if (a.branch.any()) {
                load_source<T, VEC>(a.branch, row, c, a.width, b);
#pragma unroll
                for (int i = 0; i < VEC; ++i) b[i] = a.post ? b[i] * scb * rb : b[i];
            }
        };
        auto through = [&](int c, float (&w)[VEC]) {  // gate post
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = 1.f;
            if (a.gate) load_row<T, VEC>(a.gate, gate * a.width + c, w);
            if (a.post) {
                float p[VEC];
                load_row<T, VEC>(a.post, c, p);
#pragma unroll
                for (int i = 0; i < VEC; ++i) w[i] *= p[i];
            }
        };
        float kb = 0.f;
        if (a.post && a.dbranch) {
            float bs = 0.f;
            for (int c = first; c < a.width; c += stride) {
                float D[VEC], b[VEC], w[VEC], gu[VEC];
                columns(c, D, b, gu);
                through(c, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) bs = fmaf(D[i] * w[i], b[i], bs);
            }
            kb = block_sum(bs, sh) * inv_width;
        }
        for (int c = first; c < a.width; c += stride) {
            float D[VEC], b[VEC], w[VEC], gu[VEC];
            Vals<T, VEC> o;
            columns(c, D, b, gu);
            if (pq) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) pq[c + i] = row == row_first ? gu[i] : pq[c + i] + gu[i];
            }
            if (pp) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) pp[c + i] = row == row_first ? D[i] * b[i] : fmaf(D[i], b[i], pp[c + i]);
            }
            if (a.dres) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) o.v[i] = from_f<T>(a.alpha * D[i]);
                store<T, VEC>((T *)a.dres + base + c, o.v);
            }
            if (a.dbranch) {
                through(c, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    o.v[i] = from_f<T>(a.post ? rb * scb * fmaf(-b[i], kb, D[i] * w[i]) : D[i] * w[i]);
                store<T, VEC>((T *)a.dbranch + base + c, o.v);
            }
        }
    }
}

struct JoinSumArgs {
    const float *part_pre, *part_branch;
    const void *post, *gate;
    float *dpre, *dpost, *dgate;  // null: not wanted
    long long gates;              // rows of dgate
    int blocks_per_gate, width, tiles;
};
// Terms added to a pair before its parts are set apart again. The low part takes what the high part's rounding leaves: left to
// itself it loses bits as it grows (2^20 terms of 0.7 a thread were 6e-5 off), and from 2^25 terms on neither part moves.
constexpr unsigned kPlain = 16;
// One block: eight columns of one output row (dpre, dpost, or a row of dgate), 32
// threads a column in a fixed order, as pairs.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_join_sums(JoinSumArgs a)
{
    __shared__ Two sh[kThreads / 32][8];
    tcu::grid_wait();
    const int c8 = threadIdx.x & 7, c = (int)(blockIdx.x % a.tiles) * 8 + c8, t = threadIdx.x >> 3;
    long long what = blockIdx.x / a.tiles;
    if (!a.dpre) ++what;
    if (!a.dpost && what > 0) ++what;
    const long long gate = what - 2;
    const float *part = what == 0 ? a.part_pre : a.part_branch;
    // up to 2^31 - 3 partial rows: an int would wrap behind the last of them
    const unsigned n = what < 2 ? (unsigned)a.gates * (unsigned)a.blocks_per_gate : (unsigned)a.blocks_per_gate;
    const long long at = what < 2 ? 0 : gate * a.blocks_per_gate;
    const bool weighted = what == 1 && a.gate;
    Two s = {0.f, 0.f};
    if (c < a.width) {
        for (unsigned i = t; i < n;) {
            const unsigned stop = min(n, i + 32 * kPlain);
#pragma unroll 4
            for (; i < stop; i += 32) {
                const float v = part[(at + i) * a.width + c];
                if (weighted) {
                    const float g = to_f<T>(((const T *)a.gate)[(long long)(i / (unsigned)a.blocks_per_gate) * a.width + c]);
                    const float p = __fmul_rn(v, g);
                    s = add(s, Two{p, __fmaf_rn(v, g, -p)});
                } else {
                    s = add(s, Two{v, 0.f});
                }
            }
            s = two_sum(s.hi, s.lo);
        }
    }
    // four of a warp's threads share a column, then the eight warps in order
    s = add(s, Two{__shfl_xor_sync(kFull, s.hi, 8), __shfl_xor_sync(kFull, s.lo, 8)});
    s = add(s, Two{__shfl_xor_sync(kFull, s.hi, 16), __shfl_xor_sync(kFull, s.lo, 16)});
    if ((threadIdx.x & 31) < 8) sh[threadIdx.x >> 5][c8] = s;
    __syncthreads();
    if (t == 0 && c < a.width) {
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) s = add(s, sh[i][c8]);
        const float v = s.hi + s.lo;
        if (what == 0) a.dpre[c] = v;
        else if (what == 1) a.dpost[c] = v;
        else a.dgate[gate * a.width + c] = a.post ? v * to_f<T>(((const T *)a.post)[c]) : v;
    }
}

pmha_status check_join_backward(const pmha_join_params *p, int64_t rows)
{
    pmha_status st = check_join("pmha_join_backward", p, rows);
    if (st != PMHA_OK) return st;
    if ((p->gates + 2) * ((p->width + 7) / 8) > ((int64_t)1 << 31) - 1) {  // blocks of one launch
        set_error("pmha_join_backward: %lld gates of width %lld are too many", (long long)p->gates, (long long)p->width);
        return PMHA_ERR_UNSUPPORTED;
    }
    return PMHA_OK;
}

// Blocks that share the rows of a gate, each of which writes a partial row: all gates' together about two a SM, which are
// resident, or as many times that as no block takes more than kSteps steps.
int64_t bwd_blocks(pmha_dtype dt, int64_t per_gate, int64_t gates, int64_t width)
{
    const Shape s = join_shape(dt, width);
    const int64_t per = s.lpr ? kThreads / s.lpr : 1, steps = (per_gate + per - 1) / per;
    const int64_t full = std::max<int64_t>(1, (int64_t)num_sms() * (s.lpr ? 2 : 4) / gates);
    return std::min(steps, full * ((steps + full * kSteps - 1) / (full * kSteps)));
}

}  // namespace
}  // namespace pmha

using namespace pmha;

extern "C" {

size_t pmha_join_backward_workspace_size(const pmha_join_params *params, int64_t rows)
{
    if (check_join_backward(params, rows) != PMHA_OK) return SIZE_MAX;
    if (rows == 0) return 0;
    const int64_t gates = params->gate ? params->gates : 1;
    const size_t one = (size_t)(bwd_blocks(params->dtype, rows / gates, gates, params->width) * gates) *
                       (size_t)params->width * 4;
    return 2 * ((one + 255) & ~(size_t)255);
}

pmha_status pmha_join_backward(const pmha_join_params *params, int64_t rows, const void *branch,
                               const pmha_kept *branch_kept, const void *sum, const void *dout, const void *dsum,
                               void *dbranch, void *dresidual, float *dpost, float *dgate, float *dpre, void *workspace,
                               size_t workspace_bytes, pmha_stream stream)
{
    pmha_status st = check_join_backward(params, rows);
    if (st != PMHA_OK) return st;
    const pmha_join_params &p = *params;
    cudaStream_t cs = (cudaStream_t)stream;
    const int64_t w = p.width, gates = p.gate ? p.gates : 1;
    if (!aligned(dpost, 16) || !aligned(dgate, 16) || !aligned(dpre, 16) || (dpost && !p.post) || (dgate && !p.gate) ||
        (dpre && !p.pre)) {
        set_error("pmha_join_backward: dpost, dgate or dpre is not 16-byte aligned, or has no parameter");
        return PMHA_ERR_INVALID_ARG;
    }
    if (rows == 0) {
        if (dpost) PMHA_CUDA_TRY(cudaMemsetAsync(dpost, 0, (size_t)w * 4, cs));
        if (dgate) PMHA_CUDA_TRY(cudaMemsetAsync(dgate, 0, (size_t)(w * gates) * 4, cs));
        if (dpre) PMHA_CUDA_TRY(cudaMemsetAsync(dpre, 0, (size_t)w * 4, cs));
        return PMHA_OK;
    }
    const bool need_branch = (p.post && dbranch) || dpost || dgate;
    if ((branch && branch_kept) || (need_branch && !branch && !branch_kept) || (dout != nullptr) != (p.pre != nullptr) ||
        (dout && !sum) || (!dout && !dsum)) {
        set_error("pmha_join_backward: needs one form of the branch (with post or a gate's gradient), dout and sum just if "
                  "pre is set, and dout or dsum");
        return PMHA_ERR_INVALID_ARG;
    }
    if (!aligned(branch, 16) || !whole(branch_kept) || !aligned(sum, 16) || !aligned(dout, 16) || !aligned(dsum, 16) ||
        !aligned(dbranch, 16) || !aligned(dresidual, 16)) {
        set_error("pmha_join_backward: a pointer is not 16-byte aligned, or the kept branch lacks its codes or scales");
        return PMHA_ERR_INVALID_ARG;
    }
    const size_t nb = (size_t)(rows * w) * bytes_of(p.dtype), wb = (size_t)w * bytes_of(p.dtype), fb = (size_t)w * 4;
    const Span ins[] = {{branch, nb}, codes_of(branch_kept, rows, w), scales_of(branch_kept, rows, w), {sum, nb},
                        {dout, nb}, {dsum, nb}, {p.post, wb}, {p.pre, wb}, {p.gate, wb * (size_t)p.gates}};
    const Span outs[] = {{dbranch, nb}, {dresidual, nb}, {dpost, fb}, {dgate, fb * (size_t)gates}, {dpre, fb}};
    if (any_overlap(ins, outs)) {
        set_error("pmha_join_backward: an output overlaps an input or another output");
        return PMHA_ERR_INVALID_ARG;
    }
    if (!dbranch && !dresidual && !dpost && !dgate && !dpre) return PMHA_OK;
    const bool sums = dpost || dgate || dpre;
    const size_t need = pmha_join_backward_workspace_size(params, rows);
    if (sums && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))) {
        set_error("pmha_join_backward: workspace needs %zu bytes, 256-byte aligned (got %zu at %p)", need, workspace_bytes,
                  workspace);
        return PMHA_ERR_WORKSPACE;
    }
    const int64_t per_gate = rows / gates, blocks = bwd_blocks(p.dtype, per_gate, gates, w);
    float *part_pre = dpre ? (float *)workspace : nullptr;
    float *part_branch = dpost || dgate ? (float *)((uint8_t *)workspace + need / 2) : nullptr;
    Source b = source(branch, branch_kept);
    if (!need_branch) b = Source{nullptr, {nullptr, nullptr}};
    JoinBwdArgs a{b, sum, dout, dsum, p.post, p.gate, p.pre, dbranch, dresidual, part_pre, part_branch, per_gate,
                  (int)blocks, (int)w, p.residual_scale, p.eps};
    if (!need_branch) a.post = nullptr;
    const Shape s = join_shape(p.dtype, w);
    const unsigned grid = (unsigned)(blocks * gates);
    cudaError_t attr = cudaSuccess;
    {
        StageTimer timer(branch_kept ? "join_backward_kept" : "join_backward", cs);
        if (s.lpr)
            join_dispatch(p.dtype, s, [&](auto t) {
                using G = decltype(t);
                using T = typename G::type;
                // the ring, and in its place at the end the teams' sums
                const size_t smem = std::max((size_t)w * 4 * (kThreads / std::max(G::lpr, 32)), kRingBytes<T, G::vec, G::nv>);
                auto kern = b.k.codes ? k_join_bwd<T, G::vec, G::nv, G::lpr, true> : k_join_bwd<T, G::vec, G::nv, G::lpr, false>;
                attr = smem > 48 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                        : cudaSuccess;
                if (attr == cudaSuccess) kern<<<grid, kThreads, smem, cs>>>(a);
            });
        else
            dispatch_wide(p.dtype, s.vec, [&](auto t) {
                using G = decltype(t);
                k_join_bwd_wide<typename G::type, G::vec><<<grid, kThreads, 0, cs>>>(a);
            });
    }
    PMHA_CUDA_TRY(attr);
    count_launch();
    PMHA_CUDA_TRY(cudaGetLastError());
    if (sums) {
        StageTimer timer("join_sums", cs);
        const int tiles = (int)((w + 7) / 8);
        const int64_t outs_n = (dpre ? 1 : 0) + (dpost ? 1 : 0) + (dgate ? gates : 0);
        JoinSumArgs q{part_pre, part_branch, p.post, p.gate, dpre, dpost, dgate, gates, (int)blocks, (int)w, tiles};
        const unsigned n = (unsigned)(outs_n * tiles);
        st = p.dtype == PMHA_BF16 ? tcu::launch_overlapping(k_join_sums<__nv_bfloat16>, dim3(n), kThreads, 0, cs, q)
                                  : tcu::launch_overlapping(k_join_sums<float>, dim3(n), kThreads, 0, cs, q);
        if (st != PMHA_OK) return st;
    }
    return PMHA_OK;
}

}  // extern "C"
