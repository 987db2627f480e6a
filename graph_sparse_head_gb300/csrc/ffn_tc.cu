// Tensor-core products of the gated feed-forward block (sm_103a), one kernel
// shape for all five:
//
//   up      h = act(x Wg^T + bg) * (x Wu^T + bu)      tile 256 tokens x 128 hidden, gate and up side by side
//   down    y = h Wd^T + bd + residual                tile 256 tokens x 128 or 256 outputs
//   hidden  h, dg, du of the backward pass            tile 256 tokens x 64 hidden, three products
//   dx      dg Wg + du Wu                             the down kernel with two pairs of operands
//   dw      dg^T x, du^T x, h^T dy                    tile 256 hidden x 128 or 256 columns, operands as they lie
//
// Two CTAs form a pair (tc_pair.cuh). Each has 18 warps: warp 0 copies
// 128-byte-wide operand tiles by TMA into a ring of stages, warp 1 of the even
// CTA issues tcgen05.mma into accumulators in tensor memory (two, so that the
// products of one tile run under the epilogue of the last), and sixteen
// warps turn accumulators into outputs: each thread reads its part of its
// row's columns, applies the tile's arithmetic, writes the result to a
// swizzled tile in shared memory, and one thread stores that by TMA. Pairs are
// persistent and take tiles in order, the column tiles of one row block side
// by side, so that the rows come from L2 after their first read.
//
// Ragged sizes need no code of their own: TMA fills rows and columns past a
// tensor's end with zeros and does not store them.
//
// Every mbarrier wait is bounded (tc_util.cuh); on expiry the pair gives up,
// waits for its copies and products, frees its tensor memory and returns, and
// pmha_device_status reports PMHA_ERR_TIMEOUT.
#include <algorithm>

#include "ffn_internal.h"
#include "ffn_math.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {
using namespace tcu;

constexpr int kThreads = 64 + 512;
constexpr int kBox = 128 * 128;  // bytes of a tile of 128 rows of 128 bytes
enum Kind { kUp, kUpQ8, kDown, kHidden, kDw };

// Bytes of a stage and its parts for one CTA, per kind and column tile BN.
template <int KIND, int BN>
struct Cfg {
    static constexpr bool kQ8 = KIND == kUpQ8;
    static constexpr bool kIsUp = KIND == kUp || KIND == kUpQ8;
    static constexpr int kA = KIND == kHidden ? 2 * kBox : kBox;        // x (and dy), or 128 columns of an M-major A
    static constexpr int kB = KIND == kHidden ? kBox / 2 + kBox / 4     // 64 rows of Wg or Wu, 32 of Wd^T
                              : kIsUp ? kBox                            // 128 rows of Wg or Wu
                                      : BN / 2 * 128;                   // half of the columns
    static constexpr int kStage = kA + kB;
    static constexpr int kCols = kIsUp ? 128 : KIND == kHidden ? 64 : BN;  // output columns of a tile
    // The up product's arithmetic outweighs its products: two teams of eight warps take the tiles in turn, so that
    // one team's waits run under the other's arithmetic. Elsewhere one team of sixteen shares every tile.
    static constexpr int kTeams = kIsUp ? 2 : 1;
    static constexpr int kPart = kCols * kTeams / 4;  // columns of one of a team's groups of four warps
    static constexpr int kTile = KIND == kHidden ? 3 * kBox : KIND == kDw ? 0 : kCols / 64 * kBox;  // output tile
    static constexpr int kTiles = kTile <= 2 * kBox ? 2 : 1;  // output tiles in shared memory
    static constexpr int kAccCols = KIND == kHidden ? 192 : kIsUp ? 256 : KIND == kDw ? 2 * BN : BN;
    static constexpr int kAccStride = kAccCols > 256 ? 512 : kAccCols > 128 ? 256 : 128;
    static constexpr int kAccs = kAccStride == 512 || KIND == kDw ? 1 : 2;
    static constexpr int kTmemCols = kAccs * kAccStride;
    static constexpr int kVec = KIND == kDw ? 4096 : 2 * 4 * 128 * 4;  // bias and scale columns of two tiles, or ones
    static constexpr int kBars = 512;
    static constexpr int kFit = (232448 - 1024 - kTiles * kTile - kVec - kBars) / kStage;
    static constexpr int kStages = kFit > 7 ? 7 : kFit;
    static constexpr int kSmem = 1024 + kStages * kStage + kTiles * kTile + kVec + kBars;
    static_assert(kStages >= 3, "a ring of at least three stages");
    static_assert(kSmem <= 232448, "shared memory of one CTA");
};

struct Params {
    CUtensorMap a0, a1, a2, b0, b1, b2, o0, o1, o2, res;
    int M, E, F;            // tokens (dw: hidden rows of the result), outer and hidden width
    int n_tiles, tiles_n;   // pair tiles, column tiles of one row block
    int kb;                 // K blocks of one operand pair
    int segs;               // operand pairs (down: 1; dx: 2)
    const __nv_bfloat16 *bias0, *bias1;
    const float *xs, *gs, *us;
    int has_res;
    // dw: row blocks of 64 tokens dealt to the splits; products from first_what on
    int splits, tiles_m, first_what, accumulate;
    float *part, *sums;     // dw: partial products; column sums of dy (split, E) or null. hidden: see FfnHiddenArgs
    int *err;
};

// accumulator columns of this warp's 32 rows
__device__ __forceinline__ uint32_t tmem_at(uint32_t base, int quarter, int col)
{
    return base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)col;
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps the uses of r behind the wait above.
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// named barrier 1 + team over its threads
template <int THREADS>
__device__ __forceinline__ void team_sync(int team)
{
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(THREADS) : "memory");
}

__device__ __forceinline__ void four(float (&f)[4], const float *p)
{
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}

// Partial sums: one CTA owns each value and the launches that add to it follow
// one another, so the additions' order is fixed; they need no read of their own.
__device__ __forceinline__ void put4(float *p, float a, float b, float c, float d, bool add)
{
    if (add)
        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
    else
        *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void put1(float *p, float a, bool add)
{
    if (add) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(p), "f"(a) : "memory");
    else *p = a;
}

template <int KIND, int BN, int ACT>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) k_ffn(const __grid_constant__ Params p)
{
    using C = Cfg<KIND, BN>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *out_s = smem + kStages * C::kStage;
    float *vec_s = (float *)(out_s + C::kTiles * C::kTile);     // [2][4][128]; dw: 4 KB of bf16 ones
    uint64_t *full = (uint64_t *)((uint8_t *)vec_s + C::kVec);  // [kStages], counted in the even CTA
    uint64_t *empty = full + kStages;                           // [kStages], in each CTA
    uint64_t *acc_full = empty + kStages;                       // [2], in each CTA
    uint64_t *acc_empty = acc_full + 2;                         // [2], counted in the even CTA
    uint64_t *mma_done = acc_empty + 2;
    uint64_t *res_full = mma_done + 1;                          // the residual's tile
    uint32_t *tmem_holder = (uint32_t *)(res_full + 1);
    volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
    volatile uint32_t *armed = (volatile uint32_t *)(tmem_holder + 2);  // copies counted

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), 2);  // the epilogue of either CTA
        }
        mbar_init(smem_u32(mma_done), 1);
        mbar_init(smem_u32(res_full), 1);
        *abort_flag = 0;
        *armed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), C::kTmemCols);
    if constexpr (KIND == kDw) {
        for (int i = threadIdx.x; i < 1024; i += kThreads) ((uint32_t *)vec_s)[i] = 0x3f803f80u;
        fence_async_shared();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    grid_dependency_wait();
    const uint32_t tmem = *tmem_holder;

    // tile -> (row block of 256, column tile, K blocks, product of dw)
    auto decode = [&](int tile, int &m, int &n, int &kb0, int &kb1, int &what) {
        kb0 = 0;
        kb1 = KIND == kDown ? p.segs * p.kb : p.kb;
        what = 0;
        if constexpr (KIND == kDw) {
            const int per = p.tiles_m * p.tiles_n;
            const int split = tile % p.splits;
            tile /= p.splits;
            what = p.first_what + tile / per;
            tile %= per;
            kb1 = (p.kb - split + p.splits - 1) / p.splits;  // row blocks split, split + splits, ... from the end
        }
        m = tile / p.tiles_n;
        n = tile % p.tiles_n;
    };

    if (warp == 0) {
        // ---------------- TMA producer of this CTA
        const bool one = elect_one();
        uint32_t made = 0;
        for (int tile = pair; tile < p.n_tiles && !*abort_flag; tile += n_pairs) {
            int m, n, kb0, kb1, what;
            decode(tile, m, n, kb0, kb1, what);
            const int row = m * 256 + (int)rank * 128;
            for (int kb = kb0; kb < kb1; ++kb, ++made) {
                const int stage = (int)(made % kStages);
                if (!wait_bar(smem_u32(&empty[stage]), ((made / kStages) & 1u) ^ 1u, abort_flag, p.err)) break;
                if (!one) continue;
                const uint32_t fb = map_rank(smem_u32(&full[stage]), 0);
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * C::kStage);
                *armed = made + 1;
                const uint32_t sa = smem_u32(smem + stage * C::kStage), sb = sa + C::kA;
                if constexpr (C::kIsUp) {
                    constexpr int kElems = C::kQ8 ? 128 : 64;
                    tma_load_2d_pair(sa, &p.a0, kb * kElems, row, fb);
                    tma_load_2d_pair(sb, rank ? &p.b1 : &p.b0, kb * kElems, n * 128, fb);
                } else if constexpr (KIND == kHidden) {
                    tma_load_2d_pair(sa, &p.a0, kb * 64, row, fb);
                    tma_load_2d_pair(sa + kBox, &p.a1, kb * 64, row, fb);
                    tma_load_2d_pair(sb, rank ? &p.b1 : &p.b0, kb * 64, n * 64, fb);
                    tma_load_2d_pair(sb + kBox / 2, &p.b2, kb * 64, n * 64 + (int)rank * 32, fb);
                } else if constexpr (KIND == kDown) {
                    const bool second = kb >= p.kb;
                    const int k = (second ? kb - p.kb : kb) * 64;
                    tma_load_2d_pair(sa, second ? &p.a1 : &p.a0, k, row, fb);
                    tma_load_2d_pair(sb, second ? &p.b1 : &p.b0, k, n * BN + (int)rank * (BN / 2), fb);
                } else {
                    // the last rows first: they were written last and are still in L2
                    const int k0 = (p.kb - 1 - (tile % p.splits) - kb * p.splits) * 64;
                    const CUtensorMap *ma = what == 0 ? &p.a0 : what == 1 ? &p.a1 : &p.a2;
                    const CUtensorMap *mb = what == 2 ? &p.b1 : &p.b0;
                    tma_load_2d_pair(sa, ma, row, k0, fb);
                    tma_load_2d_pair(sa + kBox / 2, ma, row + 64, k0, fb);
#pragma unroll
                    for (int j = 0; j < BN / 128; ++j)
                        tma_load_2d_pair(sb + j * (kBox / 2), mb, n * BN + (int)rank * (BN / 2) + j * 64, k0, fb);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer of the pair: the whole warp walks, so that addresses stay in uniform
            // registers; one lane issues
            const bool one = elect_one();
            uint32_t used = 0, i = 0;
            bool ok = true;
            for (int tile = pair; tile < p.n_tiles && ok; tile += n_pairs, ++i) {
                int m, n, kb0, kb1, what;
                decode(tile, m, n, kb0, kb1, what);
                const int acc = (int)(i % C::kAccs);
                if (!wait_bar(smem_u32(&acc_empty[acc]), ((i / C::kAccs) & 1u) ^ 1u, abort_flag, p.err)) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * C::kAccStride);
                for (int kb = kb0; kb < kb1; ++kb, ++used) {
                    const int stage = (int)(used % kStages);
                    ok = wait_bar(smem_u32(&full[stage]), (used / kStages) & 1u, abort_flag, p.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + stage * C::kStage), sb = sa + C::kA;
                    const uint32_t more = kb > kb0 ? 1u : 0u;
                    if (one) {
                        if constexpr (KIND == kDw) {
                            const uint64_t da = smem_desc_mn(sa, kBox / 2), db = smem_desc_mn(sb, kBox / 2);
                            // a tile of ones takes the place of an operand for the column sums of dy, beside the
                            // first row block of h^T dy
                            const uint64_t ones = smem_desc_mn(smem_u32(vec_s), 2048);
                            const bool cols = p.sums && what == 2 && m == 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {  // 16 tokens = 2048 bytes
                                const uint64_t ak = da + (uint64_t)(128 * k), bk = db + (uint64_t)(128 * k);
                                mma_pair<false>(d, ak, bk, idesc_of(false, true, 256, BN), more | (k > 0));
                                if (cols) mma_pair<false>(d + BN, ones, bk, idesc_of(false, true, 256, BN), more | (k > 0));
                            }
                        } else {
                            const uint64_t da = smem_desc(sa), db = smem_desc(sb);
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 32 bytes along K = 2 in the address field
                                mma_pair<C::kQ8>(d, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k),
                                                 idesc_of(C::kQ8, false, 256, KIND == kHidden ? 128 : C::kAccCols),
                                                 more | (k > 0));
                            if constexpr (KIND == kHidden) {
                                const uint64_t da1 = smem_desc(sa + kBox), db1 = smem_desc(sb + kBox / 2);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_pair<false>(d + 128, da1 + (uint64_t)(2 * k), db1 + (uint64_t)(2 * k),
                                                    idesc_of(false, false, 256, 64), more | (k > 0));
                            }
                        }
                        mma_commit_pair(smem_u32(&empty[stage]));
                    }
                    __syncwarp();
                }
                if (one && ok) mma_commit_pair(smem_u32(&acc_full[acc]));
                __syncwarp();
            }
            if (one) mma_commit_pair(smem_u32(mma_done));
            __syncwarp();
            int dummy = 0;
            mbar_wait(smem_u32(mma_done), 0, (volatile int *)&dummy, p.err);
        }
    } else {
        // ---------------- epilogue: teams of warps in groups of four, each group its part of a tile's columns
        constexpr int kTeam = 512 / C::kTeams;
        const int team = (threadIdx.x - 64) / kTeam, et = (threadIdx.x - 64) % kTeam;
        const int quarter = warp & 3, part = et >> 7;
        auto epi_sync = [&]() { team_sync<kTeam>(team); };
        const bool lead = et == 0;
        const int r = quarter * 32 + lane;  // row within this CTA's 128
        const int cp = part * C::kPart;     // first column within the tile
        uint32_t i = (uint32_t)team;
        for (int tile = pair + team * n_pairs; tile < p.n_tiles; tile += C::kTeams * n_pairs, i += C::kTeams) {
            const int acc = (int)(i % C::kAccs);
            int m, n, kb0, kb1, what;
            decode(tile, m, n, kb0, kb1, what);
            const int row0 = m * 256 + (int)rank * 128, c0 = n * C::kCols;
            uint8_t *tile_s = out_s + (i % C::kTiles) * C::kTile;
            float *v0 = vec_s + (i & 1u) * 512, *v1 = v0 + 128, *s0 = v0 + 256, *s1 = v0 + 384;
            float xs[4] = {};  // of rows g + 8 i of the warp's
            if constexpr (KIND != kDw) {
                // bias and scales of the tile's columns, and the residual's tile, under the products
                constexpr float kg = C::kIsUp ? Act<ACT>::kGate : 1.f, ku = C::kIsUp ? Act<ACT>::kUp : 1.f;
                const int limit = KIND == kDown ? p.E : p.F;
                const bool in = et < C::kCols && c0 + et < limit;
                const float b0 = p.bias0 && in ? kg * __bfloat162float(p.bias0[c0 + et]) : 0.f;
                float b1 = 0.f, g0 = 0.f, g1 = 0.f;
                if constexpr (KIND != kDown) b1 = p.bias1 && in ? ku * __bfloat162float(p.bias1[c0 + et]) : 0.f;
                if constexpr (C::kQ8) {
                    g0 = in ? kg * p.gs[c0 + et] : 0.f;
                    g1 = in ? ku * p.us[c0 + et] : 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = row0 + quarter * 32 + 8 * k + (lane >> 2);
                        xs[k] = row < p.M ? p.xs[row] : 0.f;
                    }
                }
                if (lead) {
                    // this thread's last store that used the tile has read it
                    if constexpr (C::kTiles == 2 && C::kTeams == 1) store_wait_read1();
                    else store_wait_read();
                    if constexpr (KIND == kDown)
                        if (p.has_res) {
                            uint32_t bytes = 0;
                            for (int j = 0; j < C::kCols / 64; ++j)
                                bytes += row0 < p.M && c0 + j * 64 < p.E ? kBox : 0;
                            if (bytes) mbar_arrive_expect_tx(smem_u32(res_full), bytes);
                            else mbar_arrive(smem_u32(res_full));
                            for (int j = 0; j < C::kCols / 64; ++j)
                                if (row0 < p.M && c0 + j * 64 < p.E)
                                    tma_load_2d(smem_u32(tile_s + j * kBox), &p.res, c0 + j * 64, row0,
                                                smem_u32(res_full));
                        }
                }
                if constexpr (KIND == kDown) {
                    // BN columns of one vector: [256] across v0 and v1
                    if (et < C::kCols) v0[et] = b0;
                } else if (et < C::kCols) {
                    v0[et] = b0;
                    v1[et] = b1;
                    if constexpr (C::kQ8) {
                        s0[et] = g0;
                        s1[et] = g1;
                    }
                }
                epi_sync();
            }
            // after an expired wait the waits return at once and the loop runs out
            wait_bar(smem_u32(&acc_full[acc]), (i / C::kAccs) & 1u, abort_flag, p.err);
            if constexpr (KIND == kDown)
                if (p.has_res) wait_bar(smem_u32(res_full), i & 1u, abort_flag, p.err);
            tc_fence_after();
            const uint32_t t0 = tmem_at(tmem, quarter, acc * C::kAccStride);
            if constexpr (KIND == kDw) {
                const int split = tile % p.splits, f = row0 + r;
                float *dst = p.part + ((size_t)split * 3 + what) * (size_t)p.F * p.E;
                float *sums = p.sums ? p.sums + (size_t)split * p.E : nullptr;
                const bool some = kb1 > kb0, add = p.accumulate;  // without tokens: zeros
#pragma unroll 1
                for (int c = cp; c < cp + C::kPart; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(t0 + (uint32_t)c, v);
                    tmem_wait();
                    pin(v);
                    if (f >= p.F || c0 + c >= p.E) continue;
                    float *d = dst + (size_t)f * p.E + c0 + c;
#pragma unroll
                    for (int q = 0; q < 16; q += 4)
                        if (c0 + c + q < p.E) {
                            if (some)
                                put4(d + q, __uint_as_float(v[q]), __uint_as_float(v[q + 1]), __uint_as_float(v[q + 2]),
                                     __uint_as_float(v[q + 3]), add);
                            else if (!add)
                                put4(d + q, 0.f, 0.f, 0.f, 0.f, false);
                        }
                }
                if (sums && what == 2 && m == 0 && quarter == 0) {  // every row holds the sums: lane 0 writes
#pragma unroll 1
                    for (int c = cp; c < cp + C::kPart; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(t0 + (uint32_t)(BN + c), v);
                        tmem_wait();
                        pin(v);
                        if (lane == 0 && rank == 0 && (some || !add))
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                if (c0 + c + q < p.E) put1(sums + c0 + c + q, some ? __uint_as_float(v[q]) : 0.f, add);
                    }
                }
            } else if constexpr (C::kIsUp) {
#pragma unroll 1
                for (int c = cp; c < cp + C::kPart; c += 16) {
                    uint32_t vg[2][8], vu[2][8];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        tmem_ld_frag(t0 + ((uint32_t)(q * 16) << 16) + (uint32_t)c, vg[q]);
                        tmem_ld_frag(t0 + ((uint32_t)(q * 16) << 16) + (uint32_t)(128 + c), vu[q]);
                    }
                    const int c2 = c + 2 * (lane & 3);
                    float bg[4], bu[4], sg[4], su[4];
                    two_pairs(bg, v0 + c2);
                    two_pairs(bu, v1 + c2);
                    if constexpr (C::kQ8) {
                        two_pairs(sg, s0 + c2);
                        two_pairs(su, s1 + c2);
                    }
                    tmem_wait();
                    // this lane's row of the four 8 x 8 matrices of 16 rows x 16 columns
                    const uint32_t at = smem_u32(tile_s + (c / 64) * kBox) +
                                        swizzled(quarter * 32 + (lane & 15), (c % 64) / 8 + (lane >> 4));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        pin(vg[q]);
                        pin(vu[q]);
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            float h[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int k = (j >> 2) * 2 + e;
                                const float a = __uint_as_float(vg[q][j + e]), b = __uint_as_float(vu[q][j + e]);
                                if constexpr (C::kQ8) {
                                    const float x = xs[2 * q + ((j >> 1) & 1)];
                                    h[e] = Act<ACT>::hidden(fmaf(a, x * sg[k], bg[k]), fmaf(b, x * su[k], bu[k]));
                                } else {
                                    h[e] = Act<ACT>::hidden(fmaf(a, Act<ACT>::kGate, bg[k]),
                                                            fmaf(b, Act<ACT>::kUp, bu[k]));
                                }
                            }
                            w[j / 2] = pack_bf16(h[0], h[1]);
                        }
                        store_frags(at + (uint32_t)(q * 16 * 128), w[0], w[1], w[2], w[3]);
                    }
                }
            } else if constexpr (KIND == kHidden) {
                float cs[8] = {};
                const int t2 = cp + 2 * (lane & 3);
                float bg[4], bu[4];
                two_pairs(bg, v0 + t2);
                two_pairs(bu, v1 + t2);
                // this lane's row of the four 8 x 8 matrices of 16 rows x 16 columns
                const uint32_t at0 = smem_u32(tile_s) + swizzled(quarter * 32 + (lane & 15), cp / 8 + (lane >> 4));
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // 16 of the warp's rows
                    uint32_t vg[8], vu[8], vd[8], w[3][4];
                    const uint32_t tq = t0 + ((uint32_t)(q * 16) << 16) + (uint32_t)cp;
                    tmem_ld_frag(tq, vg);
                    tmem_ld_frag(tq + 64, vu);
                    tmem_ld_frag(tq + 128, vd);
                    tmem_wait();
                    pin(vg);
                    pin(vu);
                    pin(vd);
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float h[2], dg[2], du[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int c = (j >> 2) * 2 + e;
                            const float b = __uint_as_float(vu[j + e]) + bu[c], dh = __uint_as_float(vd[j + e]);
                            float slope;
                            const float act = Act<ACT>::fast(__uint_as_float(vg[j + e]) + bg[c], &slope);
                            h[e] = act * b;
                            dg[e] = dh * b * slope;
                            du[e] = dh * act;
                            cs[c] += dg[e];
                            cs[4 + c] += du[e];
                        }
                        w[0][j / 2] = pack_bf16(h[0], h[1]);
                        w[1][j / 2] = pack_bf16(dg[0], dg[1]);
                        w[2][j / 2] = pack_bf16(du[0], du[1]);
                    }
#pragma unroll
                    for (int o = 0; o < 3; ++o)
                        store_frags(at0 + (uint32_t)(o * kBox + q * 16 * 128), w[o][0], w[o][1], w[o][2], w[o][3]);
                }
                if (p.sums)
                    add_column_sums(p.sums + (size_t)(blockIdx.x * 4 + quarter) * 2 * p.F, cs, c0 + cp, p.F, lane);
            } else {
#pragma unroll 1
                for (int c = cp; c < cp + C::kPart; c += 16) {
                    uint32_t v[16], w[8];
                    tmem_ld16(t0 + (uint32_t)c, v);
                    tmem_wait();
                    pin(v);
                    uint8_t *sb = tile_s + (c / 64) * kBox;
                    uint4 *p0 = reinterpret_cast<uint4 *>(sb + swizzled(r, (c % 64) / 8));
                    uint4 *p1 = reinterpret_cast<uint4 *>(sb + swizzled(r, (c % 64) / 8 + 1));
                    uint32_t rw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (p.has_res) {
                        const uint4 a = *p0, b = *p1;
                        rw[0] = a.x, rw[1] = a.y, rw[2] = a.z, rw[3] = a.w;
                        rw[4] = b.x, rw[5] = b.y, rw[6] = b.z, rw[7] = b.w;
                    }
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float b[4];
                        four(b, v0 + c + 2 * j);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            w[j + e] = pack_bf16(__uint_as_float(v[2 * (j + e)]) + b[2 * e] + __uint_as_float(rw[j + e] << 16),
                                                 __uint_as_float(v[2 * (j + e) + 1]) + b[2 * e + 1] +
                                                     __uint_as_float(rw[j + e] & 0xffff0000u));
                    }
                    *p0 = make_uint4(w[0], w[1], w[2], w[3]);
                    *p1 = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            // the accumulator is read: back to the issuer, once in each CTA; the tile goes out
            tc_fence_before();
            if constexpr (KIND != kDw) fence_async_shared();
            epi_sync();
            if (lead) {
                mbar_arrive_cluster(map_rank(smem_u32(&acc_empty[acc]), 0));
                if constexpr (KIND == kHidden) {
                    if (row0 < p.M) {
                        tma_store_tile(&p.o0, smem_u32(tile_s), c0, row0);
                        tma_store_tile(&p.o1, smem_u32(tile_s + kBox), c0, row0);
                        tma_store_tile(&p.o2, smem_u32(tile_s + 2 * kBox), c0, row0);
                    }
                } else if constexpr (KIND != kDw) {
                    const int limit = KIND == kDown ? p.E : p.F;
                    for (int j = 0; j < C::kCols / 64; ++j)
                        if (row0 < p.M && c0 + j * 64 < limit)
                            tma_store_tile(&p.o0, smem_u32(tile_s + j * kBox), c0 + j * 64, row0);
                }
                if constexpr (KIND != kDw) store_commit();
            }
        }
        if (lead && KIND != kDw) {
            store_wait_all();  // shared memory outlives its stores, and after an expired wait the residual's copy
            int dummy = 0;
            if (KIND == kDown && *abort_flag && p.has_res && i)
                mbar_wait(smem_u32(res_full), (i - 1) & 1u, (volatile int *)&dummy, p.err);
        }
    }

    __syncthreads();
    if (threadIdx.x == 0) {
        // every product has run before either CTA goes; after an expired wait the counted copies land first
        int dummy = 0;
        mbar_wait(smem_u32(mma_done), 0, (volatile int *)&dummy, p.err);
        if (*abort_flag && rank == 0)
            for (uint32_t i = *armed > kStages ? *armed - kStages : 0; i < *armed; ++i)
                mbar_wait(smem_u32(&full[i % kStages]), (i / kStages) & 1u, (volatile int *)&dummy, p.err);
    }
    __syncthreads();
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free_pair(tmem, C::kTmemCols);
}

// ---------------------------------------------------------------- host side

template <int KIND, int BN, int ACT>
pmha_status launch(Params &p, const char *stage, cudaStream_t s)
{
    using C = Cfg<KIND, BN>;
    p.err = device_error_word();
    if (!p.err) return PMHA_ERR_CUDA;
    int pairs = 0;
    auto kern = k_ffn<KIND, BN, ACT>;
    static std::atomic<int> known[kKnownDevices];
    const pmha_status st = pairs_at_once(kern, kThreads, C::kSmem, known, &pairs);
    if (st != PMHA_OK) return st;
    StageTimer timer(stage, s);
    return launch_overlapping(kern, dim3(2u * (unsigned)std::min(pairs, p.n_tiles)), kThreads, C::kSmem, s, p);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

pmha_status map_failed(const char *what)
{
    set_error("%s: cuTensorMapEncodeTiled failed", what);
    return PMHA_ERR_CUDA;
}

pmha_status too_large(const char *what, int64_t tiles)
{
    set_error("%s: %lld tiles exceed the 32-bit tile index", what, (long long)tiles);
    return PMHA_ERR_INVALID_ARG;
}

// 256 outputs a tile where there are that many; else 128 (less waste)
bool wide_tiles(int64_t n) { return n % 256 == 0 || n > 512; }

pmha_status down_like(const FfnTc &f, const void *a0, const void *a1, const void *b0, const void *b1, const void *bias,
                      const void *residual, int64_t M, void *out, const char *stage, cudaStream_t s)
{
    Params p = {};
    const bool wide = wide_tiles(f.E);
    const int bn = wide ? 256 : 128;
    p.M = (int)M, p.E = (int)f.E, p.F = (int)f.F;
    p.tiles_n = (int)ceil_div(f.E, bn);
    const int64_t tiles = ceil_div(M, 256) * p.tiles_n;
    if (tiles > 0x3fffffff) return too_large(stage, tiles);
    p.n_tiles = (int)tiles;
    p.kb = (int)ceil_div(f.F, 64);
    p.segs = a1 ? 2 : 1;
    p.bias0 = (const __nv_bfloat16 *)bias;
    p.has_res = residual != nullptr;
    bool ok = make_tile_map(&p.a0, a0, M, f.F, f.F, 2, 128) && make_tile_map(&p.b0, b0, f.E, f.F, f.F, 2, bn / 2) &&
              make_tile_map(&p.o0, out, M, f.E, f.E, 2, 128);
    if (a1) ok = ok && make_tile_map(&p.a1, a1, M, f.F, f.F, 2, 128) && make_tile_map(&p.b1, b1, f.E, f.F, f.F, 2, bn / 2);
    if (residual) ok = ok && make_tile_map(&p.res, residual, M, f.E, f.E, 2, 128);
    if (!ok) return map_failed(stage);
    return wide ? launch<kDown, 256, 0>(p, stage, s) : launch<kDown, 128, 0>(p, stage, s);
}

}  // namespace

pmha_status ffn_tc_up(const FfnTc &f, const FfnUpArgs &a, cudaStream_t s)
{
    Params p = {};
    const bool q8 = a.x_scale != nullptr;
    p.M = (int)a.M, p.E = (int)f.E, p.F = (int)f.F;
    p.tiles_n = (int)ceil_div(f.F, 128);
    const int64_t tiles = ceil_div(a.M, 256) * p.tiles_n;
    if (tiles > 0x3fffffff) return too_large("ffn_up", tiles);
    p.n_tiles = (int)tiles;
    p.kb = (int)ceil_div(f.E, q8 ? 128 : 64);
    p.bias0 = (const __nv_bfloat16 *)f.bg;
    p.bias1 = (const __nv_bfloat16 *)f.bu;
    p.xs = a.x_scale, p.gs = a.wg_scale, p.us = a.wu_scale;
    const int es = q8 ? 1 : 2;
    if (!make_tile_map(&p.a0, a.x, a.M, f.E, f.E, es, 128) || !make_tile_map(&p.b0, a.wg, f.F, f.E, f.E, es, 128) ||
        !make_tile_map(&p.b1, a.wu, f.F, f.E, f.E, es, 128) || !make_tile_map(&p.o0, a.h, a.M, f.F, f.F, 2, 128))
        return map_failed("ffn_up");
    if (q8)
        return f.act == PMHA_ACT_SILU ? launch<kUpQ8, 128, PMHA_ACT_SILU>(p, "ffn_up_quantized", s)
                                      : launch<kUpQ8, 128, PMHA_ACT_GELU>(p, "ffn_up_quantized", s);
    return f.act == PMHA_ACT_SILU ? launch<kUp, 128, PMHA_ACT_SILU>(p, "ffn_up", s)
                                  : launch<kUp, 128, PMHA_ACT_GELU>(p, "ffn_up", s);
}

pmha_status ffn_tc_down(const FfnTc &f, const void *h, const void *wd, const void *residual, int64_t M, void *out,
                        cudaStream_t s)
{
    return down_like(f, h, nullptr, wd, nullptr, f.bd, residual, M, out, "ffn_down", s);
}

pmha_status ffn_tc_dx(const FfnTc &f, const void *dg, const void *du, const void *wg_t, const void *wu_t, int64_t M,
                      void *dx, cudaStream_t s)
{
    return down_like(f, dg, du, wg_t, wu_t, nullptr, nullptr, M, dx, "ffn_dx", s);
}

pmha_status ffn_tc_hidden(const FfnTc &f, const FfnHiddenArgs &a, cudaStream_t s)
{
    Params p = {};
    p.M = (int)a.M, p.E = (int)f.E, p.F = (int)f.F;
    p.tiles_n = (int)ceil_div(f.F, 64);
    const int64_t tiles = ceil_div(a.M, 256) * p.tiles_n;
    if (tiles > 0x3fffffff) return too_large("ffn_hidden", tiles);
    p.n_tiles = (int)tiles;
    p.kb = (int)ceil_div(f.E, 64);
    p.bias0 = (const __nv_bfloat16 *)f.bg;
    p.bias1 = (const __nv_bfloat16 *)f.bu;
    p.sums = a.sums;
    if (!make_tile_map(&p.a0, a.x, a.M, f.E, f.E, 2, 128) || !make_tile_map(&p.a1, a.dy, a.M, f.E, f.E, 2, 128) ||
        !make_tile_map(&p.b0, a.wg, f.F, f.E, f.E, 2, 64) || !make_tile_map(&p.b1, a.wu, f.F, f.E, f.E, 2, 64) ||
        !make_tile_map(&p.b2, a.wd_t, f.F, f.E, f.E, 2, 32) || !make_tile_map(&p.o0, a.h, a.M, f.F, f.F, 2, 128) ||
        !make_tile_map(&p.o1, a.dg, a.M, f.F, f.F, 2, 128) || !make_tile_map(&p.o2, a.du, a.M, f.F, f.F, 2, 128))
        return map_failed("ffn_hidden");
    return f.act == PMHA_ACT_SILU ? launch<kHidden, 64, PMHA_ACT_SILU>(p, "ffn_hidden", s)
                                  : launch<kHidden, 64, PMHA_ACT_GELU>(p, "ffn_hidden", s);
}

int64_t ffn_hidden_parts(int64_t M, int64_t F)
{
    // four warps' rows in each CTA of the pairs, of which there are at most as many as tiles
    return 8 * std::min<int64_t>(num_sms() / 2, ceil_div(M, 256) * ceil_div(F, 64));
}

// Rows of one accumulator of the weights' products, 16 an addition. The tensor core cuts its sums instead of rounding
// them: measured, an addition takes some 2^-22.3 of a running sum of one sign, 4,096 of them 4e-4 in all, a fifth of what rounding
// to bf16 may take. Without a limit the chains of narrow blocks had 52,000 (20,000,000 rows, hidden width 16: 5e-3).
constexpr int64_t kChain = 65536;

int ffn_dw_splits(int64_t E, int64_t F, int64_t rows)
{
    // As many pieces of the row range as fill the pairs, each of at least 4 blocks of 64 rows; and so many times as
    // many that a piece has kChain rows at most.
    const int64_t tiles = 3 * ceil_div(F, 256) * ceil_div(E, wide_tiles(E) ? 256 : 128);
    const int64_t pairs = num_sms() / 2;
    const int64_t fill = std::max<int64_t>(1, std::min(pairs / tiles, ceil_div(rows, 256)));
    return (int)(fill * ceil_div(std::max<int64_t>(rows, 1), fill * kChain));
}

pmha_status ffn_tc_dw(const FfnTc &f, const FfnDwArgs &a, cudaStream_t s)
{
    Params p = {};
    const bool wide = wide_tiles(f.E);
    p.M = (int)f.F;  // rows of the result
    p.E = (int)f.E, p.F = (int)f.F;
    p.tiles_m = (int)ceil_div(f.F, 256);
    p.tiles_n = (int)ceil_div(f.E, wide ? 256 : 128);
    p.splits = a.splits;
    p.first_what = a.gate_up ? 0 : 2;
    const int n_what = (a.gate_up ? 2 : 0) + (a.down ? 1 : 0);
    if (!n_what) return PMHA_OK;
    const int64_t tiles = (int64_t)n_what * p.tiles_m * p.tiles_n * p.splits;
    if (tiles > 0x3fffffff) return too_large("ffn_dw", tiles);
    p.n_tiles = (int)tiles;
    p.kb = (int)ceil_div(a.M, 64);
    p.part = a.part;
    p.sums = a.sums;
    p.accumulate = a.accumulate;
    if (!make_tile_map(&p.a0, a.dg, a.M, f.F, f.F, 2, 64) || !make_tile_map(&p.a1, a.du, a.M, f.F, f.F, 2, 64) ||
        !make_tile_map(&p.a2, a.h, a.M, f.F, f.F, 2, 64) || !make_tile_map(&p.b0, a.x, a.M, f.E, f.E, 2, 64) ||
        !make_tile_map(&p.b1, a.dy, a.M, f.E, f.E, 2, 64))
        return map_failed("ffn_dw");
    return wide ? launch<kDw, 256, 0>(p, "ffn_dw", s) : launch<kDw, 128, 0>(p, "ffn_dw", s);
}

}  // namespace pmha
