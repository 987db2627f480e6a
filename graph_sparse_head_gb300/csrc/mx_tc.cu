// Products of matrices in microscaled 4 bits (mx.cuh) on the tensor cores (sm_103a), one kernel shape for two:
//
//   linear  y = x W^T + bias + residual                          tile 256 tokens x 256 or 128 outputs, bf16
//   gated   h = act(x Wg^T + bg) * (x Wu^T + bu), in 4 bits      tile 256 tokens x 64 hidden, gate and up side by side
//
// Two CTAs form a pair (tc_pair.cuh). Each has 18 warps: warp 0 copies stages of
// 256 columns of codes (128 bytes a row, two values a byte) and the scale tiles that belong to them by TMA, a lane of warp
// 1 of the even CTA copies the scale tiles to tensor memory (tcgen05.cp, into both CTAs) and issues tcgen05.mma
// kind::mxf4, whose scaling by block is the hardware's; sixteen warps turn accumulators into outputs.
// Linear, 256 outputs: accumulators and the scales of the stages leave no room for a second set in tensor memory; an
// epilogue thread takes all of its accumulators into registers (64) and hands the set back at once, so that the next
// products run under its arithmetic (8,192 x 4,096 -> 4,096 in 45.5 us, 6.0 PFLOP/s). 128 outputs: three sets, and two teams
// of eight warps that take the tiles in turn (320,000 x 128 -> 384 in 44 us, 88 % of the copy rate, with a residual 81,
// 94 %). Gated: three sets of 64 gates and 64 ups and two teams, one team's waits under the other's special functions, 16
// columns' accumulators on their way while 16 are used (320,000 x 128 x 512 in 98 us; with one set of 128 + 128, one team
// and all accumulators in registers at once 112).
// Epilogue warps go their own ways: each has its 32 rows' share of the columns, its own piece of shared memory, its own
// copies of the residual and of the result, and no barrier with the others. (With a barrier for all sixteen around each
// step the same took 152 us.)
//
// Ragged sizes need no code of their own: TMA fills rows and columns past a
// tensor's end with zeros (codes and scale tiles) and does not store them. Only
// outputs whose rows are no multiples of 16 bytes go through plain loads and stores.
//
// Every mbarrier wait is bounded (tc_util.cuh); on expiry the pair gives up,
// waits for its copies and products, frees its tensor memory and returns, and
// pmha_device_status reports PMHA_ERR_TIMEOUT.
#include <algorithm>

#include "ffn_math.cuh"
#include "mx.cuh"
#include "pair.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {
using namespace tcu;

constexpr int kThreads = 64 + 512;
constexpr int kBox = 128 * 128;       // bytes of a tile of 128 rows of 128 bytes
constexpr int kSfA = 2 * 512;         // scale tiles of a stage: 128 rows x 256 columns
// Not kept for tiles of 256 outputs: four stages, with output pieces of 64 columns (8,192 x 4,096 -> 4,096 51.5 us for 45.5);
// six, with outputs straight from registers to make room (50.0, with a residual 85 for 51).
enum Kind { kTiles, kNarrow, kGated };
template <int KIND>
struct Cfg {
    static constexpr bool kGate = KIND == kGated;
    static constexpr int kCols = kGate ? 64 : KIND == kNarrow ? 128 : 256;  // output columns of a tile: N of a product
    static constexpr int kOps = kGate ? 2 : 1;          // products side by side
    static constexpr int kRowsB = kCols / 2;            // weight rows that a CTA brings to a product
    static constexpr int kB = kOps * kRowsB * 128;
    static constexpr int kSfTiles = KIND == kNarrow ? 1 : 2;  // of 128 rows of weights (one each of gate and up)
    static constexpr int kStage = kBox + kB + kSfA + 1024 * kSfTiles;
    static_assert(kStage % 1024 == 0, "swizzled tiles lie on 1024 bytes");
    static constexpr int kAccs = KIND == kTiles ? 1 : 3, kAccCols = kOps * kCols;
    static constexpr int kTeams = KIND == kTiles ? 1 : 2;        // of epilogue warps, which take tiles in turn
    static constexpr int kStages = 5;
    static constexpr int kScaleCol = kAccs * kAccCols;  // then 24 scale columns a stage
    static_assert(kScaleCol + 24 * kStages <= 512, "tensor memory");
    // An epilogue warp's 32 x 64 outputs leave in one piece of shared memory or in two
    static constexpr int kPieceCols = KIND == kTiles ? 32 : 64, kPiece = 32 * kPieceCols * 2;
    static constexpr int kTile = kGate ? 0 : 16 * kPiece;
    static constexpr int kVec = 16 * 64 * 4;  // a warp's biases: of 64 outputs, or 32 of gate and of up
    static constexpr int kBars = 512;
    static constexpr int kSmem = 1024 + kStages * kStage + kTile + kVec + kBars;
    static_assert(kSmem <= 232448, "shared memory of one CTA");
};
constexpr int kTmemCols = 512;

struct Params {
    CUtensorMap a, b0, b1, sa, sb0, sb1, out, res;
    int M, N;               // tokens, outputs (gated: hidden width)
    int n_tiles, tiles_n, kb, k64;  // K blocks of 256 columns, products of 64
    const __nv_bfloat16 *bias0, *bias1;
    const __nv_bfloat16 *res_p;  // plain: row-wise outputs without TMA
    __nv_bfloat16 *out_p;
    uint8_t *h_codes, *h_scale;
    long long h_pitch;
    int h_blocks, h_tiles;  // blocks of a row of h, scale tiles of a row block
    int has_res;
    int *err;
};

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// A scale tile of 32 rows of 16 bytes, 8-row groups 128 bytes apart, without swizzle
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1 << 46);
}
// to 4 columns of tensor memory, the same 32 lanes for each of the four warps, in both CTAs from their own shared memory
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// kind::mxf4: A and B E2M1 (1 at bits 7-9 and 10-12), 256 x N (N >> 3 at bits 17-22, M >> 7 at bits 27-28), E8M0
// scales (bit 23); sf: which of a column's byte pairs holds the scales, 0 or 2 (bits 4-5 for B, 29-30 for A).
__host__ __device__ constexpr uint32_t idesc_mx(uint32_t n, uint32_t sf)
{
    return (sf << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | (2u << 27) | (sf << 29);
}
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// The largest magnitude, NaN before all
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}
// VARIANT: gated, the activation; else whether outputs go through plain loads and stores (which cost registers)
template <int KIND, int VARIANT>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) k_mx(const __grid_constant__ Params p)
{
    using C = Cfg<KIND>;
    constexpr bool GATED = KIND == kGated, kPlain = !GATED && VARIANT;
    constexpr int kStages = C::kStages, kStage = C::kStage, kCols = C::kCols, kAccs = C::kAccs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *tile_s = smem + kStages * kStage;
    float *vec_s = (float *)(tile_s + C::kTile);
    uint64_t *full = (uint64_t *)((uint8_t *)vec_s + C::kVec);     // [kStages], counted in the even CTA
    uint64_t *empty = full + kStages;                           // [kStages], in each CTA
    uint64_t *acc_full = empty + kStages;                       // [kAccs], in each CTA
    uint64_t *acc_empty = acc_full + kAccs;                     // [kAccs], counted in the even CTA
    uint64_t *mma_done = acc_empty + kAccs;
    uint64_t *res_full = mma_done + 1;                          // [16], of the epilogue warps
    uint32_t *tmem_holder = (uint32_t *)(res_full + 16);
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
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), 32 / C::kTeams);  // a team's warps of both CTAs
        }
        mbar_init(smem_u32(mma_done), 1);
        for (int w = 0; w < 16; ++w) mbar_init(smem_u32(&res_full[w]), 1);
        *abort_flag = 0;
        *armed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), kTmemCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    grid_dependency_wait();
    const uint32_t tmem = *tmem_holder;

    if (warp == 0) {
        // ---------------- TMA producer of this CTA
        const bool one = elect_one();
        uint32_t made = 0;
        for (int tile = pair; tile < p.n_tiles && !*abort_flag; tile += n_pairs) {
            const int m = tile / p.tiles_n, n = tile % p.tiles_n;
            const int rows = m * 2 + (int)rank;  // block of 128 tokens
            for (int kb = 0; kb < p.kb; ++kb, ++made) {
                const int stage = (int)(made % kStages);
                if (!wait_bar(smem_u32(&empty[stage]), ((made / kStages) & 1u) ^ 1u, abort_flag, p.err)) break;
                if (!one) continue;
                const uint32_t fb = map_rank(smem_u32(&full[stage]), 0);
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * kStage);
                *armed = made + 1;
                const uint32_t sa = smem_u32(smem + stage * kStage), sb = sa + kBox, ssa = sb + C::kB, ssb = ssa + kSfA;
                tma_load_2d_pair(sa, &p.a, kb * 128, rows * 128, fb);
                const int row = n * kCols + (int)rank * C::kRowsB;
                tma_load_2d_pair(sb, &p.b0, kb * 128, row, fb);
                if constexpr (GATED) tma_load_2d_pair(sb + C::kRowsB * 128, &p.b1, kb * 128, row, fb);
                tma_load_3d_pair(ssa, &p.sa, 0, kb * 2, rows, fb);
                // the scales of all columns, in both CTAs: two tiles of the weights', or the tiles of gate and of up in
                // which the 64 columns lie
                tma_load_3d_pair(ssb, &p.sb0, 0, kb * 2, GATED ? n / 2 : n * C::kSfTiles, fb);
                if constexpr (C::kSfTiles == 2)
                    tma_load_3d_pair(ssb + 1024, GATED ? &p.sb1 : &p.sb0, 0, kb * 2, GATED ? n / 2 : n * 2 + 1, fb);
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- issuer of the pair: one lane, which waits and issues by itself
            if (elect_one()) {
                uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 1;
                const uint32_t base = smem_u32(smem);
                const uint64_t a_first = smem_desc(base), b_first = smem_desc(base + kBox);
                const uint64_t sa_first = scale_desc(base + kBox + C::kB), sb_first = scale_desc(base + kBox + C::kB + kSfA);
                bool ok = true;
                for (int tile = pair; tile < p.n_tiles && ok; tile += n_pairs) {
                    if (!wait_bar(smem_u32(&acc_empty[acc]), acc_phase, abort_flag, p.err)) break;
                    tc_fence_after();
                    const uint32_t d = tmem + acc * C::kAccCols;
                    // of a scale tile's four columns of 32 rows, the first of this tile's
                    const uint32_t half = GATED ? 2u * ((uint32_t)(tile % p.tiles_n) & 1u) : 0u;
                    for (int kb = 0; kb < p.kb; ++kb) {
                        ok = wait_bar(smem_u32(&full[stage]), phase, abort_flag, p.err);
                        if (!ok) break;
                        tc_fence_after();
                        const int steps = p.k64 - 4 * kb;  // products of 64 columns left, up to the width's end
                        // scale columns of this stage: 2 x 4 of the tokens, then 2 x 8 of the weights (128 columns of K,
                        // then 256 rows, or 128 of gate and of up)
                        const uint32_t ca = tmem + C::kScaleCol + 24 * stage, cb = ca + 8;
                        const uint64_t at = (uint64_t)(stage * (kStage / 16));  // of the address field, 16 bytes each
                        const uint64_t da = a_first + at, db = b_first + at, dsa = sa_first + at, dsb = sb_first + at;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // 64 values = 32 bytes along K = 2 in the address field
                            if (k >= steps) break;
                            if (k % 2 == 0) {
                                const int h = k / 2;
                                copy_scales(ca + 4 * h, dsa + 32 * h);
                                copy_scales(cb + 8 * h, dsb + 32 * h);
                                if constexpr (C::kSfTiles == 2) copy_scales(cb + 8 * h + 4, dsb + 64 + 32 * h);
                            }
#pragma unroll
                            for (int o = 0; o < C::kOps; ++o)
                                mma_mx(d + o * kCols, da + (uint64_t)(2 * k), db + (uint64_t)(o * C::kRowsB * 8 + 2 * k),
                                       k & 1 ? idesc_mx(kCols, 2) : idesc_mx(kCols, 0), ca + 4 * (k >> 1),
                                       cb + 8 * (k >> 1) + 4 * o + half, kb > 0 || k > 0 ? 1u : 0u);
                        }
                        mma_commit_pair(smem_u32(&empty[stage]));
                        if (++stage == kStages) stage = 0, phase ^= 1u;
                    }
                    if (ok) mma_commit_pair(smem_u32(&acc_full[acc]));
                    if (++acc == kAccs) acc = 0, acc_phase ^= 1u;
                }
                mma_commit_pair(smem_u32(mma_done));
                int dummy = 0;
                mbar_wait(smem_u32(mma_done), 0, (volatile int *)&dummy, p.err);
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue: a warp 32 rows and 64 accumulator columns of a tile, of which teams take turns
        const int w = warp - 2, quarter = warp & 3, team = C::kTeams == 2 ? w >> 3 : 0;
        const int part = (w >> 2) & (C::kTeams == 2 ? 1 : 3);
        const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(GATED ? part * 32 : part * 64);
        const uint32_t empty_bar = map_rank(smem_u32(acc_empty), 0);
        const int first = pair + team * n_pairs, next = C::kTeams * n_pairs;
        float *bias = vec_s + w * 64;
        auto in_piece = [](int r, int u) {  // 16 bytes u of row r, as TMA places them (128- or 64-byte rows)
            return C::kPieceCols == 64 ? swizzled(r, u) : (uint32_t)(r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
        };
        uint8_t *piece = tile_s + w * C::kPiece;
        constexpr float kg = GATED ? Act<VARIANT>::kGate : 1.f, ku = GATED ? Act<VARIANT>::kUp : 1.f;
        auto rows_of = [&](int tile) { return tile / p.tiles_n * 256 + (int)rank * 128 + quarter * 32; };
        auto column_of = [&](int tile) { return tile % p.tiles_n * kCols + part * (GATED ? 32 : 64); };
        auto fetch_residual = [&](int tile, int half) {
            if (GATED || kPlain || !p.has_res || lane) return;
            const int row = rows_of(tile), c = column_of(tile) + half * C::kPieceCols;
            if (row < p.M && c < p.N) {
                mbar_arrive_expect_tx(smem_u32(&res_full[w]), C::kPiece);
                tma_load_2d(smem_u32(piece), &p.res, c, row, smem_u32(&res_full[w]));
            } else {
                mbar_arrive(smem_u32(&res_full[w]));
            }
        };
        // biases of the next tile: this lane's columns
        float b0 = 0.f, b1 = 0.f;
        auto fetch_bias = [&](int tile) {
            const int c = column_of(tile) + lane, c2 = GATED ? c : c + 32;
            const __nv_bfloat16 *second = GATED ? p.bias1 : p.bias0;
            b0 = p.bias0 && c < p.N ? kg * __bfloat162float(p.bias0[c]) : 0.f;
            b1 = second && c2 < p.N ? ku * __bfloat162float(second[c2]) : 0.f;
        };
        uint32_t i = (uint32_t)team, fetched = 0;  // tiles of all teams, residual copies of this warp
        if (first < p.n_tiles) {
            fetch_residual(first, 0);
            fetched = 1;
            fetch_bias(first);
        }
        for (int tile = first; tile < p.n_tiles; tile += next, i += C::kTeams) {
            const int acc = (int)(i % kAccs);
            const int row0 = rows_of(tile), c0 = column_of(tile);
            __syncwarp();
            bias[lane] = b0;
            bias[32 + lane] = b1;
            __syncwarp();
            if (tile + next < p.n_tiles) fetch_bias(tile + next);
            // after an expired wait the waits return at once and the loop runs out
            wait_bar(smem_u32(&acc_full[acc]), (i / kAccs) & 1u, abort_flag, p.err);
            tc_fence_after();
            __syncwarp();
            uint32_t v[2][KIND == kNarrow ? 16 : 32];  // 64 outputs (narrow: 16 and the next 16; gated: 32)
            auto hand_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(empty_bar + 8u * (uint32_t)acc);
            };
            if constexpr (KIND == kNarrow) tmem_ld16(t0 + (uint32_t)(acc * C::kAccCols), v[0]);
            if constexpr (KIND == kTiles) {
                tmem_ld32_nowait(t0 + (uint32_t)(acc * C::kAccCols), v[0]);
                tmem_ld32_nowait(t0 + (uint32_t)(acc * C::kAccCols + 32), v[1]);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                pin(v[0]);
                pin(v[1]);
                hand_back();
            }
            // outputs 8 u and on: eight accumulators, biases, and the residual's values
            auto sums = [&](int u, const uint32_t *acc8, const uint32_t (&rw)[4]) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 b = *reinterpret_cast<const float2 *>(bias + 8 * u + 2 * e);
                    o[e] = pack_bf16(__uint_as_float(acc8[2 * e]) + b.x + __uint_as_float(rw[e] << 16),
                                     __uint_as_float(acc8[2 * e + 1]) + b.y + __uint_as_float(rw[e] & 0xffff0000u));
                }
                return make_uint4(o[0], o[1], o[2], o[3]);
            };
            if constexpr (GATED) {
                // gate and up of 32 hidden columns, CH at a time: the next ones come from tensor memory meanwhile
                constexpr int CH = 16;
                const uint32_t tg = t0 + (uint32_t)(acc * C::kAccCols), tu = tg + (uint32_t)kCols;
                uint32_t g[2][CH], u[2][CH];
                float most = 0.f;
                tmem_ld16(tg, g[0]);
                tmem_ld16(tu, u[0]);
#pragma unroll
                for (int q = 0; q < 32 / CH; ++q) {
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    pin(g[q & 1]);
                    pin(u[q & 1]);
                    if (q + 1 < 32 / CH) {
                        tmem_ld16(tg + CH * (q + 1), g[(q + 1) & 1]);
                        tmem_ld16(tu + CH * (q + 1), u[(q + 1) & 1]);
                    } else {
                        hand_back();
                    }
#pragma unroll
                    for (int c = 0; c < CH; c += 4) {
                        const float4 gb4 = *reinterpret_cast<const float4 *>(bias + q * CH + c);
                        const float4 ub4 = *reinterpret_cast<const float4 *>(bias + 32 + q * CH + c);
                        const Pair gb[2] = {Pair(gb4.x, gb4.y), Pair(gb4.z, gb4.w)};
                        const Pair ub[2] = {Pair(ub4.x, ub4.y), Pair(ub4.z, ub4.w)};
                        auto two = [](const uint32_t *r) { return Pair(__uint_as_float(r[0]), __uint_as_float(r[1])); };
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const Pair gate = fma2(two(&g[q & 1][c + e]), Pair(kg, kg), gb[e / 2]);
                            const Pair up = fma2(two(&u[q & 1][c + e]), Pair(ku, ku), ub[e / 2]);
                            float h0, h1;
                            Act<VARIANT>::hidden2(gate, up).get(h0, h1);
                            most = max_nan(most, h0, h1);
                            v[0][q * CH + c + e] = __float_as_uint(h0);
                            v[0][q * CH + c + e + 1] = __float_as_uint(h1);
                        }
                    }
                }
                const uint32_t byte = mx_scale_byte(abs_bits(most));
                const float inv = mx_inverse(byte);
                uint32_t code[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        mul2(Pair(__uint_as_float(v[0][8 * c + e]), __uint_as_float(v[0][8 * c + e + 1])), Pair(inv, inv))
                            .get(f[e], f[e + 1]);
                    code[c] = mx_word(f);
                }
                // Straight to memory: 16 bytes of a row each, which meet those of the neighbouring blocks in L2. Blocks
                // past the last have a place in the scale tile, where they put the scale of zeros.
                const int row = row0 + lane, block = c0 / 32;
                if (row < p.M) {
                    if (block < p.h_blocks)
                        *reinterpret_cast<uint4 *>(p.h_codes + row * p.h_pitch + block * 16) =
                            make_uint4(code[0], code[1], code[2], code[3]);
                    p.h_scale[((size_t)(row0 >> 7) * p.h_tiles + (block >> 2)) * 512 + 16 * lane + 4 * quarter + (block & 3)] =
                        (uint8_t)byte;
                }
            } else {
                constexpr int kHalves = 64 / C::kPieceCols;
                bool ok = true;
                // plain rows: a lane a column, of eight rows at a time
                auto by_rows = [&](int first_col, auto load, auto store) {
                    for (int h = 0; h < C::kPieceCols / 32; ++h) {
                        const int c = lane + 32 * h, col = first_col + c;
                        if (col >= p.N) return;
                        for (int q0 = 0; q0 < 32; q0 += 8) {
                            __nv_bfloat16 x[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (row0 + q0 + q < p.M) x[q] = load(q0 + q, c, (size_t)(row0 + q0 + q) * p.N + col);
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (row0 + q0 + q < p.M) store(q0 + q, c, (size_t)(row0 + q0 + q) * p.N + col, x[q]);
                        }
                    }
                };
                auto value = [&](int q, int c) { return (__nv_bfloat16 *)(piece + in_piece(q, c >> 3) + (c & 7) * 2); };
#pragma unroll
                for (int half = 0; half < kHalves; ++half) {
                    const int col = c0 + half * C::kPieceCols;
                    if constexpr (kPlain) {
                        __syncwarp();
                        if (p.has_res) {
                            by_rows(col, [&](int q, int c, size_t at) { return p.res_p[at]; },
                                    [&](int q, int c, size_t at, __nv_bfloat16 x) { *value(q, c) = x; });
                            __syncwarp();
                        }
                    } else if (p.has_res) {
                        ok = ok && wait_bar(smem_u32(&res_full[w]), (i / C::kTeams * kHalves + half) & 1u, abort_flag, p.err);
                    } else {
                        if (lane == 0) store_wait_read();  // the last store has read the piece
                        __syncwarp();
                    }
#pragma unroll
                    for (int x = 0; x < C::kPieceCols / 8; ++x) {
                        const int u = half * (C::kPieceCols / 8) + x;
                        uint4 *at = reinterpret_cast<uint4 *>(piece + in_piece(lane, x));
                        const uint32_t *acc8;
                        if constexpr (KIND == kNarrow) {
                            const int q = u / 2;
                            if (u % 2 == 0) {
                                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                                pin(v[q & 1]);
                                if (q < 3)
                                    tmem_ld16(t0 + (uint32_t)(acc * C::kAccCols + 16 * (q + 1)), v[(q + 1) & 1]);
                                else
                                    hand_back();
                            }
                            acc8 = &v[q & 1][8 * (u % 2)];
                        } else {
                            acc8 = &v[u / 4][8 * (u % 4)];
                        }
                        uint32_t rw[4] = {0, 0, 0, 0};
                        if (p.has_res) {
                            const uint4 q = *at;
                            rw[0] = q.x, rw[1] = q.y, rw[2] = q.z, rw[3] = q.w;
                        }
                        *at = sums(u, acc8, rw);
                    }
                    if constexpr (kPlain) {
                        __syncwarp();
                        by_rows(col, [&](int q, int c, size_t at) { return *value(q, c); },
                                [&](int q, int c, size_t at, __nv_bfloat16 x) { p.out_p[at] = x; });
                    } else {
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            if (row0 < p.M && col < p.N) tma_store_tile(&p.out, smem_u32(piece), col, row0);
                            store_commit();
                            const bool last = half + 1 == kHalves;
                            if (p.has_res && ok && (!last || tile + next < p.n_tiles)) {
                                store_wait_read();
                                fetch_residual(last ? tile + next : tile, last ? 0 : half + 1);
                                ++fetched;
                            }
                        }
                    }
                }
            }
        }
        if (!GATED && lane == 0) {
            store_wait_all();  // shared memory outlives its stores, and after an expired wait the residual's copies
            int dummy = 0;
            if (*abort_flag && p.has_res && !kPlain && fetched)
                mbar_wait(smem_u32(&res_full[w]), (fetched - 1) & 1u, (volatile int *)&dummy, p.err);
        }
        __syncwarp();
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
    if (warp == 1) tmem_free_pair(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host side
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Codes as rows of bytes, boxes of 128 bytes x box_rows; scale tiles as (row block, tile, 128 words), boxes of two tiles
bool maps_of(CUtensorMap *codes, CUtensorMap *scale, const Mx &m, int64_t rows, int64_t width, uint32_t box_rows = 128)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn || !make_tile_map(codes, m.codes, rows, mx_pitch(width), mx_pitch(width), 1, box_rows)) return false;
    const cuuint64_t tiles = (cuuint64_t)ceil_div(mx_blocks(width), 4);
    cuuint64_t dims[3] = {128, tiles, (cuuint64_t)ceil_div(rows, 128)};
    cuuint64_t strides[2] = {512, 512 * tiles};
    cuuint32_t box[3] = {128, 2, 1}, estr[3] = {1, 1, 1};
    return fn(scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(m.scale), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (rows, cols) bf16 in boxes of 32 rows x piece_cols, as the epilogue warps' pieces
bool map_of_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int piece_cols)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(cols * 2)};
    cuuint32_t box[2] = {(cuuint32_t)piece_cols, 32}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, piece_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, int VARIANT>
pmha_status launch(Params &p, const char *stage, cudaStream_t s)
{
    constexpr int kSmem = Cfg<KIND>::kSmem;
    p.err = device_error_word();
    if (!p.err) return PMHA_ERR_CUDA;
    int pairs = 0;
    auto kern = k_mx<KIND, VARIANT>;
    static std::atomic<int> known[kKnownDevices];
    const pmha_status st = pairs_at_once(kern, kThreads, kSmem, known, &pairs);
    if (st != PMHA_OK) return st;
    StageTimer timer(stage, s);
    return launch_overlapping(kern, dim3(2u * (unsigned)std::min(pairs, p.n_tiles)), kThreads, kSmem, s, p);
}

pmha_status map_failed(const char *what)
{
    set_error("%s: cuTensorMapEncodeTiled failed", what);
    return PMHA_ERR_CUDA;
}

pmha_status tiles_of(Params &p, int64_t M, int64_t N, int64_t K, int cols, const char *stage)
{
    p.M = (int)M, p.N = (int)N;
    p.tiles_n = (int)ceil_div(N, cols);
    p.kb = (int)ceil_div(K, 256);
    p.k64 = (int)ceil_div(K, 64);
    const int64_t tiles = ceil_div(M, 256) * p.tiles_n;
    if (tiles > 0x3fffffff) {
        set_error("%s: %lld tiles exceed the 32-bit tile index", stage, (long long)tiles);
        return PMHA_ERR_INVALID_ARG;
    }
    p.n_tiles = (int)tiles;
    return PMHA_OK;
}

// Tiles of 128 outputs instead of 256? Short products are bound by their outputs, which two teams of epilogue warps on
// narrow tiles take without waiting for each other: 128 -> 384 at 320,000 tokens 45 us for 58, with a residual 81 for 105;
// 512 -> 128 28 for 33, with a residual 39 for 47; 32,000 x 1,024 -> 1,024 with a residual 28.6 for 31.8. Long ones are bound
// by the products, of which a narrow tile's take 0.6 of a wide one's time (8,192 x 4,096 -> 4,096 62 us for 51): there, the
// fewer rounds of tiles by that weight (300 x 4,096 -> 1,024 7.4 for 9.6; 8,192 x 4,096 -> 512 12.2 for 10.7).
bool narrow_tiles(int64_t M, int64_t N, int64_t K)
{
    const int64_t pairs = std::max(1, num_sms() / 2), rows = ceil_div(M, 256);
    auto rounds = [&](int64_t cols) { return ceil_div(rows * ceil_div(N, cols), pairs); };
    return K <= 1024 || 5 * rounds(128) < 8 * rounds(256);
}

}  // namespace

pmha_status mx_tc_linear(const MxLinear &a, const char *stage, cudaStream_t s)
{
    Params p = {};
    const bool narrow = narrow_tiles(a.M, a.N, a.K), plain = a.N % 8 != 0;
    const pmha_status st = tiles_of(p, a.M, a.N, a.K, narrow ? 128 : 256, stage);
    if (st != PMHA_OK) return st;
    const int piece = narrow ? Cfg<kNarrow>::kPieceCols : Cfg<kTiles>::kPieceCols;
    p.bias0 = (const __nv_bfloat16 *)a.bias;
    p.has_res = a.residual != nullptr;
    p.res_p = (const __nv_bfloat16 *)a.residual;
    p.out_p = (__nv_bfloat16 *)a.out;
    if (!maps_of(&p.a, &p.sa, a.x, a.M, a.K) || !maps_of(&p.b0, &p.sb0, a.w, a.N, a.K, narrow ? 64 : 128) ||
        (!plain && (!map_of_rows(&p.out, a.out, a.M, a.N, piece) ||
                    (a.residual && !map_of_rows(&p.res, a.residual, a.M, a.N, piece)))))
        return map_failed(stage);
    if (narrow) return plain ? launch<kNarrow, 1>(p, stage, s) : launch<kNarrow, 0>(p, stage, s);
    return plain ? launch<kTiles, 1>(p, stage, s) : launch<kTiles, 0>(p, stage, s);
}

pmha_status mx_tc_gated(const MxGated &a, cudaStream_t s)
{
    Params p = {};
    const char *stage = "ffn_up_mx";
    const pmha_status st = tiles_of(p, a.M, a.F, a.K, 64, stage);
    if (st != PMHA_OK) return st;
    p.bias0 = (const __nv_bfloat16 *)a.bg;
    p.bias1 = (const __nv_bfloat16 *)a.bu;
    p.h_codes = a.h_codes;
    p.h_scale = a.h_scale;
    p.h_pitch = mx_pitch(a.F);
    p.h_blocks = (int)mx_blocks(a.F);
    p.h_tiles = (int)ceil_div(mx_blocks(a.F), 4);
    p.tiles_n = 2 * p.h_tiles;  // whole scale tiles of h, to their zeros past the last block
    p.n_tiles = (int)(ceil_div(a.M, 256) * p.tiles_n);
    constexpr uint32_t kBoxRows = Cfg<kGated>::kRowsB;
    if (!maps_of(&p.a, &p.sa, a.x, a.M, a.K) || !maps_of(&p.b0, &p.sb0, a.wg, a.F, a.K, kBoxRows) ||
        !maps_of(&p.b1, &p.sb1, a.wu, a.F, a.K, kBoxRows))
        return map_failed(stage);
    return a.act == PMHA_ACT_SILU ? launch<kGated, PMHA_ACT_SILU>(p, stage, s) : launch<kGated, PMHA_ACT_GELU>(p, stage, s);
}

}  // namespace pmha
