// The gated block with its hidden rows kept on the chip (sm_103a), for
// embed_dim up to 256. A pair of CTAs (tc_pair.cuh) owns 256 rows, 128 a CTA:
// its tokens stay in shared memory while the hidden width passes in chunks of
// 64 columns, whose weights stream through two rings of TMA stages.
//
//   forward, chunk c:   S = x [Wg_c | Wu_c]^T           tensor memory, two buffers
//                       h = act(S_g + bg) * (S_u + bu)   -> shared memory, bf16
//                       Y += h Wd_c^T                    tensor memory
//   after the last:     y = Y + bd + residual
//
//   backward, chunk c:  S as above, D = dy Wd_c
//                       h, dg, du -> shared memory, and by TMA to memory (the weight gradients read them)
//                       X += dg Wg_c + du Wu_c           (embed_dim up to 128)
//   after the last:     dx = X
//
// The hidden values never go to memory in the forward pass, and the tokens are
// read once. The warps are specialised: warp 0 copies, warp 1 of the even CTA
// issues the products, sixteen warps turn S into hidden values, and four drain
// the row block's result while the next block's chunks go on. The issuer runs S
// two chunks ahead, across row blocks: S(0) S(1) | S(2) Y(0) | S(3) Y(1) ... A
// chunk's time is that of a loop, S -> epilogue -> Y and the next S of the
// buffer, over the buffers; what was measured on the way (cycles a chunk of 64
// columns, embed_dim 128, where the products take 770):
// waits with cluster-scope acquires and one wait and commit for each stage
// 3,100; one commit a step, waits for what is long loaded taken first, the
// issuing warp converged (uniform addresses) and the epilogue rolled, so that
// the warps share the instruction cache, 2,000; sixteen epilogue warps instead
// of eight 1,440 to 1,640; the result through TMA instead of 32-byte accesses (a
// warp's 32 rows cost the memory pipe 32 cycles an instruction) 1,350; the
// accumulators read as fragments (fewer bias loads), a second accumulator of the
// result instead of a third of S (with one the next row block's first Y waits
// for the drain) and a third Y stage 1,200. Slower were: reads of the next eight
// columns under this eight's arithmetic, the wait for the staged tile after the
// arithmetic (both some 5 %), and Y before S (10 %).
// 320,000 rows of embed_dim 128, 512 hidden: forward 109 us (126 GFLOP: 1.15
// PFLOP/s, 61 % of cuBLAS bf16), backward 250 of the 440 us of its pass.
//
// Every wait is bounded; after an expired one the waits return at once, the
// loops run out, and pmha_device_status reports PMHA_ERR_TIMEOUT.
#include <algorithm>

#include "ffn_internal.h"
#include "ffn_math.cuh"
#include "tc_pair.cuh"

namespace pmha {
namespace {
using namespace tcu;

constexpr int kThreads = 704;       // 2 + 16 + 4 warps
constexpr int kBox = 128 * 128;     // 128 rows of 128 bytes
constexpr int kSmemMost = 232448;

// EB: blocks of 64 output columns; KB: blocks of 128 bytes of a token.
template <int EB, bool BWD, bool Q8>
struct Cfg {
    static constexpr int KB = Q8 ? (EB + 1) / 2 : EB;
    static constexpr bool kOut = !BWD || EB <= 2;               // the kernel forms y, or dx
    static constexpr int SB = 2;                                // S buffers in tensor memory
    static constexpr int kX = (BWD ? 2 : 1) * KB * kBox;        // x (and dy) of a row block
    static constexpr int kSBlock = BWD ? 12288 : 8192;          // 64 rows of Wg or Wu (and 32 of Wd^T), one K block
    static constexpr int SG = BWD ? 1 : !Q8 && EB == 4 ? 2 : KB;        // K blocks of a stage of the S ring
    static constexpr int kSSlot = SG * kSBlock;
    static constexpr int kYSlot = kOut ? EB * (BWD ? 8192 : 4096) : 0;  // half of the output columns of a chunk
    static constexpr int kNY = !kOut ? 0 : !BWD && EB <= 2 ? 3 : 2;
    static constexpr int kMaxHidden = 2048;                     // bias (and scale) columns held
    static constexpr int kStaged = BWD ? 3 * kBox : kBox;       // dg, du and h, or h
    static constexpr int kStages = BWD ? 1 : SB;
    static constexpr int kOT = BWD ? 1 : 2;                     // tiles of 64 result columns
    static constexpr int kOutTiles = kOut ? kOT * kBox : 0;
    static constexpr int kSCols = BWD ? 192 : 128;
    static constexpr int kVec = kMaxHidden * (BWD ? 4 : 8) + 1024;      // gate and up biases; output bias
    static constexpr int kScales = Q8 ? kMaxHidden * 8 : 0;
    static constexpr int kBars = 512;
    static constexpr int kFixed = 1024 + kNY * kYSlot + kStages * kStaged + kOutTiles + kVec + kScales + kBars;
    static constexpr int kXB = kFixed + 2 * kX + 3 * kSSlot <= kSmemMost ? 2 : 1;  // token buffers
    static constexpr int kNSFit = (kSmemMost - kFixed - kXB * kX) / kSSlot;
    static constexpr int kNS = kNSFit > 4 ? 4 : kNSFit;
    static constexpr int kOB = SB * kSCols + 2 * EB * 64 <= 512 ? 2 : 1;  // output accumulators
    static constexpr int kSmem = kFixed + kXB * kX + kNS * kSSlot;
    static_assert(kNS >= 3, "a ring of at least three stages");
    static_assert(KB <= kNS * SG || !kOut, "the down product's weights come after the tokens");
    static_assert(SG == KB || kXB == 1, "the reuse of a second token buffer is known from the S ring");
    static_assert(!kOut || SB * kSCols + kOB * EB * 64 <= 512, "tensor memory");
};

struct Params {
    CUtensorMap x, dy, wg, wu, wd;  // wd: Wd (E, F), or Wd^T (F, E) in the backward pass
    CUtensorMap wgt, wut;           // (E, F): Wg^T, Wu^T
    CUtensorMap h, dg, du;          // (M, F)
    CUtensorMap out, res;           // (M, E)
    int M, E, F;
    int items, parts;               // row blocks x parts of the hidden width
    int chunks, per_part;           // chunks of 64 hidden columns, and of one part
    const __nv_bfloat16 *bg, *bu, *bd;
    const float *xs, *gs, *us;
    int has_res, has_out;
    float *sums;                    // (CTA, quarter of its rows, 2, F) column sums of dg and du, or null
    int *err;
};

__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// Waits for this thread's tensor-memory reads; the values' uses stay behind it.
template <typename... R>
__device__ __forceinline__ void tmem_wait(R &...regs)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    (pin(regs), ...);
}

// named barrier 4 over the chunk epilogue's 512 threads
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 4, 512;" ::: "memory"); }

template <int EB, bool BWD, bool Q8, int ACT>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) k_block(const __grid_constant__ Params p)
{
    using C = Cfg<EB, BWD, Q8>;
    constexpr int KB = C::KB, NS = C::kNS, NY = C::kNY > 0 ? C::kNY : 1, XB = C::kXB, OB = C::kOB, SB = C::SB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *x_s = smem;                              // [XB][x blocks, dy blocks]
    uint8_t *s_ring = x_s + XB * C::kX;               // [NS]
    uint8_t *y_ring = s_ring + NS * C::kSSlot;        // [kNY]
    uint8_t *staged = y_ring + C::kNY * C::kYSlot;    // [kStages]
    uint8_t *out_s = staged + C::kStages * C::kStaged;  // [kOT] tiles of 64 result columns
    float *bd_s = (float *)(out_s + C::kOutTiles);      // [256]
    float *bg_s = bd_s + 256, *bu_s = bg_s + C::kMaxHidden;  // forward: float32, times the activation's constants
    uint32_t *bias_s = (uint32_t *)bg_s;                  // backward: (bg, bu) as bf16
    float *gs_s = (float *)((uint8_t *)bd_s + C::kVec), *us_s = gs_s + C::kMaxHidden;
    uint64_t *bar = (uint64_t *)((uint8_t *)gs_s + C::kScales);
    uint64_t *x_full = bar, *s_full = x_full + 2, *s_empty = s_full + 4, *y_full = s_empty + 4, *step = y_full + 4,
             *h_full = step + 4, *out_full = h_full + 3, *out_empty = out_full + 2, *res_full = out_empty + 2,
             *y_done = res_full + 2, *mma_done = y_done + 4;
    uint32_t *tmem_holder = (uint32_t *)(mma_done + 1);
    volatile int *abort_flag = (volatile int *)(tmem_holder + 1);
    volatile uint32_t *armed = (volatile uint32_t *)(tmem_holder + 2);  // copies counted: x, S and Y slots, residual

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&x_full[i]), 1);
            mbar_init(smem_u32(&out_full[i]), 1);
            mbar_init(smem_u32(&out_empty[i]), 2);  // the group in either CTA
            mbar_init(smem_u32(&res_full[i]), 1);
        }
        for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&h_full[i]), 2);  // the group in either CTA
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_empty[i]), 1);
            mbar_init(smem_u32(&y_full[i]), 1);
            mbar_init(smem_u32(&step[i]), 1);
            mbar_init(smem_u32(&y_done[i]), 1);
        }
        mbar_init(smem_u32(mma_done), 1);
        *abort_flag = 0;
        armed[0] = armed[1] = armed[2] = armed[3] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    grid_dependency_wait();

    // item -> row block, first chunk; every item has the chunks of one part (the last part may have fewer)
    auto chunks_of = [&](int item) { return min(p.per_part, p.chunks - (item % p.parts) * p.per_part); };

    // Step k: S of chunk k into the buffer that chunk k - SB's epilogue has read, then Y of chunk k - SB. Four
    // barriers each in turn tell that S(k) can be read, and that Y(k) is over: its staged values and weights are
    // free. Either is over before the one four later can be issued, whoever waits for it.
    auto wait_s = [&](uint32_t k) { return wait_bar(smem_u32(&step[k & 3u]), (k >> 2) & 1u, abort_flag, p.err); };
    auto wait_y = [&](uint32_t k) { return wait_bar(smem_u32(&y_done[k & 3u]), (k >> 2) & 1u, abort_flag, p.err); };

    if (warp == 0) {
        // ---------------- TMA producer of this CTA, in the issuer's order
        const bool one = elect_one();
        uint32_t ns = 0, ny = 0, nx = 0, k = 0;  // copies made into each ring; steps
        uint32_t last1 = 0, last2 = 0;           // 1 + the last step of the row blocks one and two back
        auto load_x = [&](int row) {
            const int b = (int)(nx % XB);
            const uint32_t before = XB == 1 ? last1 : last2;
            // a step more than NS back is known to be over (load_s of this step waited for a later one)
            if (before && (C::SG < KB || before + NS > k) && !wait_s(before - 1)) return;
            if (one) {
                const uint32_t fb = map_rank(smem_u32(&x_full[b]), 0);
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&x_full[b]), 2 * C::kX);
                armed[0] = nx + 1;
                const uint32_t a = smem_u32(x_s + b * C::kX);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    tma_load_2d_pair(a + j * kBox, &p.x, j * (Q8 ? 128 : 64), row, fb);
                    if constexpr (BWD) tma_load_2d_pair(a + (KB + j) * kBox, &p.dy, j * 64, row, fb);
                }
            }
            ++nx;
        };
        // where a chunk has more stages than the ring, the tokens of a new row block (row >= 0) come before those
        // that wait for its first products
        auto load_s = [&](int f0, int row) {
            for (int j = 0; j < KB; j += C::SG, ++ns) {
                const int slot = (int)(ns % NS);
                if (j == NS * C::SG && row >= 0) load_x(row);
                if constexpr (C::SG < KB) {
                    if (!wait_bar(smem_u32(&s_empty[slot]), ((ns / NS) & 1u) ^ 1u, abort_flag, p.err)) return;
                } else if (k >= (uint32_t)NS && !wait_s(k - NS)) return;
                if (one) {
                    const uint32_t fb = map_rank(smem_u32(&s_full[slot]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&s_full[slot]), 2 * C::kSSlot);
                    armed[1] = ns + 1;
#pragma unroll
                    for (int i = 0; i < C::SG; ++i) {
                        const uint32_t a = smem_u32(s_ring + slot * C::kSSlot + i * C::kSBlock);
                        const int c = (j + i) * (Q8 ? 128 : 64);
                        tma_load_2d_pair(a, rank ? &p.wu : &p.wg, c, f0, fb);
                        if constexpr (BWD) tma_load_2d_pair(a + 8192, &p.wd, c, f0 + (int)rank * 32, fb);
                    }
                }
            }
        };
        auto load_y = [&](int f0) {
            const int slot = (int)(ny % NY);
            if (ny >= (uint32_t)NY && !wait_y(ny - NY)) return;
            if (one) {
                const uint32_t fb = map_rank(smem_u32(&y_full[slot]), 0);
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&y_full[slot]), 2 * C::kYSlot);
                armed[2] = ny + 1;
                const uint32_t a = smem_u32(y_ring + slot * C::kYSlot);
                if constexpr (BWD) {
                    tma_load_2d_pair(a, &p.wgt, f0, (int)rank * EB * 32, fb);
                    tma_load_2d_pair(a + EB * 4096, &p.wut, f0, (int)rank * EB * 32, fb);
                } else {
                    tma_load_2d_pair(a, &p.wd, f0, (int)rank * EB * 32, fb);
                }
            }
            ++ny;
        };
        int yf[3] = {-1, -1, -1};  // hidden columns of the chunks one, two and three steps back
        for (int item = pair; item < p.items && !*abort_flag; item += n_pairs) {
            const int n = chunks_of(item), f_first = (item % p.parts) * p.per_part * 64;
            const int row = (item / p.parts) * 256 + (int)rank * 128;
            for (int c = 0; c < n && !*abort_flag; ++c, ++k) {
                constexpr bool kInside = KB > NS * C::SG;
                if (BWD && C::kOut && yf[SB - 1] >= 0) load_y(yf[SB - 1]);
                load_s(f_first + c * 64, kInside && c == 0 ? row : -1);
                // a second token buffer is filled as early as can be; a single one waits for the last step
                if (XB == 2 && c == 0) load_x(row);
                if (!BWD && C::kOut && yf[SB - 1] >= 0) load_y(yf[SB - 1]);
                if (XB == 1 && !kInside && c == 0) load_x(row);
                yf[2] = yf[1];
                yf[1] = yf[0];
                yf[0] = f_first + c * 64;
            }
            last2 = last1;
            last1 = k;
        }
        if constexpr (C::kOut)
#pragma unroll
            for (int z = SB - 1; z >= 0; --z)
                if (!*abort_flag && yf[z] >= 0) load_y(yf[z]);
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer of the pair: the whole warp walks the steps, so that addresses stay in
            // uniform registers; one lane issues
            const bool one = elect_one();
            uint32_t ns = 0, nx = 0, k = 0, n_out = 0;
            bool ok = true;
            auto wait_for = [&](uint64_t *b, uint32_t parity) {
                if (ok) ok = wait_bar(smem_u32(b), parity, abort_flag, p.err);
            };
            // y: (first | last << 1 | 4) of the chunk SB steps back, 0: none
            auto run_step = [&](uint32_t y, bool has_s, bool first, bool last) {
                const uint32_t ky = k - SB;  // the chunk of Y
                const int ys = (int)(ky % NY), yb = (int)(ky % SB), xb = (int)(nx % XB), ob = (int)(n_out % OB);
                auto wait_inputs = [&]() {
                    if (first) wait_for(&x_full[xb], (nx / XB) & 1u);
                    if constexpr (C::SG == KB) wait_for(&s_full[ns % NS], (ns / NS) & 1u);
                };
                if (has_s && !BWD) wait_inputs();  // long there: before the wait that counts
                if (y) wait_for(&h_full[yb], (ky / SB) & 1u);
                if (!ok) return;
                tc_fence_after();
                auto issue_s = [&]() {
                    if constexpr (BWD) {
                        wait_inputs();
                        if (!ok) return;
                        tc_fence_after();
                    }
                    const uint32_t d = tmem + (k % SB) * C::kSCols;
                    const uint32_t xa = smem_u32(x_s + xb * C::kX);
#pragma unroll
                    for (int j0 = 0; j0 < KB; j0 += C::SG, ++ns) {
                        const int slot = (int)(ns % NS);
                        if constexpr (C::SG < KB) {
                            wait_for(&s_full[slot], (ns / NS) & 1u);
                            if (!ok) return;
                            tc_fence_after();
                        }
                        if (one) {
#pragma unroll
                            for (int i = 0; i < C::SG; ++i) {
                                const int j = j0 + i;
                                const uint32_t b = smem_u32(s_ring + slot * C::kSSlot + i * C::kSBlock);
                                const uint64_t da = smem_desc(xa + j * kBox), db = smem_desc(b);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    mma_pair<Q8>(d, da + (uint64_t)(2 * q), db + (uint64_t)(2 * q),
                                                 idesc_of(Q8, false, 256, 128), (uint32_t)(j > 0 || q > 0));
                                if constexpr (BWD) {
                                    const uint64_t da1 = smem_desc(xa + (KB + j) * kBox), db1 = smem_desc(b + 8192);
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
                                        mma_pair<false>(d + 128, da1 + (uint64_t)(2 * q), db1 + (uint64_t)(2 * q),
                                                        idesc_of(false, false, 256, 64), (uint32_t)(j > 0 || q > 0));
                                }
                            }
                            if constexpr (C::SG < KB) mma_commit_pair(smem_u32(&s_empty[slot]));
                        }
                    }
                    if (last) ++nx;
                    if (one) mma_commit_pair(smem_u32(&step[k & 3u]));
                };
                auto issue_y = [&]() {
                    if constexpr (C::kOut) {
                        wait_for(&y_full[ys], (ky / NY) & 1u);
                        if (y & 1u) wait_for(&out_empty[ob], ((n_out / OB) & 1u) ^ 1u);
                        if (!ok) return;
                        tc_fence_after();
                        if (one) {
                            const uint32_t d = tmem + SB * C::kSCols + (uint32_t)(ob * EB * 64);
                            const uint32_t a = smem_u32(staged + (BWD ? 0 : yb) * C::kStaged);
                            const uint32_t b = smem_u32(y_ring + ys * C::kYSlot);
#pragma unroll
                            for (int z = 0; z < (BWD ? 2 : 1); ++z) {
                                const uint64_t da = smem_desc(a + z * kBox), db = smem_desc(b + z * EB * 4096);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    mma_pair<false>(d, da + (uint64_t)(2 * q), db + (uint64_t)(2 * q),
                                                    idesc_of(false, false, 256, EB * 64), z + q ? 1u : (y & 1u) ^ 1u);
                            }
                            mma_commit_pair(smem_u32(&y_done[ky & 3u]));
                            if (y & 2u) mma_commit_pair(smem_u32(&out_full[ob]));
                        }
                        if (y & 2u) ++n_out;
                    }
                };
                // Forward, S comes first: the next chunks' hidden values can be worked on while Y waits for the last
                // row block to be drained. Backward, where the next chunk's epilogue waits for Y to have read the
                // staged tiles, Y does, but for that first one.
                const bool y_first = BWD && C::kOut && !(y & 1u);
                if (y && y_first) issue_y();
                if (has_s && ok) issue_s();
                if (y && !y_first && ok) issue_y();
                __syncwarp();
                ++k;
            };
            uint32_t back = 0;  // three bits for each of the last SB chunks
            for (int item = pair; item < p.items && ok; item += n_pairs) {
                const int n = chunks_of(item);
                for (int c = 0; c < n && ok; ++c) {
                    run_step((back >> (3 * SB - 3)) & 7u, true, c == 0, c == n - 1);
                    back = back << 3 | (uint32_t)(c == 0) | (uint32_t)(c == n - 1) << 1 | 4u;
                }
            }
            for (int z = 0; z < SB && ok; ++z) {
                run_step((back >> (3 * SB - 3)) & 7u, false, false, false);
                back <<= 3;
            }
            if (one) mma_commit_pair(smem_u32(mma_done));
            __syncwarp();
            int dummy = 0;
            mbar_wait(smem_u32(mma_done), 0, (volatile int *)&dummy, p.err);
        }
    } else if (warp < 18) {
        // ---------------- chunk epilogue, 16 warps
        const int quarter = warp & 3;
        for (int i = threadIdx.x - 64; i < p.chunks * 64; i += 512) {
            const bool in = i < p.F;
            const float g = in && p.bg ? __bfloat162float(p.bg[i]) : 0.f, u = in && p.bu ? __bfloat162float(p.bu[i]) : 0.f;
            if constexpr (BWD) {
                bias_s[i] = pack_bf16(g, u);
            } else {
                bg_s[i] = Act<ACT>::kGate * g;
                bu_s[i] = Act<ACT>::kUp * u;
                if constexpr (Q8) {
                    gs_s[i] = in ? Act<ACT>::kGate * p.gs[i] : 0.f;
                    us_s[i] = in ? Act<ACT>::kUp * p.us[i] : 0.f;
                }
            }
        }
        epi_sync();  // the vectors are there
        uint32_t k = 0;
        if constexpr (!BWD) {
            // two groups of eight warps take the chunks in turn, a warp 32 of the columns
            const int g = (warp - 2) >> 3, half = ((warp - 2) >> 2) & 1;
            const bool lead = threadIdx.x == 64 + 256 * g;
            for (int item = pair; item < p.items; item += n_pairs) {
                const int n = chunks_of(item), f_first = (item % p.parts) * p.per_part * 64;
                float xs[4] = {};  // of rows g + 8 i of the warp's
                if constexpr (Q8)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = (item / p.parts) * 256 + (int)rank * 128 + quarter * 32 + 8 * i + (lane >> 2);
                        xs[i] = row < p.M ? p.xs[row] : 0.f;
                    }
                for (int c = 0; c < n; ++c, ++k) {
                    if ((k & 1u) != (uint32_t)g) continue;
                    const int f0 = f_first + c * 64, sb = (int)(k % SB);
                    const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(sb * C::kSCols);
                    uint8_t *st = staged + sb * C::kStaged;
                    wait_s(k);
                    if (k >= (uint32_t)SB) wait_y(k - SB);  // of the values that were staged here
                    tc_fence_after();
#pragma unroll 1
                    for (int s = half * 32; s < half * 32 + 32; s += 16) {  // rolled: the SM's warps share its instruction cache
                        uint32_t vg[2][8], vu[2][8];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            tmem_ld_frag(t0 + ((uint32_t)(q * 16) << 16) + (uint32_t)s, vg[q]);
                            tmem_ld_frag(t0 + ((uint32_t)(q * 16) << 16) + (uint32_t)(64 + s), vu[q]);
                        }
                        const int c2 = f0 + s + 2 * (lane & 3);
                        float bg[4], bu[4], mg[4] = {}, mu[4] = {};
                        two_pairs(bg, bg_s + c2);
                        two_pairs(bu, bu_s + c2);
                        if constexpr (Q8) {
                            two_pairs(mg, gs_s + c2);
                            two_pairs(mu, us_s + c2);
                        }
                        tmem_wait(vg[0], vu[0], vg[1], vu[1]);
                        const uint32_t at = smem_u32(st) + swizzled(quarter * 32 + (lane & 15), s / 8 + (lane >> 4));
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                float h[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int i = (j >> 2) * 2 + e;
                                    const float a = __uint_as_float(vg[q][j + e]), b = __uint_as_float(vu[q][j + e]);
                                    if constexpr (Q8) {
                                        const float x = xs[2 * q + ((j >> 1) & 1)];
                                        h[e] = Act<ACT>::hidden(fmaf(a, x * mg[i], bg[i]), fmaf(b, x * mu[i], bu[i]));
                                    } else {
                                        h[e] = Act<ACT>::hidden(fmaf(a, Act<ACT>::kGate, bg[i]),
                                                                fmaf(b, Act<ACT>::kUp, bu[i]));
                                    }
                                }
                                w[j / 2] = pack_bf16(h[0], h[1]);
                            }
                            store_frags(at + (uint32_t)(q * 16 * 128), w[0], w[1], w[2], w[3]);
                        }
                    }
                    tc_fence_before();
                    fence_async_shared();
                    asm volatile("bar.sync %0, 256;" ::"r"(1 + g) : "memory");
                    if (lead) mbar_arrive_cluster(map_rank(smem_u32(&h_full[sb]), 0));
                }
            }
        } else {
            // all warps on every chunk, a warp 16 of the columns: the three tiles that go out fit in shared
            // memory once, and a chunk's values wait in registers until the last chunk's have left it
            const int s = ((warp - 2) >> 2) * 16;
            const bool lead = threadIdx.x == 64;
            float *sums = p.sums + (size_t)(blockIdx.x * 4 + quarter) * 2 * p.F;
            // this lane's row of the four 8 x 8 matrices of 16 rows x 16 columns
            const uint32_t staged_at =
                smem_u32(staged) + swizzled(quarter * 32 + (lane & 15), s / 8 + (lane >> 4));
            for (int item = pair; item < p.items; item += n_pairs) {
                const int n = chunks_of(item), f_first = (item % p.parts) * p.per_part * 64;
                const int row0 = (item / p.parts) * 256 + (int)rank * 128;
                for (int c = 0; c < n; ++c, ++k) {
                    const int f0 = f_first + c * 64, sb = (int)(k % SB);
                    const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(sb * C::kSCols + s);
                    wait_s(k);
                    tc_fence_after();
                    uint32_t wg[8], wu[8], wh[8];
                    float cs[8] = {};
                    uint32_t bias[4];
                    *reinterpret_cast<uint2 *>(bias) = *reinterpret_cast<const uint2 *>(bias_s + f0 + s + 2 * (lane & 3));
                    *reinterpret_cast<uint2 *>(bias + 2) = *reinterpret_cast<const uint2 *>(bias_s + f0 + s + 8 + 2 * (lane & 3));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {  // 16 of the warp's rows
                        uint32_t vg[8], vu[8], vd[8];
                        const uint32_t tq = t0 + ((uint32_t)(q * 16) << 16);
                        tmem_ld_frag(tq, vg);
                        tmem_ld_frag(tq + 64, vu);
                        tmem_ld_frag(tq + 128, vd);
                        tmem_wait(vg, vu, vd);
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            float h[2], dg[2], du[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int c = (j >> 2) * 2 + e;
                                const float u = __uint_as_float(vu[j + e]) + __uint_as_float(bias[c] & 0xffff0000u);
                                const float d = __uint_as_float(vd[j + e]);
                                float slope;
                                const float act =
                                    Act<ACT>::fast(__uint_as_float(vg[j + e]) + __uint_as_float(bias[c] << 16), &slope);
                                h[e] = act * u;
                                du[e] = d * act;
                                dg[e] = d * u * slope;
                                cs[c] += dg[e];
                                cs[4 + c] += du[e];
                            }
                            wg[(8 * q + j) / 2] = pack_bf16(dg[0], dg[1]);
                            wu[(8 * q + j) / 2] = pack_bf16(du[0], du[1]);
                            wh[(8 * q + j) / 2] = pack_bf16(h[0], h[1]);
                        }
                    }
                    if (p.sums) add_column_sums(sums, cs, f0 + s, p.F, lane);
                    tc_fence_before();
                    if (lead) store_wait_read();  // the last chunk's tiles have been copied out
                    epi_sync();
                    if (C::kOut && k) wait_y(k - 1);  // and multiplied
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t at = staged_at + (uint32_t)(q * 16 * 128);
                        store_frags(at, wg[4 * q], wg[4 * q + 1], wg[4 * q + 2], wg[4 * q + 3]);
                        store_frags(at + kBox, wu[4 * q], wu[4 * q + 1], wu[4 * q + 2], wu[4 * q + 3]);
                        store_frags(at + 2 * kBox, wh[4 * q], wh[4 * q + 1], wh[4 * q + 2], wh[4 * q + 3]);
                    }
                    fence_async_shared();
                    epi_sync();
                    if (lead) {
                        mbar_arrive_cluster(map_rank(smem_u32(&h_full[sb]), 0));
                        // whole lines by TMA: stored from registers, a warp's 32 rows cost the memory pipe 32
                        // cycles an instruction
                        if (row0 < p.M && f0 < p.F) {
                            tma_store_tile(&p.dg, smem_u32(staged), f0, row0);
                            tma_store_tile(&p.du, smem_u32(staged + kBox), f0, row0);
                            tma_store_tile(&p.h, smem_u32(staged + 2 * kBox), f0, row0);
                        }
                        store_commit();
                    }
                }
            }
            if (lead) store_wait_all();
        }
    } else if constexpr (C::kOut) {
        // ---------------- the row block's result, 64 columns at a time through two tiles in shared memory: the
        // residual comes in by TMA long before, the sum goes out by TMA
        const int quarter = warp & 3, r = quarter * 32 + lane;
        const bool lead = threadIdx.x == 64 + 512, with_res = !BWD && p.has_res;
        for (int i = threadIdx.x - 576; i < EB * 64; i += 128)
            bd_s[i] = p.bd && i < p.E ? __bfloat162float(p.bd[i]) : 0.f;
        // residual of pass n (row block n / EB of this pair, columns 64 (n % EB)) into tile n % kOT
        uint32_t loaded = 0;
        auto load_res = [&]() {
            const uint32_t n = loaded++;
            const int item = pair + (int)(n / EB) * n_pairs;
            if (item >= p.items) return;
            const int row0 = (item / p.parts) * 256 + (int)rank * 128;
            const uint32_t rb = smem_u32(&res_full[n % C::kOT]);
            armed[3] = n + 1;
            if (row0 < p.M) {
                mbar_arrive_expect_tx(rb, kBox);
                tma_load_2d(smem_u32(out_s + (n % C::kOT) * kBox), &p.res, (int)(n % EB) * 64, row0, rb);
            } else {
                mbar_arrive(rb);
            }
        };
        if (lead && with_res)
            while (loaded < (uint32_t)C::kOT) load_res();
        group_sync(2);
        uint32_t i = 0, q = 0;
        for (int item = pair; item < p.items; item += n_pairs, ++i) {
            const int ob = (int)(i % OB);
            const int row0 = (item / p.parts) * 256 + (int)rank * 128;
            const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(SB * C::kSCols + ob * EB * 64);
#pragma unroll 1
            for (int cb = 0; cb < EB; ++cb, ++q) {
                uint8_t *st = out_s + (q % C::kOT) * kBox;
                if (cb == 0) {
                    wait_bar(smem_u32(&out_full[ob]), (i / OB) & 1u, abort_flag, p.err);
                    tc_fence_after();
                }
                if (with_res) {
                    wait_bar(smem_u32(&res_full[q % C::kOT]), (q / C::kOT) & 1u, abort_flag, p.err);
                } else {
                    if (lead) {  // the tile's last columns have been copied out
                        if constexpr (C::kOT == 2) store_wait_read1();
                        else store_wait_read();
                    }
                    group_sync(2);
                }
#pragma unroll 1
                for (int s = 0; s < 64; s += 32) {
                    uint32_t v0[16], v1[16];
                    tmem_read(t0 + (uint32_t)(cb * 64 + s), v0);
                    tmem_read(t0 + (uint32_t)(cb * 64 + s + 16), v1);
                    tmem_wait(v0, v1);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint4 *at = reinterpret_cast<uint4 *>(st + swizzled(r, s / 8 + u));
                        const uint4 a = with_res ? *at : make_uint4(0, 0, 0, 0);
                        const float4 b0 = *reinterpret_cast<const float4 *>(bd_s + cb * 64 + s + 8 * u);
                        const float4 b1 = *reinterpret_cast<const float4 *>(bd_s + cb * 64 + s + 8 * u + 4);
                        const uint32_t e[4] = {a.x, a.y, a.z, a.w};
                        const float bb[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t *v = u < 2 ? v0 + 8 * u : v1 + 8 * (u - 2);
                            w[j] = pack_bf16(__uint_as_float(v[2 * j]) + bb[2 * j] + __uint_as_float(e[j] << 16),
                                             __uint_as_float(v[2 * j + 1]) + bb[2 * j + 1] +
                                                 __uint_as_float(e[j] & 0xffff0000u));
                        }
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (cb == EB - 1) tc_fence_before();
                fence_async_shared();
                group_sync(2);
                if (lead) {
                    if (cb == EB - 1) mbar_arrive_cluster(map_rank(smem_u32(&out_empty[ob]), 0));
                    if (p.has_out && row0 < p.M) tma_store_tile(&p.out, smem_u32(st), cb * 64, row0);
                    store_commit();
                    // a tile takes its next residual when its store has read it: within a row block only the one
                    // that is needed next (the store before this one is long read), at its end all
                    if (with_res && (cb == EB - 1 || loaded <= q + 1)) {
                        if (cb == EB - 1) store_wait_read();
                        else store_wait_read1();
                        while (loaded <= (cb == EB - 1 ? q + C::kOT : q + 1)) load_res();
                    }
                }
            }
        }
        if (lead) store_wait_all();
    }

    __syncthreads();
    if (threadIdx.x == 0) {
        // every product has run before either CTA goes; after an expired wait the counted copies land first
        int dummy = 0;
        wait_bar(smem_u32(mma_done), 0, (volatile int *)&dummy, p.err);
        if (*abort_flag && rank == 0) {
            auto drain = [&](uint64_t *full, uint32_t made, uint32_t slots) {
                for (uint32_t i = made > slots ? made - slots : 0; i < made; ++i)
                    wait_bar(smem_u32(&full[i % slots]), (i / slots) & 1u, (volatile int *)&dummy, p.err);
            };
            drain(x_full, armed[0], XB);
            drain(s_full, armed[1], NS);
            drain(y_full, armed[2], NY);
        }
        if (*abort_flag && armed[3])
            for (uint32_t i = armed[3] > C::kOT ? armed[3] - C::kOT : 0; i < armed[3]; ++i)
                mbar_wait(smem_u32(&res_full[i % C::kOT]), (i / C::kOT) & 1u, (volatile int *)&dummy, p.err);
    }
    __syncthreads();
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------- host side

template <int EB, bool BWD, bool Q8, int ACT>
pmha_status launch(Params &p, const char *stage, cudaStream_t s)
{
    using C = Cfg<EB, BWD, Q8>;
    static_assert(C::kSmem <= kSmemMost, "shared memory of one CTA");
    p.err = device_error_word();
    if (!p.err) return PMHA_ERR_CUDA;
    int pairs = 0;
    auto kern = k_block<EB, BWD, Q8, ACT>;
    static std::atomic<int> known[kKnownDevices];
    const pmha_status st = pairs_at_once(kern, kThreads, C::kSmem, known, &pairs);
    if (st != PMHA_OK) return st;
    if (C::kOut) p.parts = 1;
    else {
        // parts of the hidden width even out the last wave of row blocks
        int best = 1;
        double best_cost = 1e30;
        for (int parts = 1; parts <= std::min(p.chunks, 8); ++parts) {
            const int per = (p.chunks + parts - 1) / parts;
            const int64_t waves = ((int64_t)p.items * ((p.chunks + per - 1) / per) + pairs - 1) / pairs;
            const double cost = (double)waves * (per + 1);  // a part costs about a chunk more for its tokens
            if (cost < best_cost) best_cost = cost, best = parts;
        }
        p.parts = best;
    }
    p.per_part = (p.chunks + p.parts - 1) / p.parts;
    p.parts = (p.chunks + p.per_part - 1) / p.per_part;
    p.items *= p.parts;
    StageTimer timer(stage, s);
    return launch_overlapping(kern, dim3(2u * (unsigned)std::min(pairs, p.items)), kThreads, C::kSmem, s, p);
}

template <int EB, bool BWD, bool Q8>
pmha_status launch_act(pmha_act act, Params &p, const char *stage, cudaStream_t s)
{
    return act == PMHA_ACT_SILU ? launch<EB, BWD, Q8, PMHA_ACT_SILU>(p, stage, s)
                                : launch<EB, BWD, Q8, PMHA_ACT_GELU>(p, stage, s);
}

template <bool BWD, bool Q8>
pmha_status launch_width(pmha_act act, Params &p, const char *stage, cudaStream_t s)
{
    switch ((p.E + 63) / 64) {
    case 1: return launch_act<1, BWD, Q8>(act, p, stage, s);
    case 2: return launch_act<2, BWD, Q8>(act, p, stage, s);
    case 3: return launch_act<3, BWD, Q8>(act, p, stage, s);
    default: return launch_act<4, BWD, Q8>(act, p, stage, s);
    }
}

}  // namespace

bool ffn_fused_supported(int64_t E, int64_t F)
{
    return E <= 256 && F <= Cfg<1, false, false>::kMaxHidden;
}
bool ffn_fused_dx(int64_t E) { return E <= 128; }

pmha_status ffn_fused_forward(const FfnTc &f, const FfnUpArgs &a, const void *wd, const void *residual, void *out,
                              cudaStream_t s)
{
    Params p = {};
    const bool q8 = a.x_scale != nullptr;
    const int es = q8 ? 1 : 2;
    const int eb = (int)((f.E + 63) / 64);
    p.M = (int)a.M, p.E = (int)f.E, p.F = (int)f.F;
    p.items = (int)((a.M + 255) / 256);
    p.chunks = (int)((f.F + 63) / 64);
    p.bg = (const __nv_bfloat16 *)f.bg, p.bu = (const __nv_bfloat16 *)f.bu, p.bd = (const __nv_bfloat16 *)f.bd;
    p.xs = a.x_scale, p.gs = a.wg_scale, p.us = a.wu_scale;
    p.has_out = 1;
    p.has_res = residual != nullptr;
    if (!make_tile_map(&p.x, a.x, a.M, f.E, f.E, es, 128) || !make_tile_map(&p.wg, a.wg, f.F, f.E, f.E, es, 64) ||
        !make_tile_map(&p.wu, a.wu, f.F, f.E, f.E, es, 64) ||
        !make_tile_map(&p.wd, wd, f.E, f.F, f.F, 2, (uint32_t)(eb * 32)) ||
        !make_tile_map(&p.out, out, a.M, f.E, f.E, 2, 128) ||
        (residual && !make_tile_map(&p.res, residual, a.M, f.E, f.E, 2, 128))) {
        set_error("ffn_block: cuTensorMapEncodeTiled failed");
        return PMHA_ERR_CUDA;
    }
    return q8 ? launch_width<false, true>(f.act, p, "ffn_block_quantized", s)
              : launch_width<false, false>(f.act, p, "ffn_block", s);
}

pmha_status ffn_fused_backward(const FfnTc &f, const FfnHiddenArgs &a, const void *wg_t, const void *wu_t, void *dx,
                               cudaStream_t s)
{
    Params p = {};
    const int eb = (int)((f.E + 63) / 64);
    p.M = (int)a.M, p.E = (int)f.E, p.F = (int)f.F;
    p.items = (int)((a.M + 255) / 256);
    p.chunks = (int)((f.F + 63) / 64);
    p.bg = (const __nv_bfloat16 *)f.bg, p.bu = (const __nv_bfloat16 *)f.bu;
    p.has_out = dx != nullptr;
    p.sums = a.sums;
    if (!make_tile_map(&p.x, a.x, a.M, f.E, f.E, 2, 128) || !make_tile_map(&p.dy, a.dy, a.M, f.E, f.E, 2, 128) ||
        !make_tile_map(&p.wg, a.wg, f.F, f.E, f.E, 2, 64) || !make_tile_map(&p.wu, a.wu, f.F, f.E, f.E, 2, 64) ||
        !make_tile_map(&p.wd, a.wd_t, f.F, f.E, f.E, 2, 32) ||
        !make_tile_map(&p.h, a.h, a.M, f.F, f.F, 2, 128) || !make_tile_map(&p.dg, a.dg, a.M, f.F, f.F, 2, 128) ||
        !make_tile_map(&p.du, a.du, a.M, f.F, f.F, 2, 128) ||
        (dx && !make_tile_map(&p.out, dx, a.M, f.E, f.E, 2, 128)) ||
        !make_tile_map(&p.wgt, wg_t, f.E, f.F, f.F, 2, (uint32_t)(eb * 32)) ||
        !make_tile_map(&p.wut, wu_t, f.E, f.F, f.F, 2, (uint32_t)(eb * 32))) {
        set_error("ffn_block_backward: cuTensorMapEncodeTiled failed");
        return PMHA_ERR_CUDA;
    }
    return launch_width<true, false>(f.act, p, "ffn_block_backward", s);
}

}  // namespace pmha
