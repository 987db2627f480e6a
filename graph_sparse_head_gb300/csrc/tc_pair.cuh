// Building blocks of kernels whose CTAs work in pairs (a cluster of two): one
// tcgen05.mma covers 256 rows, 128 in each CTA's tensor memory, and each CTA
// brings half of the B operand, so that an SM fills its shared memory with
// half the operand bytes of a CTA working alone. The even CTA (rank 0) issues
// the products; its barriers count the copies and arrivals of both.
#pragma once

#include <atomic>

#include "tc_util.cuh"

namespace pmha {
namespace tcu {
namespace {

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// address of the same shared-memory word in CTA `rank` of the pair
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrival on a barrier of either CTA (a shared::cluster address). What the
// barriers of a pair hand over is read and written by the tensor core and the
// copy engine, ordered by fence.proxy.async and tcgen05.fence; the arrivals
// and waits keep CTA scope. (An acquire or release of cluster scope
// costs 400 to 600 cycles each: a chunk of the fused block took 3,100 cycles
// with them, most of it in waits on barriers already complete.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait with the usual case, a phase already complete, in line.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *err)
{
    return mbar_try_wait(bar, parity) || mbar_wait(bar, parity, abort_flag, err);
}
// Waits for the launches this one was allowed to start before the end of; lets
// the next one start likewise (its blocks come up as this one's leave, which
// hides the launch). Everything that touches global memory comes after.
__device__ __forceinline__ void grid_dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait()
{
    grid_dependents_may_start();
    grid_wait();
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// A tile into this CTA's shared memory, its bytes counted by a barrier of either CTA.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// kind::f16 (16-bit operands) or kind::f8f6f4 (E4M3), 256 rows over the pair
template <bool Q8>
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate)
{
    if constexpr (Q8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// arrives on the barrier at this offset in both CTAs when the products issued so far are done
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t holder, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(holder), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t base, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// Descriptor of an operand whose M (or N) index is contiguous, written by TMA
// as boxes of 64 such columns (128 bytes, 128-byte swizzle) by K rows: 8-row
// atoms 1024 bytes apart along K (stride offset), boxes `box_bytes` apart
// along M (leading offset). A step of 16 along K is 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t box_bytes)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor: D float32 (bits 4-5 = 1), types of A and B at bits
// 7-9 and 10-12 (kind::f16: 1 = bf16; kind::f8f6f4: 0 = E4M3), A and B
// contiguous along M / N instead of K (bits 15, 16), N >> 3 at bits 17-22,
// M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t idesc_of(bool q8, bool mn_major, int m, int n)
{
    return (1u << 4) | (q8 ? 0u : (1u << 7) | (1u << 10)) | (mn_major ? (1u << 15) | (1u << 16) : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// 16 accumulator columns of this warp's 32 rows
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tma_store_tile(const CUtensorMap *map, uint32_t src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// named barrier 1 + g over 128 threads
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
// 16 rows (taddr's lane and on) x 16 accumulator columns, eight values a lane,
// spread like the result of a warp's matrix product: with g = lane / 4, t = lane % 4,
// r[4 c + 2 h + e] is row g + 8 h, column 8 c + 2 t + e. A lane so holds four
// columns of several rows: column sums are mostly its own additions, and it
// needs four columns' biases instead of sixteen.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
// Four 8 x 8 matrices of 16-bit values in that layout (two columns a register)
// to shared memory; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void store_frags(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// The values of columns 2 t, 2 t + 1, 8 + 2 t, 9 + 2 t; p is at the first.
__device__ __forceinline__ void two_pairs(float (&f)[4], const float *p)
{
    const float2 a = *reinterpret_cast<const float2 *>(p), b = *reinterpret_cast<const float2 *>(p + 8);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
// Adds the sums over a warp's rows of 16 columns' dg and du (float32, before
// their rounding: the bias gradients) to this warp's row of partial sums, [2][F]
// from `sums`, columns col .. col + 15. v: the lane's own sums, dg's columns
// 8 c + 2 t + e at v[2 c + e], du's four further. One warp owns each value, so the
// additions' order is fixed, and they need no read.
__device__ __forceinline__ void add_column_sums(float *sums, float (&v)[8], int col, int F, int lane)
{
#pragma unroll
    for (int h = 4, o = 16; h > 0; h >>= 1, o >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const bool up = lane & o;
            const float keep = up ? v[i + h] : v[i], send = up ? v[i] : v[i + h];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    const int i = lane >> 2, c = col + ((i >> 1) & 1) * 8 + 2 * (lane & 3) + (i & 1);
    if (c < F)
        asm volatile("red.global.add.f32 [%0], %1;" ::"l"(sums + (i >= 4 ? (size_t)F : 0) + c), "f"(v[0]) : "memory");
}

// 16-byte unit u (0..7) of row r of a 128-byte-wide tile with 128-byte swizzle
__device__ __forceinline__ uint32_t swizzled(int r, int u) { return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4)); }

// A launch of `grid` CTAs that may come up before the launch before it has
// ended (the kernel calls grid_wait before it reads what that one writes).
template <typename P>
pmha_status launch_overlapping(void (*kern)(P), dim3 grid, int threads, int smem, cudaStream_t s, const P &p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    PMHA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, p));
    count_launch();
    return PMHA_OK;
}

// Pairs of `threads`-thread CTAs with `smem` bytes that run at once on the
// current device, and the kernel's permission to use that much shared memory.
// `known` holds the answer for the first devices; two threads that ask at once
// both find it.
constexpr int kKnownDevices = 64;
template <typename P>
pmha_status pairs_at_once(void (*kern)(P), int threads, int smem, std::atomic<int> (&known)[kKnownDevices], int *pairs)
{
    int dev = 0;
    PMHA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < kKnownDevices && (*pairs = known[dev].load(std::memory_order_acquire)) > 0) return PMHA_OK;
    PMHA_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    PMHA_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
    const int most = num_sms() / 2;
    *pairs = n < 1 ? 1 : n < most ? n : most;
    if (dev < kKnownDevices) known[dev].store(*pairs, std::memory_order_release);
    return PMHA_OK;
}

// 2-D map of rows x cols elements of es bytes (1: bytes, 2: bf16), row pitch
// in elements, box of 128 bytes x box_rows, 128-byte swizzle.
inline bool make_tile_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t pitch, int es,
                          uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(pitch * es)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / es), box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace
}  // namespace tcu
}  // namespace pmha
