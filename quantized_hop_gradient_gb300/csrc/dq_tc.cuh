// dq_tc.cuh -- tensor-core plumbing of the attention kernels (sm_103a):
// bounded mbarrier waits, tensor-map copies into 128-byte swizzled tiles,
// tcgen05 products with accumulators in tensor memory.
//
// A tile is 128 rows of 64 or 128 16-bit elements, kept as one or two boxes
// of 128 rows x 128 bytes (16 KiB, 1024-byte aligned); within a box the
// hardware exchanges a row's 16-byte pieces by the row number mod 8.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dq {
namespace tc {

constexpr int kTile = 128;                 // rows of a tile, lanes of tensor memory
constexpr int kBoxBytes = kTile * 128;
constexpr long long kWaitCycles = 2000000000ll;   // bound of a wait: about a second
// Of one for work, which may be far: empty slots and padding are passed over at 8.6 ns a block of the grid (32 million
// blocks in 276 ms), 18 s for the largest grid.
constexpr long long kQueueCycles = 64 * kWaitCycles;

// ---- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Waits for the phase of that parity.  False once `abort` is set or the time
// is up, which sets it, so that every role of the block gives up together.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort, long long most)
{
    const long long start = clock64();
    while (!mbar_try(bar, parity)) {
        if (*abort) return false;
        if (clock64() - start > most) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
// Called by whole warps; the answer is the same in every lane.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort, long long most = kWaitCycles)
{
    if (__all_sync(0xFFFFFFFFu, mbar_try(bar, parity))) return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait_slow(bar, parity, abort, most));
}

// For a block that gives up: waits, still with a limit, until what it has sent
// off has landed.  Called by whole warps.  A barrier that was never used counts
// as landed: its phase before the first is odd.
__device__ __forceinline__ void mbar_land(uint32_t bar, uint32_t parity)
{
    const long long start = clock64();
    while (!__all_sync(0xFFFFFFFFu, mbar_try(bar, parity) || clock64() - start > kWaitCycles)) {
    }
}

// Register split between warpgroups; the shares must add up to what the block
// was launched with.  Executed by all warps of a warpgroup.
template <int REGS> __device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS> __device__ __forceinline__ void give_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// The same by a single thread.
__device__ __forceinline__ bool mbar_wait_one(uint32_t bar, uint32_t parity, volatile int *abort,
                                              long long most = kWaitCycles)
{
    return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, abort, most);
}
// One thread of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- the grid's blocks that have not started yet
// Asks for one of them; the answer, 16 bytes at `answer`, completes `bar`.
// Only while no earlier request has been refused.
__device__ __forceinline__ void claim_block(uint32_t answer, uint32_t bar)
{
    mbar_expect(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar)
                 : "memory");
}
// Whether a block was given, which will then not start by itself, and its index.
__device__ __forceinline__ bool claimed_block(uint32_t answer, unsigned &block)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
                 "ld.shared.b128 r, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
                 : "=r"(ok), "=r"(block)
                 : "r"(answer)
                 : "memory");
    return ok != 0;
}

// ---- copies
__device__ __forceinline__ void load_box(uint32_t dst, const void *map, int x, int h, int t, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(h), "r"(t), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void prefetch_map(const void *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory
template <int COLS> __device__ __forceinline__ void tmem_alloc(uint32_t dst_smem)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "n"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS> __device__ __forceinline__ void tmem_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLS));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_smem_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define DQ_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                    "=r"(r[i + 6]), "=r"(r[i + 7])
#define DQ_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                    "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of the thread's own lane (lane 32 (warp mod 4) + lane of the warp).
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : DQ_R8(r, 0), DQ_R8(r, 8), DQ_R8(r, 16), DQ_R8(r, 24)
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : DQ_R8(r, 0), DQ_R8(r, 8)
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
                 DQ_I8(r, 0), DQ_I8(r, 8), DQ_I8(r, 16), DQ_I8(r, 24)
                 : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 DQ_I8(r, 0), DQ_I8(r, 8)
                 : "memory");
}

// ---- products
// Shared-memory operand: start address, leading and stride byte offsets (in
// 16-byte units), descriptor version 1, 128-byte swizzle.
//   K-major (rows x K, K contiguous): stride = 1024 between groups of 8 rows;
//     16 elements of K further = 32 bytes, 64 elements = the next box.
//   MN-major (K x columns, columns contiguous): leading = the distance of the
//     next 64 columns (a box), stride = 1024 between groups of 8 K rows; 16
//     rows of K further = 2048 bytes.
// Only the low word differs between operands, and steps along K add to it: one
// addition a product, because a lone thread issues them and must keep ahead
// of the tensor pipe (64 cycles for 128 x 128 x 16).  With the descriptors
// put together anew for each product the issue bounded the forward kernel,
// which took 16% longer (15,193 tokens of 32 heads of 128).
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
// An operand's address is its offset in the block's shared memory; in a cluster
// a shared-memory address carries the block's rank above its 18 bits.
template <bool CLUSTER> __device__ __forceinline__ uint32_t operand(uint32_t addr) { return CLUSTER ? addr & 0x3FFFFu : addr; }
__device__ __forceinline__ uint32_t k_major(uint32_t addr) { return addr >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t mn_major(uint32_t addr) { return addr >> 4 | (uint32_t)(kBoxBytes >> 4) << 16; }
// Instruction descriptor: fp32 accumulators, M = 128, operands bf16 or fp16.
__host__ __device__ constexpr uint32_t instr(bool bf16, int n, bool b_mn_major)
{
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 |
           (uint32_t)(kTile / 16) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHigh)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "mov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHigh)
                 : "memory");
}
// The barrier completes a phase once all products issued before by this thread are done.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// D[128 x 128] = a b^T over 16 STEPS elements; a and b are tiles in shared
// memory.  (STEPS is a constant of the kernel: with a count at run time the
// product thread fell behind, 671 us for a forward pass against 588.)
template <int STEPS> __device__ __forceinline__ void product_abt(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc)
{
    const uint32_t da = k_major(a), db = k_major(b);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const uint32_t off = (uint32_t)(k >> 2) * (kBoxBytes >> 4) + (uint32_t)(k & 3) * 2;
        mma_ss(d, da + off, db + off, idesc, k > 0);
    }
}
// D[128 x n] (+)= a b over 128 rows of b, n by idesc; a in tensor memory, two
// elements a column, in PARTS parts that lie 128 / PARTS columns apart; b as
// it lies in memory (MN-major).
template <int PARTS> __device__ __forceinline__ void product_ab(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    const uint32_t db = mn_major(b);
    constexpr int kSteps = 8 / PARTS;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_ts(d, a + k / kSteps * (128 / PARTS) + k % kSteps * 8, db + (2048 >> 4) * k, idesc, add || k > 0);
}

// ---- arithmetic
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// Zeroes rows [first, 128) of a tile; called by a whole warp.
template <int BOXES> __device__ __forceinline__ void zero_rows(uint32_t tile, int first, int lane)
{
    for (int b = 0; b < BOXES; ++b)
        for (int i = first * 8 + lane; i < kTile * 8; i += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * kBoxBytes + i * 16), "r"(0)
                         : "memory");
    fence_smem_to_async();
    __syncwarp();
}

}  // namespace tc
}  // namespace dq
