// tcgen05.cuh -- inline-PTX wrappers for the fifth-generation tensor cores
// (sm_103a): tensor memory, e4m3 matrix products with fp32 accumulators, tiled
// bulk tensor loads, and the descriptors they take.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

// ------------------------------------------------------------ tensor memory

// kCtas = 2: a pair of blocks (a cluster of two) works on one product, each
// block holding half of the rows of A and of the result, and half of B.

// Whole warp (of each block of a pair).  Writes the base address of the
// allocated columns to *slot.
template <int kCtas, int kColumns>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot) {
    if (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "n"(kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "n"(kColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <int kCtas, int kColumns>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    if (kCtas == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(kColumns));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(kColumns));
}

// 32 lanes x 16 columns of fp32: thread = lane (row), one register per column.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// Waits for the loads of tensor memory this thread has issued.  Nothing may
// touch a load's registers before, so they pass through here.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tcgen05_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ------------------------------------------------------------- descriptors

// Shared-memory operand descriptor of a 128-byte-swizzled tile: start address,
// leading and stride byte offsets (16-byte units), version 1, swizzle code 2.
// K-major (a row of 128 bytes along K): stride = 1024 between groups of 8
// rows; the leading offset is not used.  MN-major (a row of 128 bytes along M
// or N): leading = distance of the next 128 bytes along M or N, stride = 1024
// between groups of 8 steps along K.
__device__ __forceinline__ uint64_t smem_descriptor(uint32_t addr, uint32_t leading, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: e4m3 x e4m3, fp32 accumulators, M x N, A K-major.
__host__ __device__ constexpr uint32_t f8_instruction(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The instructions below that one thread issues take `issue`: the warp runs
// them together and the thread that has it set issues.  A predicate costs
// nothing, where a branch around them splits the warp and joins it again
// (tens of cycles each time, on the path that feeds the tensor cores).

// d (tensor memory) = a x b, or += with accumulate; K = 32.  One thread of a
// block, of a pair's first block.
template <int kCtas>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, bool accumulate,
                                       bool issue) {
    if (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(instruction), "r"((uint32_t)accumulate), "r"((uint32_t)issue)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(instruction), "r"((uint32_t)accumulate), "r"((uint32_t)issue)
            : "memory");
}

// Arrives once on `bar` (of both blocks of a pair) when every product this
// thread has issued is complete.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint32_t bar, bool issue) {
    if (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
                "r"(bar),
            "h"((uint16_t)3), "r"((uint32_t)issue)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"((uint32_t)issue)
            : "memory");
}

// ------------------------------------------------------ tiled tensor loads

// Into this block's shared memory; the bytes count on `bar`, for a pair on the
// barrier at that place in its first block.
template <int kCtas>
__device__ __forceinline__ uint32_t barrier_address(uint32_t bar) {
    return kCtas == 2 ? bar & 0xfeffffffu : bar;   // bit 24: which block of the pair
}

template <int kCtas>
__device__ __forceinline__ void tensor_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar,
                                               bool issue) {
    if (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(barrier_address<2>(bar)), "r"((uint32_t)issue)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(barrier_address<1>(bar)), "r"((uint32_t)issue)
            : "memory");
}

template <int kCtas>
__device__ __forceinline__ void tensor_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar,
                                               bool issue) {
    if (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(barrier_address<2>(bar)), "r"((uint32_t)issue)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(barrier_address<1>(bar)), "r"((uint32_t)issue)
            : "memory");
}

__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------- barriers

// Waits for a barrier's phase with a limit of a second or two: false if it did
// not complete.  The limit counts polls, so that a wait costs no look at a
// clock: a poll answers in about 55 cycles if the phase is complete and else
// suspends the warp for up to 1.3 us (measured), until it is.
__device__ __forceinline__ bool mbar_wait_polls(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, more;\n\t.reg .b32 n;\n\t"
        "mov.b32 n, 1048576;\n"
        "POLL:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.s32 n, n, 1;\n\t"
        "setp.gt.s32 more, n, 0;\n\t"
        "@more bra POLL;\n"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar, bool issue) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"((uint32_t)issue)
        : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes, bool issue) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"((uint32_t)issue)
        : "memory");
}

// The address, for the cluster, of a place of this block's shared memory in
// another of its blocks.
__device__ __forceinline__ uint32_t block_address(uint32_t p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(p), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t first_block_address(uint32_t p) { return block_address(p, 0); }

__device__ __forceinline__ void st_cluster_v4(uint32_t p, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// Arrives on a barrier by such an address.  Relaxed: what it orders are reads of
// tensor memory, behind tcgen05 fences (a release at cluster scope took about
// 900 cycles, twice a stage's products).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar, bool issue) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"((uint32_t)issue)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of every block of the cluster; a warp's lanes arrive together.
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_mbarrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// 16 bytes of shared memory by its address.
__device__ __forceinline__ void st_shared_v4(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}

// A warpgroup's share of the block's registers (whole warpgroup; the shares
// may not sum to more than the block was launched with).
template <int kRegisters>
__device__ __forceinline__ void registers_increase() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegisters));
}
template <int kRegisters>
__device__ __forceinline__ void registers_decrease() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegisters));
}

}  // namespace moe
