// Device helpers for matrix products on the 5th-generation tensor cores by a
// pair of CTAs: tiled bulk copies into swizzled shared memory, mbarriers with
// bounded waits, and the tcgen05 instructions.  All take part in a cluster of
// two CTAs (cta_group::2); CTA 0 of the pair, the leader, issues the products.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "ar_kernels_tma.cuh"

namespace tps {

constexpr unsigned long long kUmmaTimeoutNs = 2ull * 1000 * 1000 * 1000;

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One lane of the (whole) warp.  The warps that feed the tensor cores run their loops together and
// only issue from one lane: what the instructions take then stays in uniform registers (a loop run by
// lane 0 alone took 68 cycles for each product, whatever its size, and was the bound of small tiles).
__device__ __forceinline__ bool elect_one() {
    unsigned p;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xFFFFFFFF; selp.u32 %0, 1, 0, q; }" : "=r"(p));
    return p != 0;
}
// The address, in the cluster's shared memory, of the leader's copy of a variable of this CTA.
__device__ __forceinline__ unsigned leader_addr(unsigned local) {
    unsigned a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(local));
    return a;
}

__device__ __forceinline__ bool mbar_try(unsigned addr, unsigned parity) {
    unsigned done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    return done != 0;
}
// Wait for the phase of the given parity; false when kUmmaTimeoutNs ran out or another warp gave up.
// The clock and the flag are read only once the first try has failed: the threads that feed the
// tensor cores have a few hundred cycles for a block of K.
__device__ __forceinline__ bool mbar_wait_slow(unsigned addr, unsigned parity, const volatile unsigned *abort_flag) {
    const unsigned long long deadline = global_ns() + kUmmaTimeoutNs;
    while (!mbar_try(addr, parity))
        if (*abort_flag || global_ns() > deadline) return false;
    return true;
}
__device__ __forceinline__ bool mbar_wait_bounded(unsigned addr, unsigned parity, const volatile unsigned *abort_flag) {
    return mbar_try(addr, parity) || mbar_wait_slow(addr, parity, abort_flag);
}
__device__ __forceinline__ void mbar_arrive_cluster(unsigned cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Copy a box of a 3-D tensor into this CTA's shared memory; its bytes count on the barrier at
// `cluster_bar`, which may be the leader's.  x starts on a 16-byte boundary of its row; what lies
// outside the tensor arrives as zeros.
__device__ __forceinline__ void tma_load_3d(unsigned smem_dst, const CUtensorMap *map, unsigned cluster_bar, int x, int y,
                                            int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(smem_dst),
        "l"(map), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Shared-memory operand descriptor of a 128-byte swizzled tile (its start 1024-byte aligned).
//   K-major: rows of 64 elements along K, eight-row groups 1024 bytes apart (`lead` unused).
//   MN-major: chunks of 64 elements along M or N; within a chunk one 128-byte row for each k, groups
//   of eight k 1024 bytes apart, and chunks `lead` bytes apart.
__device__ __forceinline__ uint64_t umma_desc(unsigned smem, unsigned lead) {
    return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: float accumulators, A and B both f16 or both bf16, M = 256 over the pair.
__host__ __device__ constexpr uint32_t umma_idesc(bool bf16, bool a_mn, bool b_mn, unsigned n) {
    return (1u << 4) | (static_cast<uint32_t>(bf16) << 7) | (static_cast<uint32_t>(bf16) << 10) |
           (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) | ((n >> 3) << 17) | ((256u >> 4) << 24);
}

// D[tmem] (+)= A B^T over 16 elements of K; one thread of the leader issues it for the pair.
__device__ __forceinline__ void umma(unsigned tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(accumulate))
        : "memory");
}
// Arrive on the barrier at this offset in both CTAs once all products issued so far have finished.
__device__ __forceinline__ void umma_commit(unsigned bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<unsigned short>(3))
        : "memory");
}
__device__ __forceinline__ void tmem_alloc(unsigned smem_dst, unsigned cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols)
                 : "memory");
}
__device__ __forceinline__ void tmem_dealloc(unsigned tmem, unsigned cols) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 TMEM lanes, one lane per thread.
__device__ __forceinline__ void tmem_load32(unsigned addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
}

// The same, added to `sum`.
__device__ __forceinline__ void tmem_add32(unsigned addr, float *sum) {
    float v[32];
    tmem_load32(addr, v);
#pragma unroll
    for (int k = 0; k < 32; ++k) sum[k] = __fadd_rn(sum[k], v[k]);
}

}  // namespace tps
