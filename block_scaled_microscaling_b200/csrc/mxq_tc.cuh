// mxq_tc.cuh -- PTX wrappers for the 5th-generation tensor cores (sm_100a): tensor memory,
// block-scaled tcgen05.mma, scale copies into tensor memory, descriptors.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "mxq_device.cuh"

namespace mxq {

// ---- tensor memory ------------------------------------------------------------------------

// PAIR: the two CTAs of a cluster work on one tile (cta_group::2); one value throughout a kernel.

// a whole warp (PAIR: of each CTA) allocates / frees NCOL columns (a power of two, 32 .. 512); the address goes
// to shared memory
template <int NCOL, bool PAIR = false> __device__ __forceinline__ void tmem_alloc(uint32_t smem_dst) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "n"(NCOL) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "n"(NCOL) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int NCOL, bool PAIR = false> __device__ __forceinline__ void tmem_free(uint32_t taddr) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(NCOL));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(NCOL));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive columns of the warp's 32 lanes; tmem_wait_ld before the registers are used
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- descriptors --------------------------------------------------------------------------

// A shared-memory descriptor is a constant high word and a low word that is the address / 16 (and a constant), so a
// step along the operand is one 32-bit addition.
struct SmemDesc {
    uint32_t lo, hi;
    __device__ __forceinline__ SmemDesc operator+(uint32_t bytes) const { return {lo + (bytes >> 4), hi}; }
};
// operand tile, K-major rows of 128 bytes with the 128-byte swizzle (1024-byte aligned groups of eight rows, 1024
// bytes apart)
__device__ __forceinline__ SmemDesc desc_sw128(uint32_t saddr) {
    return {((saddr >> 4) & 0x3FFFu) | (1u << 16), 64u | (1u << 14) | (2u << 29)};
}
// 512-byte scale tile: 32 rows of 16 bytes, no swizzle (groups of eight rows 128 bytes apart)
__device__ __forceinline__ SmemDesc desc_scales(uint32_t saddr) { return {(saddr >> 4) & 0x3FFFu, 8u | (1u << 14)}; }
// one thread of a converged warp; the operands that the whole warp computes stay in uniform registers
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}
// instruction descriptor of the block-scaled kinds: both operands of element format F, K-major, E8M0 scales
template <int F> __host__ __device__ constexpr uint32_t idesc_block_scaled(int m, int n) {
    const uint32_t fmt = F == F_E2M1 ? 1u : 0u;  // mxf4: E2M1 = 1; mxf8f6f4: E4M3 = 0
    return (fmt << 7) | (fmt << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24);
}

// kind::f16, f16 operands, fp32 accumulators, both K-major
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ---- instructions (one thread issues) -------------------------------------------------------

// scale tile -> four tensor-memory columns: row r of 128 at lane r % 32, column r / 32 (copied to all four
// lane groups), its four block scales in the column's four bytes (PAIR: in both CTAs, each from its own tile)
template <bool PAIR = false> __device__ __forceinline__ void tc_copy_scales(uint32_t taddr, SmemDesc d) {
    if constexpr (PAIR)
        asm volatile("{ .reg .b64 d; mov.b64 d, {%1, %2};\n tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d; }" ::"r"(taddr),
                     "r"(d.lo), "r"(d.hi)
                     : "memory");
    else
        asm volatile("{ .reg .b64 d; mov.b64 d, {%1, %2};\n tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d; }" ::"r"(taddr),
                     "r"(d.lo), "r"(d.hi)
                     : "memory");
}
// D += A B^T with the scales of A's rows at tensor-memory column sfa and of B's rows at sfb (PAIR: each CTA holds
// half of A's and of B's rows, and all of B's scales)
#define MXQ_MMA(GROUP, KIND, VEC)                                                                                      \
    asm volatile("{ .reg .pred p; .reg .b64 a, b; setp.ne.u32 p, %8, 0;\n"                                            \
                 "mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"                                                       \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC                         \
                 " [%0], a, b, %5, [%6], [%7], p; }" ::"r"(d),                                                         \
                 "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate) \
                 : "memory")
template <int F, bool PAIR = false>
__device__ __forceinline__ void tc_mma_block_scaled(uint32_t d, SmemDesc a, SmemDesc b, uint32_t idesc,
                                                    uint32_t sfa, uint32_t sfb, bool accumulate) {
    if constexpr (F == F_E2M1 && PAIR) MXQ_MMA("2", "mxf4", "2X");
    else if constexpr (F == F_E2M1) MXQ_MMA("1", "mxf4", "2X");
    else if constexpr (PAIR) MXQ_MMA("2", "mxf8f6f4", "1X");
    else MXQ_MMA("1", "mxf8f6f4", "1X");
}
#undef MXQ_MMA
// D (+)= A B^T, f16: A from shared memory, or from tensor memory (row per lane, two values of k per column)
__device__ __forceinline__ void tc_mma_f16(uint32_t d, SmemDesc a, SmemDesc b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 a, b; setp.ne.u32 p, %6, 0;\n"
        "mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p; }" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, SmemDesc b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 b; setp.ne.u32 p, %5, 0;\n"
        "mov.b64 b, {%2, %3};\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p; }" ::"r"(d),
        "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// arrive on an mbarrier once everything this thread issued to the tensor core has completed (PAIR: on the barrier
// at this address in both CTAs)
template <bool PAIR = false> __device__ __forceinline__ void tc_commit(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- clusters -----------------------------------------------------------------------------

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// cluster address of this CTA's shared address `saddr` in the CTA of rank `rank`
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
    uint32_t p;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(saddr), "r"(rank));
    return p;
}
// arrive on an mbarrier of any CTA of the cluster (a cluster address)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t caddr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
// a float at this CTA's shared address `saddr`, read from the CTA of rank `rank`
__device__ __forceinline__ float ld_peer_f32(uint32_t saddr, uint32_t rank) {
    uint32_t p;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_peer_f32x4(uint32_t saddr, uint32_t rank) {  // four of them, 16-byte aligned
    uint32_t p;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
    return v;
}

}  // namespace mxq
