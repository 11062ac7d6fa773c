// mxq_tc.cuh -- PTX wrappers for the 5th-generation tensor cores (sm_100a): tensor memory,
// block-scaled tcgen05.mma, scale copies into tensor memory, descriptors.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "mxq_device.cuh"

namespace mxq {

// ---- tensor memory ------------------------------------------------------------------------

// a whole warp allocates / frees NCOL columns (a power of two, 32 .. 512); the address goes to shared memory
template <int NCOL> __device__ __forceinline__ void tmem_alloc(uint32_t smem_dst) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "n"(NCOL) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int NCOL> __device__ __forceinline__ void tmem_free(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(NCOL));
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- descriptors --------------------------------------------------------------------------

// operand tile in shared memory, K-major rows of 128 bytes with the 128-byte swizzle (1024-byte aligned
// groups of eight rows, 1024 bytes apart)
__device__ __forceinline__ unsigned long long desc_sw128(uint32_t saddr) {
    return (unsigned long long)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// 512-byte scale tile: 32 rows of 16 bytes, no swizzle (groups of eight rows 128 bytes apart)
__device__ __forceinline__ unsigned long long desc_scales(uint32_t saddr) {
    return (unsigned long long)((saddr >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
}
// instruction descriptor of the block-scaled kinds: both operands of element format F, K-major, E8M0 scales
template <int F> __host__ __device__ constexpr uint32_t idesc_block_scaled(int m, int n) {
    const uint32_t fmt = F == F_E2M1 ? 1u : 0u;  // mxf4: E2M1 = 1; mxf8f6f4: E4M3 = 0
    return (fmt << 7) | (fmt << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 4) << 24);
}

// ---- instructions (one thread issues) -------------------------------------------------------

// scale tile -> four tensor-memory columns: row r of 128 at lane r % 32, column r / 32 (copied to all four
// lane groups), its four block scales in the column's four bytes
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, unsigned long long desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// D += A B^T with the scales of A's rows at tensor-memory column sfa and of B's rows at sfb
template <int F>
__device__ __forceinline__ void tc_mma_block_scaled(uint32_t d, unsigned long long a, unsigned long long b,
                                                    uint32_t idesc, uint32_t sfa, uint32_t sfb, bool accumulate) {
    if constexpr (F == F_E2M1)
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p; }" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
            : "memory");
}
// arrive on an mbarrier once everything this thread issued to the tensor core has completed
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- clusters -----------------------------------------------------------------------------

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// a float at this CTA's shared address `saddr`, read from the CTA of rank `rank`
__device__ __forceinline__ float ld_peer_f32(uint32_t saddr, uint32_t rank) {
    uint32_t p;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(p) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
    return v;
}

}  // namespace mxq
