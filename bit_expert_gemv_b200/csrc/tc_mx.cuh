// tcgen05 helpers of the microscaled product: block-scaled MMA, scale copies
// into TMEM, cluster barrier and distributed shared memory.
#pragma once
#include "tc_prefill.cuh"

namespace gale {

// Instruction descriptor of kind::mxf8f6f4: A e2m1 (5), B e4m3 (0), scales
// ue8m0, fp32 accumulators, both operands K-major, M x N.  The scale byte used
// by one MMA (K = 32) is chosen by the two 2-bit ids.
__host__ __device__ constexpr uint32_t umma_idesc_mx(int M, int N) {
    return (5u << 7) | (0u << 10)          // A, B format
           | (uint32_t(N >> 3) << 17)      // N / 8
           | (1u << 23)                    // scale format ue8m0
           | (uint32_t(M >> 4) << 24);     // M / 16
}
__device__ __forceinline__ uint32_t umma_idesc_scale_id(uint32_t idesc, uint32_t id) {
    return idesc | id << 4 | id << 29;
}

// D[tmem] (+)= (A * 2^sfa) (B * 2^sfb)^T for one block of 32 columns.
__device__ __forceinline__ void umma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// A 512-byte scale atom (32 rows of 16 bytes, 8-row groups 128 bytes apart, no
// swizzle) as a copy source, and its copy to four TMEM columns, repeated over
// the four lane quarters.
__device__ __forceinline__ uint64_t scale_atom_desc(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
    d |= uint64_t(128u >> 4) << 32;     // stride byte offset (16 B units)
    d |= uint64_t(1u) << 46;            // version; layout type 0: no swizzle
    return d;
}
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 2-D tiled TMA load into shared memory, completing on `bar` (no multicast).
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

}  // namespace gale
