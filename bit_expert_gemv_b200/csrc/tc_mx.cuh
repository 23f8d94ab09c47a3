// tcgen05 helpers of the microscaled product: block-scaled MMA, scale copies
// into TMEM, cluster barrier and distributed shared memory.
//
// The issuing functions are called by a whole warp and predicated on `lead`,
// true in one lane (elect_one): the warp stays converged, and the compiler keeps
// descriptors and addresses in uniform registers, where these instructions take
// their operands.  Behind a branch on the lane every operand was moved there
// first, about 40 cycles per instruction.
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
__device__ __forceinline__ void umma_mx(bool lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate),
          "r"(uint32_t(lead))
        : "memory");
}

// The same over a pair of CTAs: M = 256 (128 rows of either CTA), each CTA's
// shared memory holding half of B's N rows; issued by the pair's first CTA.
__device__ __forceinline__ void umma_mx_pair(bool lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate),
          "r"(uint32_t(lead))
        : "memory");
}
// Arrive on the barrier at this address in both CTAs of the pair once every
// MMA issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(bool lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        ::"r"(smem_u32(bar)), "h"(uint16_t(3)), "r"(uint32_t(lead))
        : "memory");
}
// The same for one CTA's own MMAs.
__device__ __forceinline__ void umma_commit_one(bool lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(uint32_t(lead))
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_copy_scales_pair(bool lead, uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc), "r"(uint32_t(lead))
        : "memory");
}
// The cluster's address of what CTA `rank` has at this shared-memory address.
__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    return remote;
}
// Arrive on the barrier at this address in CTA `rank` of the cluster, with release.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar, uint32_t rank) {
    const uint32_t remote = cluster_address(bar, rank);
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
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
__device__ __forceinline__ void tmem_copy_scales(bool lead, uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc), "r"(uint32_t(lead))
        : "memory");
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// One try of an mbarrier phase; CLUSTER: with acquire at cluster scope (an
// arrival may come from the pair's other CTA).
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}

// Bounded wait of a whole warp on an mbarrier phase, by the SM's cycle counter
// (about 2 s); false in every lane if it runs out in one.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity) {
    bool ok = mbar_try<CLUSTER>(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const long long t0 = clock64();
        while (!ok && clock64() - t0 < 4000000000ll) ok = mbar_try<CLUSTER>(bar, parity);
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// 2-D tiled TMA load into this CTA's shared memory that completes on a barrier of
// the pair's first CTA (`bar`: its cluster address; no multicast).
__device__ __forceinline__ void tma_load_2d_pair(bool lead, uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                                 int c1) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];\n\t}"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar), "r"(uint32_t(lead))
        : "memory");
}

// 2-D tiled TMA load into shared memory, completing on `bar` (no multicast).
__device__ __forceinline__ void tma_load_2d(bool lead, uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar), "r"(uint32_t(lead))
        : "memory");
}
__device__ __forceinline__ void bulk_load_lead(bool lead, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "r"(uint32_t(lead))
        : "memory");
}
__device__ __forceinline__ void mbar_expect_lead(bool lead, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(uint32_t(lead))
        : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same without ordering memory: only to keep a CTA alive until its peers have
// read its shared memory (the values they read have been used by then).
__device__ __forceinline__ void cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Four floats at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
    const uint32_t remote = cluster_address(addr, rank);
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

// 16 consecutive fp32 columns of this warp's 32 TMEM lanes, complete after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

}  // namespace gale
