// mxfp4_tcgen05.cuh -- thin wrappers over the block-scaled 4-bit tensor-core
// instructions (tcgen05 kind::mxf4, one E8M0 scale per 32 k).
#pragma once

#include "q4_0_tcgen05.cuh"

namespace q4dev {

// Instruction descriptor of kind::mxf4: both operands E2M1 and K-major, E8M0
// scales, D of M x N in fp32.  sf: which byte pair of a scale column the MMA
// takes (0: the first two blocks of 128 k, 2: the last two), for both operands.
__host__ __device__ constexpr uint32_t mxf4_idesc(int M, int N, int sf) {
    return (uint32_t(sf) << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (1u << 23) |
           (uint32_t(M >> 4) << 24) | (uint32_t(sf) << 29);
}

// D[tmem] (+)= A[smem] * B[smem]^T over K = 64, scales in tensor memory.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// 512 scale bytes (128 rows x 4 blocks: 32 rows of 16 bytes) from shared
// memory to 4 tensor-memory columns, the same in each quarter of the lanes.
// Ordered before the MMAs that the same thread issues after it.
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Shared-memory descriptor of such 512 bytes: no swizzle, 8-row groups of 128 bytes.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem_byte_addr) {
    return ((uint64_t(smem_byte_addr) >> 4) & 0x3FFFull) | (1ull << 16) | (uint64_t(128 >> 4) << 32) | (1ull << 46);
}

// The same for a pair of CTAs (cta_group::2).  One thread of the first CTA
// issues: each CTA gives 128 rows of A (and the accumulator of those rows),
// half the rows of B and, for its own accumulator, the scales of its A rows
// and of all rows of B; the copy takes each CTA's scales from its own shared
// to its own tensor memory.
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tc_cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrives on the barrier at the same place in both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Arrives on the issuing CTA's barrier only.
__device__ __forceinline__ void tc_commit_pair_own(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// TMA load of a box of whole 1 KB rows from row y on, into this CTA's shared
// memory; `bar` is a shared::cluster address and may lie in the pair's other CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

}  // namespace q4dev
