// PTX building blocks of the 4-bit products, beside those shared by the tcgen05 kernels.
#pragma once

#include "q8_fp8_ptx.cuh"

namespace q8 {
namespace tc {

// Instruction descriptor of the block-scaled kinds with e2m1 A and B, both K-major, fp32 D: scales e4m3 for blocks of 16 K
// (scale_vec::4X), powers of two for blocks of 32 (2X). `id` picks the scale bytes within a 32-bit column of tensor memory: 0,
// or 2 for the upper two of 2X.
constexpr uint32_t idesc_fp4(int m, int n, int block, int id) {
    return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((block == 32 ? 1u : 0u) << 23) |
           ((uint32_t)(m >> 4) << 24) | ((uint32_t)id << 29);
}

// 64 K: D += (A scaled) (B scaled)^T. sa, sb: tensor memory of the scales, row r of 128 at lane r % 32, column r / 32.
template <int kBlock, int kGroup>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sa,
                                        uint32_t sb, uint32_t accumulate) {
    if constexpr (kBlock == 16 && kGroup == 1)
        asm volatile(
            "{\n.reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else if constexpr (kBlock == 16)
        asm volatile(
            "{\n.reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else if constexpr (kGroup == 1)
        asm volatile(
            "{\n.reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// Shared-memory descriptor of a tile of scales: 32 rows of 16 bytes, one after the other (eight-row groups 128 bytes apart).
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// A tile of scales (512 bytes: 32 rows of four columns) into tensor memory, to the lanes of all four warps. Ordered before the
// MMAs that the same thread issues after it. cta_group::2: from each CTA's own shared memory into its own tensor memory.
template <int kGroup>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (kGroup == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

}  // namespace tc
}  // namespace q8
