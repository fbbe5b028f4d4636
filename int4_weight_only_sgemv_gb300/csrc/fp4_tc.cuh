// The tensor cores' instructions for block-scaled 4-bit operands.
#pragma once

#include "fp4_common.cuh"
#include "tcgen05.cuh"

namespace sgemv {

// Operand descriptor without swizzling: 128-byte groups of 8 rows of 16 bytes, `next` bytes from one 16-byte column to the next.
__device__ __forceinline__ uint64_t tc_desc_plain(uint32_t addr, uint32_t next) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(next >> 4) << 16) | (8ull << 32) | (1ull << 46);
}
// m x n x 64 of e2m1 operands, both with the inner axis contiguous, 32-bit sums; scales e4m3 (block 16) or powers of two (block 32), which
// of a column's four: id (0, or for block 32 also 2).
template <int kBlock>
__host__ __device__ constexpr uint32_t tc_idesc_fp4(int m, int n, int id) {
    return (static_cast<uint32_t>(id) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n / 8) << 17) |
           ((kBlock == 32 ? 1u : 0u) << 23) | (static_cast<uint32_t>(m / 16) << 24) | (static_cast<uint32_t>(id) << 29);
}
// 512 bytes of scales (128 rows, 4 scales each) into 4 columns of tensor memory.
template <int kPair>
__device__ __forceinline__ void tc_copy_scales(uint32_t to, uint64_t desc) {
    if constexpr (kPair == 1) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(desc) : "memory");
}
// d += a b (or d = a b); scales in tensor memory. kPair CTAs work on it together.
template <int kBlock, int kPair>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add) {
#define SGEMV_MMA_FP4(group, kind)                                                                                                  \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"                                                                  \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a), "l"(b), \
                 "r"(idesc), "r"(sa), "r"(sb), "r"(add ? 1u : 0u)                                                                   \
                 : "memory")
    if constexpr (kPair == 1) {
        if constexpr (kBlock == 16) SGEMV_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
        else SGEMV_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
    } else {
        if constexpr (kBlock == 16) SGEMV_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else SGEMV_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
    }
#undef SGEMV_MMA_FP4
}

// A sum times the scales of its two rows (powers of two, whose product may leave binary32 where the result does not; NaN for a row
// that held no number).
__device__ __forceinline__ float row_scaled(float sum, float a, float b) {
    const float f = a * b;
    if (f >= 1.17549435e-38f && f < INFINITY) return sum * f;
    if (!(f == f)) return f;
    return ldexpf(sum, static_cast<int>(__float_as_uint(a) >> 23) + static_cast<int>(__float_as_uint(b) >> 23) - 254);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// Without waiting for this thread's memory operations (prefetches among them): for barriers, whose initialisation has a fence of its own.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {  // the same place in another CTA's shared memory
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

struct ProductParams {
    Fp4Matrix w, x;
    void* y;
    int64_t stride;
    int32_t* status;
    int x_tiles, k_stages;
    int split, ring;  // fp4_few_kernel: CTAs a tile; stages of the ring
    int tiles_w, tiles_x;  // fp4_many_kernel
};

}  // namespace sgemv
