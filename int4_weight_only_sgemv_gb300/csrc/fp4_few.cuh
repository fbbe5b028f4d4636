// The product of two 4-bit matrices: the kernel of calls with few tiles, down to one token.
//
// With few tokens the weights' bytes bound the work (0.56 bytes a weight against 2 operations a token), and with the tensor cores' block-
// scaled instruction nothing has to be unpacked: copies of contiguous bytes go from HBM to shared memory and are multiplied as they are.
// The weights are the instruction's 128 rows and the tokens its narrow side (8 to 128), so that one token costs no more than eight. A
// CTA has one tile of 128 weight rows, and where there are fewer tiles than places (two CTAs an SM), a cluster of up to 8 CTAs shares it: each
// sums a run of the columns, and they join their sums over distributed shared memory, in the order of the columns.
// Roles: warp 0 issues the copies, warp 1 the products, warps 2-5 take the sums out; all warps join and write.
#pragma once

#include "fp4_tc.cuh"

namespace sgemv {

constexpr int kFewThreads = 192;
constexpr int kFewSmem = 108 * 1024;  // of the ring: two CTAs an SM, and never three (their tensor memory, 256 columns each, is full)
constexpr int kFewCols = 256;
constexpr int kFewMaxRing = 8;

// Bytes of a stage: codes of 128 weight rows and of the tokens, scales of both.
__host__ __device__ inline int few_stage_bytes(int block, int x_tile) {
    return 128 * kStageK / 2 + x_tile * kStageK / 2 + 2 * (kStageK / (4 * block)) * 512;
}

__device__ __forceinline__ void cluster_arrive_wait() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_peer(uint32_t addr, uint32_t rank) {  // of the same place in another CTA's shared memory
    float4 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

template <typename T, int kBlock>
__global__ void __launch_bounds__(kFewThreads, 2) fp4_few_kernel(const ProductParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kFewMaxRing], free_[kFewMaxRing], done;
    __shared__ uint32_t s_tmem;
    constexpr int kGroups = kStageK / (4 * kBlock);  // of 4 scales, a stage
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
    const int wt = tile / p.x_tiles, xt = tile % p.x_tiles;
    const int st0 = static_cast<int>(static_cast<int64_t>(p.k_stages) * rank / p.split);
    const int n = static_cast<int>(static_cast<int64_t>(p.k_stages) * (rank + 1) / p.split) - st0;
    const uint32_t stage_bytes = few_stage_bytes(kBlock, p.x.tile);
    const int chunks = p.w.kp / 32;
    const uint8_t* const w_codes = p.w.codes + (static_cast<int64_t>(wt) * chunks + 8 * st0) * p.w.tile * 16;
    const uint8_t* const w_scales = p.w.scales + (static_cast<int64_t>(wt) * p.w.groups + kGroups * st0) * 512;
    const int cols = min(p.x.tile, p.x.rows - xt * 128);  // tokens of this tile
    const int rows = min(128, p.w.rows - wt * 128);

    if (tid == 0) {
        for (int i = 0; i < p.ring; ++i) mbar_init(&full[i], 1), mbar_init(&free_[i], 1);
        mbar_init(&done, 1);
        mbar_fence_init();
        // into L2 while the kernel before this one ends (nothing is read before it has)
        const int early = min(n, p.ring);
        const int many = min(8 * early, chunks - 8 * st0), groups = min(kGroups * early, p.w.groups - kGroups * st0);
        for (int b = 0; b < many * p.w.tile * 16; b += kPrefetchPiece) prefetch_l2(w_codes + b, min(static_cast<int>(kPrefetchPiece), many * p.w.tile * 16 - b));
        prefetch_l2(w_scales, groups * 512);
    }
    pdl_launch_dependents();
    if (warp == 1) tc_alloc(&s_tmem, kFewCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = s_tmem, t_sa = tmem + 128, t_sb = tmem + 128 + 4 * kGroups;
    pdl_wait();

    bool dead = false;  // a wait gave up: nothing is waited for any more, and what comes out is reported as invalid
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || mbar_wait(bar, parity)) return;
        dead = true;
        report(p.status, SGEMV_ERR_TIMEOUT);
    };
    // a stage: weights' codes, tokens' codes, weights' scales, tokens' scales
    const uint32_t at_x = 128 * kStageK / 2, at_sw = at_x + p.x.tile * kStageK / 2, at_sx = at_sw + kGroups * 512;
    if (warp == 0) {
        if (lane == 0) {
            const uint8_t* const x_codes = p.x.codes + (static_cast<int64_t>(xt) * chunks + 8 * st0) * p.x.tile * 16;
            const uint8_t* const x_scales = p.x.scales + (static_cast<int64_t>(xt) * p.x.groups + kGroups * st0) * 512;
            int i = 0;
            for (; i < n; ++i) {
                const int b = i % p.ring;
                if (i >= p.ring) wait(&free_[b], (i / p.ring - 1) & 1);
                if (dead) break;
                const int c = min(8, chunks - 8 * (st0 + i)), g = min(kGroups, p.w.groups - kGroups * (st0 + i));
                uint8_t* const to = smem + b * stage_bytes;
                mbar_arrive_expect_tx(&full[b], c * (p.w.tile + p.x.tile) * 16 + 2 * g * 512);
                bulk_g2s(to, w_codes + static_cast<int64_t>(i) * 8 * p.w.tile * 16, c * p.w.tile * 16, &full[b]);
                bulk_g2s(to + at_x, x_codes + static_cast<int64_t>(i) * 8 * p.x.tile * 16, c * p.x.tile * 16, &full[b]);
                bulk_g2s(to + at_sw, w_scales + static_cast<int64_t>(i) * kGroups * 512, g * 512, &full[b]);
                bulk_g2s(to + at_sx, x_scales + static_cast<int64_t>(i) * kGroups * 512, g * 512, &full[b]);
            }
            // (none may be under way when the CTA leaves; all have landed when the products are done, unless someone gave up)
            for (int j = max(0, i - p.ring); j < i; ++j) mbar_wait(&full[j % p.ring], (j / p.ring) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t base = smem_addr(smem);
        const uint32_t idesc = tc_idesc_fp4<kBlock>(128, (cols + 7) / 8 * 8, 0);
        int i = 0;
        for (; i < n; ++i) {
            const int b = i % p.ring;
            wait(&full[b], (i / p.ring) & 1);
            dead = __any_sync(0xFFFFFFFFu, dead);
            if (dead) break;
            tc_after_sync();
            const int steps = min(4, chunks / 2 - 4 * (st0 + i)), g = min(kGroups, p.w.groups - kGroups * (st0 + i));
            const uint32_t at = base + b * stage_bytes;
            if (elect_one()) {
                for (int j = 0; j < g; ++j) {
                    tc_copy_scales<1>(t_sa + 4 * j, tc_desc_plain(at + at_sw + 512 * j, 0));
                    tc_copy_scales<1>(t_sb + 4 * j, tc_desc_plain(at + at_sx + 512 * j, 0));
                }
                const uint64_t wd = tc_desc_plain(at, p.w.tile * 16), xd = tc_desc_plain(at + at_x, p.x.tile * 16);
                for (int j = 0; j < steps; ++j) {
                    const uint32_t col = kBlock == 16 ? 4 * j : 4 * (j / 2), id = kBlock == 16 ? 0 : 2 * (j & 1);
                    tc_mma_fp4<kBlock, 1>(tmem, wd + j * 2 * p.w.tile, xd + j * 2 * p.x.tile, idesc | (id << 4) | (id << 29), t_sa + col,
                                          t_sb + col, i > 0 || j > 0);
                }
                tc_commit(&free_[b]);
                if (i == n - 1) tc_commit(&done);
            }
            __syncwarp();
        }
        // the last products: none may be under way when the CTA's tensor memory goes
        for (int j = max(0, i - p.ring); j < i; ++j) mbar_wait(&free_[j % p.ring], (j / p.ring) & 1);
    } else {
        wait(&done, 0);
        __syncwarp();
        tc_after_sync();
        // sums [token][weight row] over the ring, which nobody needs any more
        float* const part = reinterpret_cast<float*>(smem);
        const int row = 32 * (warp & 3) + lane;
        for (int c = 0; c < cols; c += 8) {
            uint32_t r[8];
            tc_ld8(r, tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < cols) part[(c + j) * 128 + row] = __uint_as_float(r[j]);
        }
    }
    __syncwarp();
    tc_before_sync();
    if (p.split > 1) cluster_arrive_wait();
    else __syncthreads();
    tc_after_sync();
    // four weight rows of a token a thread
    const uint32_t part = smem_addr(smem);
    const int quads = (rows + 3) / 4, items = cols * 32;
    T* const y = static_cast<T*>(p.y) + static_cast<int64_t>(xt) * 128 * p.stride + wt * 128;
    const bool vec = p.stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 7) == 0;
    for (int item = items * rank / p.split + tid; item < items * (rank + 1) / p.split; item += kFewThreads) {
        const int t = item >> 5, q = item & 31;
        if (q >= quads) continue;
        float4 v;
        if (p.split == 1) {
            v = *reinterpret_cast<const float4*>(smem + item * 16);
        } else {
            v = ld_peer(part + item * 16, 0);
            for (int r = 1; r < p.split; ++r) {
                const float4 o = ld_peer(part + item * 16, r);
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
        }
        const float xs = p.x.row_scale[xt * 128 + t];
        const float4 ws = *reinterpret_cast<const float4*>(p.w.row_scale + wt * 128 + 4 * q);
        const float f[4] = {row_scaled(v.x, xs, ws.x), row_scaled(v.y, xs, ws.y), row_scaled(v.z, xs, ws.z), row_scaled(v.w, xs, ws.w)};
        T* const to = y + t * p.stride + 4 * q;
        if (vec && 4 * q + 4 <= rows) {
            *reinterpret_cast<uint2*>(to) = make_uint2(pack_two<T>(f[0], f[1]), pack_two<T>(f[2], f[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * q + j < rows) to[j] = from_f32<T>(f[j]);
        }
    }
    __syncwarp();
    if (p.split > 1) cluster_arrive_wait();  // (the others may still read this one's sums)
    if (warp == 1) tc_dealloc(tmem, kFewCols);
}

}  // namespace sgemv
