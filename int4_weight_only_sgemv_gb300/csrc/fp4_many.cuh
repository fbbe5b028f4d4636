// The product of two 4-bit matrices: the kernel of calls with many tiles.
//
// Bound by the products' rate, and by what feeds them: a CTA that computes 128 x 128 outputs reads 36 KB for 256 columns, 256 cycles of the tensor
// cores, and an SM takes in about 50 bytes a cycle. So two SMs share a tile of 256 tokens x 256 weight rows (cta_group::2): each holds the
// codes of 128 tokens and of 128 weight rows, and its tensor memory the sums of its 128 tokens; 38 KB for 512 cycles.
// One CTA an SM goes through tiles, tokens fastest within groups of 8 token tiles, so that what the SMs read at a time stays in L2. Roles:
//   warps 0-3   issue the copies of its SM's half, one each a stage (a copy takes 200 cycles to issue: five by one warp took 1270 a stage); what
//               lands in either is counted on the first one's barriers
//   warps 4-11  take the sums out, two threads a token, and write them
//   warp 12     of the first CTA issues the products of both
// Tensor memory: two sets of sums, columns 0..255 and 208..463, and the scales in the last 48. The columns that the sets share are taken out
// first, and then the next tile's products start while the rest is written. Where tiles are fewer than pairs of SMs they are half as wide (kN = 128).
#pragma once

#include <cuda.h>

#include "fp4_tc.cuh"

namespace sgemv {

template <int kBlock, int kN>
struct ManyShape {
    static constexpr int kStageK = 256, kChunks = kStageK / 32, kGroups = kStageK / (4 * kBlock);
    static constexpr int kCodes = 128 * kStageK / 2, kScales = kGroups * 512;      // of 128 tokens
    static constexpr int kWCodes = kN / 2 * kStageK / 2, kWScales = kN / 128 * kScales;  // of kN / 2 weight rows; of kN
    static constexpr int kStage = kCodes + kWCodes + kScales + kWScales;
    static constexpr int kRing = kN == 256 ? 5 : 6, kThreads = 416;
    static constexpr int kSmem = kRing * kStage + 8 * 4096;  // and 32 rows of 64 outputs a warp
    static constexpr int kSecond = kN == 256 ? 208 : 128;    // columns
    static constexpr int kScaleCols = kSecond + kN;
    static constexpr int kParts = kN / 64;
    static_assert(kScaleCols + (4 + kN / 32) * kGroups <= 512 && kSmem <= 227 * 1024, "tensor memory and shared memory");
};
constexpr int kManyGroup = 8;  // token tiles

// A 4-bit matrix as tensors of 8-byte elements: codes [tile][chunk of 32 columns][2048 bytes], scales [tile][group][512 bytes] (the tokens' in boxes of
// one tile, the weights' of two).
struct Fp4Maps {
    CUtensorMap codes, scales;
};
// A box of a tensor into this CTA's shared memory, counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_addr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tc_alloc_pair(uint32_t* smem_slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// On the barrier at this place in both CTAs, once the products issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "h"(static_cast<unsigned short>(3))
                 : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {  // in any CTA of the cluster
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits for arrivals from the other CTA too.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return done != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((i & 63u) == 0 && global_ns() - t0 > kMbarWaitNs) return false;
    }
}

template <typename T, int kBlock, int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(ManyShape<kBlock, kN>::kThreads, 1) fp4_many_kernel(const __grid_constant__ Fp4Maps x_maps, const __grid_constant__ Fp4Maps w_maps, const __grid_constant__ ProductParams p) {
    using S = ManyShape<kBlock, kN>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[S::kRing], free_[S::kRing], sums_full, sums_free, other_ready;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) float s_w_scale[kN];
    __shared__ float s_least[8], s_most[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int rank = blockIdx.x & 1, me_pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int chunks = p.w.kp / 32, tiles = p.tiles_x * p.tiles_w;
    if (tid == 0) {
        for (int i = 0; i < S::kRing; ++i) mbar_init(&full[i], 1), mbar_init(&free_[i], 1);
        mbar_init(&sums_full, 1), mbar_init(&sums_free, 8), mbar_init(&other_ready, 1);
        mbar_fence_init();
    }
    pdl_launch_dependents();
    __syncthreads();
    cluster_arrive_relaxed();
    cluster_wait();
    pdl_wait();
    bool dead = false;  // a wait gave up: nothing is waited for any more, and what comes out is reported as invalid
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || mbar_wait(bar, parity)) return;
        dead = true;
        report(p.status, SGEMV_ERR_TIMEOUT);
    };
    const auto tile_at = [&](int tile, int& xt, int& wt) {
        const int per = kManyGroup * p.tiles_w, group = tile / per, in = tile % per;
        const int width = min(kManyGroup, p.tiles_x - group * kManyGroup);
        xt = group * kManyGroup + in % width, wt = in / width;
    };

    if (warp < 4) {
        const uint32_t first_full = peer_addr(full, 0);
        int g = 0;
#pragma unroll 1
        for (int tile = me_pair; tile < tiles && !dead; tile += pairs) {
            int xt, wt;
            tile_at(tile, xt, wt);
#pragma unroll 1
            for (int i = 0; i < p.k_stages; ++i, ++g) {
                const int b = g % S::kRing;
                if (g >= S::kRing) wait(&free_[b], (g / S::kRing - 1) & 1);
                dead = __any_sync(0xFFFFFFFFu, dead);
                if (dead) break;
                // (whole boxes, zeros where the matrices end)
                if (elect_one()) {
                    uint8_t* const to = smem + b * S::kStage;
                    const uint32_t bar = first_full + 8 * b;
                    if (warp == 0) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[b], 2 * S::kStage);
                        tma_load_pair(to, &x_maps.codes, 0, S::kChunks * i, 2 * xt + rank, bar);
                    } else if (warp == 1) {
                        if constexpr (kN == 256) tma_load_pair(to + S::kCodes, &w_maps.codes, 0, S::kChunks * i, 2 * wt + rank, bar);
                        else tma_load_pair(to + S::kCodes, &w_maps.codes, 128 * rank, S::kChunks * i, wt, bar);
                    } else if (warp == 2) {
                        tma_load_pair(to + S::kCodes + S::kWCodes, &x_maps.scales, 0, S::kGroups * i, 2 * xt + rank, bar);
                    } else {
                        tma_load_pair(to + S::kCodes + S::kWCodes + S::kScales, &w_maps.scales, 0, S::kGroups * i, kN / 128 * wt, bar);
                    }
                }
                __syncwarp();
            }
        }
        // (all have landed, unless someone gave up: the first CTA sees it, and the second leaves after it)
        if (warp == 0 && rank == 0)
            for (int i = max(0, g - S::kRing); i < g; ++i) mbar_wait(&full[i % S::kRing], (i / S::kRing) & 1);
    } else if (warp == 12) {
        // Tensor memory only once the kernels before this one have ended: who held some while waiting for them could keep it from one of their CTAs.
        tc_alloc_pair(&s_tmem, 512);
        tc_before_sync();
        named_bar_sync(2, 288);
        if (rank == 1 && lane == 0) arrive_at(peer_addr(&other_ready, 0));
        const uint32_t tmem = s_tmem;
        int g = 0, turn = 0;
        if (rank == 0) {
            if (!mbar_wait_cluster(&other_ready, 0)) {
                dead = true;
                report(p.status, SGEMV_ERR_TIMEOUT);
            }
            dead = __any_sync(0xFFFFFFFFu, dead);
            tc_after_sync();
            const uint32_t base = __shfl_sync(0xFFFFFFFFu, smem_addr(smem), 0), t_sa = tmem + S::kScaleCols, t_sb = t_sa + 4 * S::kGroups;
            constexpr uint32_t idesc = tc_idesc_fp4<kBlock>(256, kN, 0);
            constexpr int kWCols = kN / 32;  // of scales, 64 or 128 columns of k
#pragma unroll 1
            for (int tile = me_pair; tile < tiles; tile += pairs, ++turn) {
                if (turn > 0 && !dead && !mbar_wait_cluster(&sums_free, (turn - 1) & 1)) {
                    dead = true;
                    report(p.status, SGEMV_ERR_TIMEOUT);
                }
                const uint32_t d = tmem + ((turn & 1) ? S::kSecond : 0);
#pragma unroll 1
                for (int i = 0; i < p.k_stages; ++i, ++g) {
                    const int b = g % S::kRing;
                    wait(&full[b], (g / S::kRing) & 1);
                    dead = __any_sync(0xFFFFFFFFu, dead);
                    tc_after_sync();
                    const int steps = min(S::kStageK / 64, chunks / 2 - S::kStageK / 64 * i), n = min(S::kGroups, p.w.groups - S::kGroups * i);
                    const uint32_t at = base + b * S::kStage;
                    if (elect_one()) {
                        if (!dead) {
                            const uint64_t sd = tc_desc_plain(at + S::kCodes + S::kWCodes, 0);
#pragma unroll
                            for (int j = 0; j < S::kGroups; ++j) {
                                if (j < n) {
                                    tc_copy_scales<2>(t_sa + 4 * j, sd + 32 * j);
#pragma unroll
                                    for (int h = 0; h < kN / 128; ++h) tc_copy_scales<2>(t_sb + kWCols * j + 4 * h, sd + 32 * (j + (1 + h) * S::kGroups));
                                }
                            }
                            const uint64_t xd = tc_desc_plain(at, 2048), wd = tc_desc_plain(at + S::kCodes, kN / 2 * 16);
#pragma unroll
                            for (int j = 0; j < S::kStageK / 64; ++j) {
                                const uint32_t col = kBlock == 16 ? j : j / 2, id = kBlock == 16 ? 0 : 2 * (j & 1);
                                if (j < steps)
                                    tc_mma_fp4<kBlock, 2>(d, xd + j * 256, wd + j * kN, idesc | (id << 4) | (id << 29), t_sa + 4 * col, t_sb + kWCols * col,
                                                          i > 0 || j > 0);
                            }
                        }
                        tc_commit_pair(&free_[b]);
                        if (i == p.k_stages - 1) tc_commit_pair(&sums_full);
                    }
                    __syncwarp();
                }
            }
        }
        // the last products: none may be under way when the CTA's memory goes
        for (int i = max(0, g - S::kRing); i < g; ++i) mbar_wait(&free_[i % S::kRing], (i / S::kRing) & 1);
    } else {
        const int me = tid - 128, row = 32 * (warp & 3) + lane, half = (warp - 4) >> 2;
        named_bar_sync(2, 288);
        tc_after_sync();
        const uint32_t tmem = s_tmem;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16, told = peer_addr(&sums_free, 0);
        const bool vec = p.stride % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
        int turn = 0;
#pragma unroll 1
        for (int tile = me_pair; tile < tiles; tile += pairs, ++turn) {
            int xt, wt;
            tile_at(tile, xt, wt);
            const int token = xt * 256 + rank * 128 + row, n0 = wt * kN;
            // the scales of the rows, and whether any product of two leaves binary32's normal range
            const float xs = token < p.x.rows ? p.x.row_scale[token] : 1.0f;
            float least, most;
            {
                const float f = me < kN && n0 + me < p.w.rows ? p.w.row_scale[n0 + me] : 1.0f;
                if (me < kN) s_w_scale[me] = f;
                least = f == f ? f : 0.0f, most = f;
            }
            const unsigned lo = __reduce_min_sync(0xFFFFFFFFu, __float_as_uint(least)), hi = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
            if (lane == 0) s_least[warp - 4] = __uint_as_float(lo), s_most[warp - 4] = __uint_as_float(hi);
            named_bar_sync(1, 256);
#pragma unroll
            for (int i = 0; i < 8; ++i) least = fminf(least, s_least[i]), most = fmaxf(most, s_most[i]);
            const bool plain = __all_sync(0xFFFFFFFFu, xs * least >= 1.17549435e-38f && xs * most < INFINITY);
            wait(&sums_full, turn & 1);
            __syncwarp();
            tc_after_sync();
            const uint32_t from = tmem + lanes + ((turn & 1) ? S::kSecond : 0);
            const int token0 = token - lane, rows = min(32, p.x.rows - token0);
            // 64 columns at a time, first those that the other set of sums shares, through shared memory, so that whole lines of rows are written
            uint8_t* const stage = smem + S::kRing * S::kStage + (warp - 4) * 4096;
#pragma unroll 1
            for (int k = 0; k < S::kParts / 2; ++k) {
                const int part = kN == 256 ? ((turn & 1) ? k : k + 3) + 2 * half & 3 : half, col = n0 + 64 * part;
                uint32_t r[2][32];
                tc_ld32(r[0], from + 64 * part);
                tc_ld32(r[1], from + 64 * part + 32);
                tc_wait_ld();
                if (k == 0 && half == 0) {
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_at(told);
                }
                if (col >= p.w.rows) continue;
                if (plain) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int n = 8 * i + 4 * e;
                            const float4 ws = *reinterpret_cast<const float4*>(&s_w_scale[64 * part + n]);
                            const uint32_t* const v = &r[n / 32][n % 32];
                            const float2 a = parts_of(mul2(pair(__uint_as_float(v[0]), __uint_as_float(v[1])), mul2(pair(xs, xs), pair(ws.x, ws.y))));
                            const float2 b = parts_of(mul2(pair(__uint_as_float(v[2]), __uint_as_float(v[3])), mul2(pair(xs, xs), pair(ws.z, ws.w))));
                            h[2 * e] = pack_two<T>(a.x, a.y), h[2 * e + 1] = pack_two<T>(b.x, b.y);
                        }
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ lane) & 7) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 64; ++n)
                        *reinterpret_cast<T*>(stage + lane * 128 + ((n / 8 ^ lane) & 7) * 16 + n % 8 * 2) =
                            from_f32<T>(row_scaled(__uint_as_float(r[n / 32][n % 32]), xs, s_w_scale[64 * part + n]));
                }
                __syncwarp();
                T* y = static_cast<T*>(p.y) + token0 * p.stride + col;
                const int cols = min(64, p.w.rows - col);
                if (vec && col + 64 <= p.w.rows) {
                    T* to = y + (lane >> 3) * p.stride + 8 * (lane & 7);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = 4 * i + (lane >> 3);
                        const uint4 h = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((lane ^ rr) & 7) * 16);
                        if (rr < rows) *reinterpret_cast<uint4*>(to) = h;
                        to += 4 * p.stride;
                    }
                } else {
#pragma unroll 4
                    for (int rr = 0; rr < rows; ++rr) {
                        const uint8_t* const line = stage + rr * 128;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int n = 32 * i + lane;
                            if (n < cols) y[rr * p.stride + n] = *reinterpret_cast<const T*>(line + ((n / 8 ^ rr) & 7) * 16 + n % 8 * 2);
                        }
                    }
                }
                __syncwarp();
            }
            named_bar_sync(1, 256);  // (the scales' place; and nobody is a tile behind)
        }
    }
    __syncwarp();
    tc_before_sync();
    cluster_arrive();
    cluster_wait();
    tc_after_sync();
    if (warp == 12) tc_dealloc_pair(s_tmem, 512);
}

}  // namespace sgemv
