// The product of two 4-bit matrices: the kernel of calls with few tiles, down to one token.
//
// With few tokens the weights' bytes bound the work (0.56 bytes a weight against 2 operations a token), and with the tensor cores' block-
// scaled instruction nothing has to be unpacked: copies of contiguous bytes go from HBM to shared memory and are multiplied as they are.
// The weights are the instruction's 128 rows and the tokens its narrow side (8 to 128), so that one token costs no more than eight. A
// CTA has one tile of 128 weight rows, and where there are fewer tiles than places, a cluster of up to 8 CTAs shares it: each sums a run of the
// columns, and sends every other one its share of the outputs' sums over distributed shared memory, where they are joined in the order of
// the columns. (With sums read by their users between two barriers of the cluster, a call of one token took 1 us more.) What is sent has a
// place of its own where tiles are narrow; with 64 or 128 tokens it comes where the ring was, so that two CTAs fit an SM, after a barrier of the cluster.
// Roles: warps 0-3 issue the copies, one each a stage (90 ns a copy to issue, whoever's lane does, bound everything with one warp for all four);
// warps 4-7 take the sums out, send, join and write; warp 8 issues the products.
#pragma once

#include <algorithm>

#include "fp4_tc.cuh"

namespace sgemv {

constexpr int kFewThreads = 288;
// Of the ring and what is sent: two CTAs an SM. (With 108 KB, 17 to 32 tokens in blocks of 16 had one place where a tile is split by 5 or more, and copies waited
// for products: 20 x 4096 x 11008 10.5 us, 9.1 with two; 20 x 5120 x 8192 15.2, 13.0.)
constexpr int kFewSmem = 112 * 1024;
constexpr int kFewLeast = 80 * 1024;   // and never three, whose tensor memory (256 columns each) would not fit
constexpr int kFewMost = 216 * 1024;
constexpr int kFewCols = 256;
constexpr int kFewMaxRing = 8;

// Columns of a stage. A stage costs its copies (60 to 90 ns each), its barriers and commits (170 ns) whatever its size: one token, 11008 x 4096: 0.9 us
// less a call with 512 columns than with 256 (8.1 now). With 64 or 128 tokens a tile, two stages of 512 would not fit.
__host__ __device__ constexpr int few_stage_k(int x_tile) { return x_tile <= 32 ? 512 : 256; }
// Bytes of a stage: codes of 128 weight rows and of the tokens, scales of both.
__host__ __device__ constexpr int few_stage_bytes(int block, int x_tile) {
    const int k = few_stage_k(x_tile);
    return 128 * k / 2 + x_tile * k / 2 + 2 * (k / (4 * block)) * 512;
}
// Float4s of sums that a CTA of a cluster joins, and bytes of what the others send it.
__host__ __device__ inline int few_share(int x_tile, int split) { return (x_tile * 32 + split - 1) / split; }
__host__ __device__ inline int few_sent(int x_tile, int split) { return (split - 1) * few_share(x_tile, split) * 16; }

// Host: CTAs a tile, places of the ring, and bytes of shared memory, for a call of `tiles` tiles of `stages` stages.
struct FewPlan {
    int split, ring, smem;
};
inline FewPlan few_plan(int block, int x_tile, int64_t tiles, int stages, int sms) {
    FewPlan f;
    // As many as fill two places an SM, each with two stages at least (4096 x 4096, one token: 4 CTAs 5.2 us, 8 5.7). From 5 on, what
    // tiles of 128 tokens are sent leaves one place an SM, and not every SM is in a cluster (512 x 512 x 8192: 6 CTAs 10.5 us, 8 16.9).
    f.split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, 2 * sms / tiles, stages / 2})));
    if (x_tile == 128 && f.split > 4) f.split = std::min(f.split, std::max(4, static_cast<int>(2 * sms / 3 / tiles)));
    const int stage = few_stage_bytes(block, x_tile), sent = f.split > 1 ? few_sent(x_tile, f.split) : 0;
    const bool early = few_stage_k(x_tile) == 512;
    f.ring = std::min({kFewMaxRing, (kFewSmem - (early ? sent : 0)) / stage, (stages + f.split - 1) / f.split});
    // (the sums of a tile take the ring's place, and in wide tiles what is sent too)
    f.smem = std::max(early ? std::max(f.ring * stage, x_tile * 512) + sent : std::max(f.ring * stage, x_tile * 512 + sent), kFewLeast);
    return f;
}

// 16 bytes into a peer's shared memory, counted on its barrier.
__device__ __forceinline__ void send16(uint32_t to, float4 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}

template <typename T, int kBlock, int kStageK>
__global__ void __launch_bounds__(kFewThreads, 2) fp4_few_kernel(const ProductParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kFewMaxRing], free_[kFewMaxRing], done, sent;
    __shared__ uint32_t s_tmem;
    __shared__ float s_x_scale[128];
    constexpr int kGroups = kStageK / (4 * kBlock);  // of 4 scales, a stage
    constexpr int kChunks = kStageK / 32;            // of 16 bytes of codes
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
    const int wt = tile / p.x_tiles, xt = tile % p.x_tiles;
    const int st0 = static_cast<int>(static_cast<int64_t>(p.k_stages) * rank / p.split);
    const int n = static_cast<int>(static_cast<int64_t>(p.k_stages) * (rank + 1) / p.split) - st0;
    const uint32_t stage_bytes = few_stage_bytes(kBlock, p.x.tile);
    const int chunks = p.w.kp / 32;
    const uint8_t* const w_codes = p.w.codes + (static_cast<int64_t>(wt) * chunks + kChunks * st0) * p.w.tile * 16;
    const uint8_t* const w_scales = p.w.scales + (static_cast<int64_t>(wt) * p.w.groups + kGroups * st0) * 512;
    const int cols = min(p.x.tile, p.x.rows - xt * 128);  // tokens of this tile
    const int rows = min(128, p.w.rows - wt * 128);
    // Sums go by four weight rows of a token (32 a token); this CTA joins [item0, item1) of them, at most `share`, and gets the others' behind its own.
    const int share = few_share(p.x.tile, p.split), items = cols * 32;
    const int item0 = min(items, share * rank), item1 = min(items, share * (rank + 1));
    constexpr bool kEarly = kStageK == 512;  // what is sent has a place of its own
    float4* const got = reinterpret_cast<float4*>(smem + max(kEarly ? p.ring * stage_bytes : 0u, p.x.tile * 512u));

    if (tid == 0) {
        for (int i = 0; i < p.ring; ++i) mbar_init(&full[i], 1), mbar_init(&free_[i], 1);
        mbar_init(&done, 1), mbar_init(&sent, 1);
        mbar_fence_init();
        // into L2 while the kernel before this one ends (nothing is read before it has)
        const int early = min(n, p.ring);
        const int many = min(kChunks * early, chunks - kChunks * st0), groups = min(kGroups * early, p.w.groups - kGroups * st0);
        for (int b = 0; b < many * p.w.tile * 16; b += kPrefetchPiece) prefetch_l2(w_codes + b, min(static_cast<int>(kPrefetchPiece), many * p.w.tile * 16 - b));
        prefetch_l2(w_scales, groups * 512);
        if (p.split > 1) mbar_arrive_expect_tx(&sent, (p.split - 1) * (item1 - item0) * 16);
    }
    __syncthreads();
    if (kEarly && p.split > 1 && warp != 8) cluster_arrive_relaxed();  // (barriers are there; waited for before anything is sent)
    pdl_launch_dependents();
    pdl_wait();

    bool dead = false;  // a wait gave up: nothing is waited for any more, and what comes out is reported as invalid
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || mbar_wait(bar, parity)) return;
        dead = true;
        report(p.status, SGEMV_ERR_TIMEOUT);
    };
    // a stage: weights' codes, tokens' codes, weights' scales, tokens' scales
    const uint32_t at_x = 128 * kStageK / 2, at_sw = at_x + p.x.tile * kStageK / 2, at_sx = at_sw + kGroups * 512;
    if (warp < 4) {
        // this warp's copy of a stage: weights' codes, tokens' codes, weights' scales, tokens' scales
        const int64_t x_chunk = static_cast<int64_t>(xt) * chunks + kChunks * st0, x_group = static_cast<int64_t>(xt) * p.x.groups + kGroups * st0;
        const uint8_t* const from = warp == 0 ? w_codes : warp == 1 ? p.x.codes + x_chunk * p.x.tile * 16 : warp == 2 ? w_scales : p.x.scales + x_group * 512;
        const uint32_t unit = warp == 0 ? p.w.tile * 16 : warp == 1 ? p.x.tile * 16 : 512;  // bytes of a chunk or group
        const uint32_t to = warp == 0 ? 0 : warp == 1 ? at_x : warp == 2 ? at_sw : at_sx;
        int i = 0;
        for (; i < n; ++i) {
            const int b = i % p.ring;
            if (i >= p.ring) wait(&free_[b], (i / p.ring - 1) & 1);
            dead = __any_sync(0xFFFFFFFFu, dead);
            if (dead) break;
            const int c = min(kChunks, chunks - kChunks * (st0 + i)), g = min(kGroups, p.w.groups - kGroups * (st0 + i));
            if (lane == 0) {
                if (warp == 0) mbar_arrive_expect_tx(&full[b], c * (p.w.tile + p.x.tile) * 16 + 2 * g * 512);
                bulk_g2s(smem + b * stage_bytes + to, from + static_cast<int64_t>(i) * (warp < 2 ? kChunks : kGroups) * unit, (warp < 2 ? c : g) * unit, &full[b]);
            }
            __syncwarp();
        }
        // (none may be under way when the CTA leaves; all have landed when the products are done, unless someone gave up)
        for (int j = max(0, i - p.ring); j < i; ++j) mbar_wait(&full[j % p.ring], (j / p.ring) & 1);
        __syncwarp();
        if (p.split > 1) {
            if (!kEarly) cluster_arrive();
            cluster_wait();
            cluster_arrive_relaxed();
        }
    } else if (warp == 8) {
        // Tensor memory only once the kernels before this one have ended: who held some while waiting for them could keep it from one of their CTAs
        // (what this costs where calls follow one another: 0.8 to 1.7 us).
        tc_alloc(&s_tmem, kFewCols);
        __syncwarp();
        if (kEarly && p.split > 1) cluster_arrive_relaxed();
        tc_before_sync();
        named_bar_sync(2, 160);
        tc_after_sync();
        const uint32_t tmem = s_tmem, t_sa = tmem + 128, t_sb = tmem + 128 + 4 * kGroups;
        const uint32_t base = smem_addr(smem);
        const uint32_t idesc = tc_idesc_fp4<kBlock>(128, (cols + 7) / 8 * 8, 0);
        int i = 0;
        for (; i < n; ++i) {
            const int b = i % p.ring;
            wait(&full[b], (i / p.ring) & 1);
            dead = __any_sync(0xFFFFFFFFu, dead);
            if (dead) break;
            tc_after_sync();
            const int steps = min(kStageK / 64, chunks / 2 - kStageK / 64 * (st0 + i)), g = min(kGroups, p.w.groups - kGroups * (st0 + i));
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
        __syncwarp();
        if (p.split > 1) {
            if (!kEarly) cluster_arrive();
            cluster_wait();
            cluster_arrive_relaxed();
        }
    } else {
        const int me = tid - 128;  // of 128
        // the scales of rows and tokens, while the products run
        const int item_first = item0 + me, q = item_first & 31;  // (the same four rows for all of them)
        const float4 ws = *reinterpret_cast<const float4*>(p.w.row_scale + wt * 128 + 4 * q);
        if (me < cols) s_x_scale[me] = p.x.row_scale[xt * 128 + me];
        __syncwarp();
        named_bar_sync(2, 160);
        tc_after_sync();
        const uint32_t tmem = s_tmem;
        wait(&done, 0);
        __syncwarp();
        tc_after_sync();
        if (!kEarly && p.split > 1) cluster_arrive();
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
        __syncwarp();
        named_bar_sync(1, 128);
        const float4* const sums = reinterpret_cast<const float4*>(smem);
        if (p.split > 1) {
            cluster_wait();
            for (int d = 1; d < p.split; ++d) {
                const int to = rank + d < p.split ? rank + d : rank + d - p.split;  // (not all to the same one at a time)
                const int from0 = min(items, share * to), from1 = min(items, share * (to + 1));
                const uint32_t place = peer_addr(got + share * (rank < to ? rank : rank - 1), to), bar = peer_addr(&sent, to);
                for (int item = from0 + me; item < from1; item += 128) send16(place + (item - from0) * 16, sums[item], bar);
            }
            __syncwarp();
            cluster_arrive_relaxed();  // (this thread sends nothing any more)
            wait(&sent, 0);
        }
        // four weight rows of a token a thread
        const int quads = (rows + 3) / 4;
        T* const y = static_cast<T*>(p.y) + static_cast<int64_t>(xt) * 128 * p.stride + wt * 128;
        const bool vec = p.stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 7) == 0;
        for (int item = item_first; item < item1; item += 128) {
            const int t = item >> 5;
            if (q >= quads) break;
            const float xs = s_x_scale[t];
            float4 v = rank == 0 ? sums[item] : got[item - item0];
            for (int r = 1; r < p.split; ++r) {
                const float4 o = r == rank ? sums[item] : got[share * (r < rank ? r : r - 1) + item - item0];
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
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
    }
    __syncwarp();
    if (p.split > 1) {
        // Who gave up waiting for sums does not leave while they may still be sent: not before all have issued theirs, and these have landed. (0 to 0.2 us a
        // call, as far as this cluster's CTAs are apart.)
        cluster_wait();
        if (dead && warp >= 4 && warp < 8) mbar_wait(&sent, 0);
        __syncwarp();
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 8) tc_dealloc(s_tmem, kFewCols);
}

}  // namespace sgemv
