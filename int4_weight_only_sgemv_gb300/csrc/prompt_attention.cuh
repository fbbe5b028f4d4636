// Causal attention over packed prompts: softmax(scale q K^T) V of each request's own tokens, unquantised keys and values.
//
// Bound by the products, 4 D operations a (row, key), where prompts are long. Both go to the 5th-generation tensor cores with 128 x 128 x 16 and 128
// x D x 16 instructions. A row is a (token, query head) of one KV head, token after token, so that grouped heads share the keys they read and
// a tile's rows see about the same keys. A segment is two 128-row tiles against the same 128-key tiles: while one is in its softmax the
// other's products run. Each SM has one CTA, which goes through segments, the longest first; its roles run ahead of one another from one segment into
// the next, so that the start of a segment (queries, first keys, first scores) hides under the end of the one before. Roles, by warp:
//   0-3, 4-7  softmax of the first and of the second row tile: a thread a row, scores from tensor memory, weights back over them; the outputs
//   8, 9      issue the products, a row tile each
//   10        finds the segments and issues the copies of their queries and K and V tiles (two buffers each)
//   11        looks through V tiles that are masked for some row (below)
// The softmax's reference m moves only when a tile's sum of weights passes a limit (and in a row's first tile), so that the largest score is
// looked for in few tiles and the output's sums are rarely rescaled.
//
// Roundings: scores are sums of exact products in 32 bits, scaled in 32 bits. Weights 2^(t - m) are rounded to the type of V, since the
// instruction takes one type for both (11 bits for fp16, 8 for bf16).
//
// What a row does not see must not enter its sums whatever it holds, but 0 * NaN is NaN in the tensor cores. Scores are selected, so K needs
// nothing. V tiles that some row does not see in full are looked through (one product with 0 a word); elements that are no numbers are taken
// out and remembered, and if there were any, the rows that see them get them at their end.
//
// What bounds it now: with heads of 128 a key tile takes some 2950 cycles for both row tiles, of which the tensor cores need 2560 (64 a product
// of P and V, 96 of Q and K, which reads 8 KB of shared memory) and a row tile's chain (softmax 1030, its hand-over 360, products and their latency
// 1460) is as long. One prompt of 16384 tokens, 8 KV and 32 query heads of 128: 1362 to 1440 us, 1530 to 1610 TFLOP/s. With heads of 64 it is the chain
// of a row tile alone: 1970 cycles a tile, with the tensor cores, the exponentials' pipe (1024) and the issue slots at half each (72 us for 4096 tokens of
// the same heads). A segment costs 4500 cycles beside its tiles: 16 prompts of up to 2048 tokens take 185 to 200 us, 1070 to 1150 TFLOP/s.
#pragma once

#include <cuda.h>

#include "fp4_common.cuh"
#include "tcgen05.cuh"

namespace sgemv {

struct PromptParams {
    sgemv_prompt_query q;
    int32_t* status;
    int ratio;      // query heads a KV head
    int sub;        // of them, in a row tile: the largest divisor of ratio up to 128
    int tokens;     // of a row tile: 128 / sub
    int out32;      // rows of out start at multiples of 32 bytes
    int groups;     // heads * ratio / sub: KV heads, each as often as it has groups of `sub` query heads
    int most;       // segments that requests in order can have
    float scale_log2;
    float unscale;  // scale / scale_log2: ln 2, and what scale_log2 was rounded by
};

template <int D>
struct PromptShape {
    static constexpr int kTile = 128, kKeys = 128;
    static constexpr int kAtoms = D / 64;  // 128-byte columns of a row
    static constexpr int kBufs = 2;        // of K and of V (the product warps count on two)
    static constexpr int kSegs = 4;        // segments known ahead
    static constexpr int kQBytes = kTile * D * 2, kKvBytes = kKeys * D * 2;
    static constexpr int kWarps = 12, kThreads = 32 * kWarps;
    // Registers a thread at launch, and after the split: the softmax's 8 warps, whose rows' 128 scores stay in them, and 4.
    static constexpr int kRegs = 168, kRegsSoftmax = 200, kRegsOther = 104;
    static_assert(8 * kRegsSoftmax + 4 * kRegsOther == kWarps * kRegs, "the split of the launch's registers");
    static constexpr int kSmem = 1024 + 2 * kQBytes + 2 * kBufs * kKvBytes;
    // Tensor memory: O of both row tiles, and S, 128 columns a tile. With heads of 64 there is room for a third S: a row tile's next scores are then
    // formed before its weights are taken, so that they are there when its softmax is done with the last ones.
    static constexpr bool kAhead = D == 64;
    static constexpr int kCols = 512, kOCols = kAhead ? 384 : 256;
    // Columns of the scores of row tile x and the CTA's g-th key tile: the places go round in the order of the turns.
    static __device__ __forceinline__ uint32_t scores_at(int g, int x) { return 128u * (kAhead ? static_cast<uint32_t>(2 * g + x) % 3u : static_cast<uint32_t>(x)); }
};

// Weights 2^(t - m): the largest is 2^kTop when the reference m is set, which happens anew when a tile's sum passes kBig (or, where the largest score
// is looked for, when a weight would pass 2^kFar: 128 of those are that sum). fp16's weights end at 2^16 and have steps of 2^-24 below 2^-14: a row's
// largest being 2^kTop or more, each is held to 2^(-25 - kTop) of it, and n keys down there add up to n times that (for 2^16 keys as much as the rounding
// of the others). kTop is low enough that a window's first few keys rarely set a reference that the next tile moves. bf16 has 8 bits of exponent: sums of
// weights stay below 2^-23 a tile and, over the 2^23 tiles that a request can have, below 1, so that sums of V do not leave binary32 where V does not (with
// 2^-16 and 1 a tile, seven tiles of 2^127 did); V's elements below 2^-87 lose bits.
template <typename T>
struct PromptWeights {
    static constexpr float kTop = 2.0f, kBig = 32768.0f, kFar = 8.0f;
};
template <>
struct PromptWeights<__nv_bfloat16> {
    static constexpr float kTop = -39.0f, kBig = 1.1920928955078125e-7f, kFar = -30.0f;
};
constexpr float kPromptRound = 67108864.0f;  // past this, scores are rounded before the reference comes off

// A request's tokens.
struct PromptSpan {
    int first, n;
};
__device__ __forceinline__ PromptSpan prompt_span(const PromptParams& p, int r) {
    const int a = p.q.start_dev[r], b = p.q.start_dev[r + 1];
    const int n = p.q.length_dev != nullptr ? p.q.length_dev[r] : b - a;
    if (a < 0 || b < a || b > p.q.n_tokens || n < 0 || n > b - a) {
        report(p.status, SGEMV_ERR_ARG);
        return {0, 0};
    }
    return {a, n};
}
__device__ __forceinline__ int prompt_blocks(const PromptParams& p, int n) { return (n + 2 * p.tokens - 1) / (2 * p.tokens); }

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_addr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, int x, int y, int z) {  // into L2
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}
// Operand descriptor of V [key][64 dims] tiles as the instruction's transposed side: 128-byte swizzle, 8 keys every 1024 bytes, `next`
// bytes from 64 dims to the next 64.
__device__ __forceinline__ uint64_t tc_desc_v(uint32_t addr, uint32_t next) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(next >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
template <typename T>
__host__ __device__ constexpr uint32_t tc_idesc_type() {
    return std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
}

// A segment: a request's tokens from t0 on, as many as two row tiles hold, and `sub` query heads of one KV head.
struct PromptSegment {
    int first, n;   // the request's tokens; n < 0: no more segments
    int group, t0;
};
// Key tiles [from, to) that row tile x of a segment has; tiles in positions [clear0, clear1) are seen in full by all its rows.
struct PromptRange {
    int from, to, clear0, clear1;
};
__device__ __forceinline__ PromptRange prompt_range(const PromptParams& p, const PromptSegment& s, int x) {
    const int ia = s.t0 + p.tokens * x;
    if (ia >= s.n) return {INT_MAX, 0, INT_MIN, INT_MAX};
    const int ib = min(ia + p.tokens, s.n) - 1;
    const int lo = p.q.window > 0 ? max(0, ia - p.q.window + 1) : 0, hi = p.q.causal ? ib + 1 : s.n;
    return {lo / 128, (hi + 127) / 128, p.q.window > 0 ? max(0, ib - p.q.window + 1) : 0, p.q.causal ? ia + 1 : s.n};
}
struct PromptTiles {
    PromptRange r0, r1;  // of the two row tiles
    __device__ __forceinline__ int from(int x) const { return x == 0 ? r0.from : r1.from; }
    __device__ __forceinline__ int to(int x) const { return x == 0 ? r0.to : r1.to; }
    __device__ __forceinline__ int first() const { return r0.from; }
    __device__ __forceinline__ int last() const { return max(r0.to, r1.to); }
    __device__ __forceinline__ bool has(int x, int j) const { return j >= from(x) && j < to(x); }
    __device__ __forceinline__ bool masked(int j) const {  // for some row that has it
        const int pos0 = j * 128, pos1 = pos0 + 128;
        return (has(0, j) && (pos0 < r0.clear0 || pos1 > r0.clear1)) || (has(1, j) && (pos0 < r1.clear0 || pos1 > r1.clear1));
    }
};
__device__ __forceinline__ PromptTiles prompt_tiles(const PromptParams& p, const PromptSegment& s) {
    return {prompt_range(p, s, 0), prompt_range(p, s, 1)};
}
// Whether `bytes` bytes (a multiple of 4096) of shared memory hold elements that are no numbers; by a whole warp.
template <typename T>
__device__ __forceinline__ bool no_numbers(const uint8_t* at, int bytes, int lane) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 sum[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(&sum[i]) = 0;
    const T2 zero = sum[0];
#pragma unroll 1
    for (int n = 0; n < bytes; n += 4096) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint4*>(at + n + 512 * i + 16 * lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const T2* const h = reinterpret_cast<const T2*>(&w[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __hfma2(h[e], zero, sum[e]);
        }
    }
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) odd |= (*reinterpret_cast<const uint32_t*>(&sum[e]) & 0x7FFF7FFFu) != 0;
    return __any_sync(0xFFFFFFFFu, odd);
}

template <typename T, int D>
__global__ void __launch_bounds__(PromptShape<D>::kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptParams p) {
    using S = PromptShape<D>;
    using W = PromptWeights<T>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* const s_q = smem;
    uint8_t* const s_k = s_q + 2 * S::kQBytes;
    uint8_t* const s_v = s_k + S::kBufs * S::kKvBytes;
    __shared__ __align__(8) uint64_t k_full[S::kBufs], k_free[S::kBufs], v_full[S::kBufs], v_ok[S::kBufs], v_free[S::kBufs];
    __shared__ __align__(8) uint64_t q_full[2], q_free[2], s_full[2][2], p_full[2][2], o_full[2][2], seg_full[S::kSegs], seg_free[S::kSegs], turn[2];
    __shared__ PromptSegment s_seg[S::kSegs];
    __shared__ int s_odd[S::kSegs];                                             // a segment's V has elements that are no numbers
    __shared__ int t_before[S::kThreads], t_blocks[S::kThreads];  // where segments are, below
    __shared__ PromptSpan t_span[S::kThreads];
    __shared__ uint32_t s_tmem;
    __shared__ int64_t s_sum[S::kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&k_full[i], 1), mbar_init(&k_free[i], 2);
            mbar_init(&v_full[i], 1), mbar_init(&v_ok[i], 32), mbar_init(&v_free[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1), mbar_init(&q_free[i], 1);
            mbar_init(&turn[i], 1);
            for (int e = 0; e < 2; ++e) mbar_init(&s_full[i][e], 1), mbar_init(&p_full[i][e], 128), mbar_init(&o_full[i][e], 1);
        }
        for (int i = 0; i < S::kSegs; ++i) mbar_init(&seg_full[i], 1), mbar_init(&seg_free[i], 11);
        mbar_fence_init();
        mbar_arrive(&turn[0]);
    }
    pdl_launch_dependents();
    pdl_wait();
    // Tensor memory only once the kernels before this one have ended: who held some while waiting for them could keep it from one of their CTAs.
    if (warp == 8) tc_alloc(&s_tmem, S::kCols);

    // The list of segments. Thread x has requests [x * run, (x + 1) * run). Where that is one each, they are sorted by descending length, and
    // t_blocks, t_span have their blocks (two row tiles of tokens) and tokens; t_before is where what thread x adds to the list starts:
    //   causal: by descending block, whose number says how many keys it sees, over all requests that have it: thread x adds the blocks that
    //           requests 0..x have and x + 1.. have not
    //   else:   request after request
    const int run = (p.q.n_req + S::kThreads - 1) / S::kThreads;
    const bool by_block = run == 1 && p.q.causal != 0;
    int64_t mine = 0;
    if (run == 1) {
        int* const t_len = t_before;
        PromptSpan s = {0, 0};
        if (tid < p.q.n_req) s = prompt_span(p, tid), t_len[tid] = s.n;
        __syncthreads();
        if (tid < p.q.n_req) {
            int rank = 0;
#pragma unroll 1
            for (int r = 0; r < p.q.n_req; ++r) rank += t_len[r] > s.n || (t_len[r] == s.n && r < tid);
            t_span[rank] = s;
            t_blocks[rank] = prompt_blocks(p, s.n);
        }
        __syncthreads();
        if (tid < p.q.n_req) {
            const int b = t_blocks[tid], next = tid + 1 < p.q.n_req ? t_blocks[tid + 1] : 0;
            mine = (by_block ? static_cast<int64_t>(b - next) * (tid + 1) : b) * p.groups;
        }
    } else {
#pragma unroll 1
        for (int64_t r = static_cast<int64_t>(tid) * run; r < min(static_cast<int64_t>(tid + 1) * run, static_cast<int64_t>(p.q.n_req)); ++r)
            mine += static_cast<int64_t>(prompt_blocks(p, prompt_span(p, static_cast<int>(r)).n)) * p.groups;
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t total = 0, before = incl - mine;
#pragma unroll 1
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    if (total > p.most) {  // (requests that overlap: their starts are not in order)
        report(p.status, SGEMV_ERR_ARG);
        total = 0;
    }
    t_before[tid] = static_cast<int>(before);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = s_tmem;
    bool dead = false;  // a wait gave up: nothing is waited for any more, and what comes out is reported as invalid
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || mbar_wait(bar, parity)) return;
        dead = true;
        report(p.status, SGEMV_ERR_TIMEOUT);
    };
    // Segment `it` of this CTA, by a whole warp; n < 0 where there is none (or a wait gave up).
    const auto segment = [&](int it) {
        wait(&seg_full[it % S::kSegs], (it / S::kSegs) & 1);
        dead = __any_sync(0xFFFFFFFFu, dead);
        PromptSegment s = s_seg[it % S::kSegs];
        if (dead) s.n = -1;
        return s;
    };
    const auto release = [&](int it) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_free[it % S::kSegs]);
    };

    if (warp < 8) {
        regs_inc<S::kRegsSoftmax>();
        // ---------------------------------------------------------------------------------------- softmax
        const int x = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + S::kOCols + (S::kAhead ? 64 : 128) * x;
        const float c = p.scale_log2;
        uint32_t tiles = 0;  // that this row tile has had
        int before_segment = 0;  // key tiles of the CTA before the segment
#pragma unroll 1
        for (int it = 0;; ++it) {
            const PromptSegment sg = segment(it);
            if (sg.n < 0) break;
            const PromptTiles all = prompt_tiles(p, sg);
            const PromptRange rg = x == 0 ? all.r0 : all.r1;
            const int g0 = before_segment - all.first();  // key tile j is the CTA's g0 + j th
            before_segment += all.last() - all.first();
            if (rg.from >= rg.to) {
                release(it);
                continue;
            }
            // this thread's token and query head (rows that there are not: as the last token's)
            const int i0 = sg.t0 + p.tokens * x, i = min(i0 + r / p.sub, min(i0 + p.tokens, sg.n) - 1), a = sg.group * p.sub + r % p.sub;
            const bool live = i == i0 + r / p.sub;
            // this row sees positions [see0, see0 + see)
            const int see0 = p.q.window > 0 ? max(0, i - p.q.window + 1) : 0;
            const uint32_t see = static_cast<uint32_t>((p.q.causal ? i + 1 : sg.n) - see0);
            float ref = 0.0f;   // the reference
            bool seen = !live;  // whether it was set (rows that there are not hold anything, and nothing waits for them)
            uint64_t l2 = 0;    // two sums
#pragma unroll 1
            for (int j = rg.from; j < rg.to; ++j, ++tiles) {
                const int pos0 = j * S::kKeys;
                const uint32_t ts = tmem + lanes + S::scores_at(g0 + j, x);
                wait(&s_full[x][tiles & 1], (tiles >> 1) & 1);
                __syncwarp();
                tc_after_sync();
                const bool plain = pos0 >= rg.clear0 && pos0 + S::kKeys <= rg.clear1;
                // Weights in one go. Whether the reference has to move shows in their sum, so that the largest score is looked for in few tiles.
                // (Past kPromptRound: slow, below, as is a scale of 0, which cannot carry the mask.)
                const int rel0 = see0 - pos0, rel1 = rel0 + static_cast<int>(see);
                const auto seen_bits = [&](int q) {  // of keys 32 q .. 32 q + 31
                    const int lo = min(32, max(0, rel0 - 32 * q)), hi = min(32, max(0, rel1 - 32 * q));
                    return static_cast<uint32_t>((1ull << hi) - 1) & ~static_cast<uint32_t>((1ull << lo) - 1);
                };
                bool done = false;
                if (c != 0.0f) {
                    uint32_t raw[4][32], w[64];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_ld32(raw[q], ts + 32 * q);
                    tc_wait_ld();
                    if (!plain) {
                        const uint32_t none = c > 0.0f ? 0xFF800000u : 0x7F800000u;  // a score of -inf
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t bits = seen_bits(q);
#pragma unroll
                            for (int n = 0; n < 32; ++n)
                                if (!((bits >> n) & 1)) raw[q][n] = none;
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, !seen)) {
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int n = 0; n < 128; ++n) top[n & 3] = fmaxf(top[n & 3], __uint_as_float(raw[n / 32][n % 32]) * c);
                        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                        if (!seen && most > -INFINITY) ref = most - W::kTop, seen = true;
                    }
                    uint64_t sums[4] = {0, 0, 0, 0};
                    const uint64_t cc = pair(c, c), mm = pair(-ref, -ref);
#pragma unroll
                    for (int n = 0; n < 128; n += 2) {
                        const float2 t = parts_of(fma2(pair(__uint_as_float(raw[n / 32][n % 32]), __uint_as_float(raw[n / 32][n % 32 + 1])), cc, mm));
                        const float e0 = exp2_approx(t.x), e1 = exp2_approx(t.y);
                        sums[n / 2 % 4] = add2(sums[n / 2 % 4], pair(e0, e1));
                        w[n / 2] = pack_two<T>(e0, e1);
                    }
                    sums[0] = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
                    const float2 both = parts_of(sums[0]);
                    done = !__any_sync(0xFFFFFFFFu, live && (both.x + both.y > W::kBig || fabsf(ref) > kPromptRound));
                    if (done) {
                        l2 = add2(l2, sums[0]);
                        tc_st32(ts, *reinterpret_cast<const uint32_t(*)[32]>(w));
                        tc_st32(ts + 32, *reinterpret_cast<const uint32_t(*)[32]>(w + 32));
                    }
                }
                if (!done) {
                    // 32 keys at a time, in little code: the largest score that each row sees, then the weights. (Those of 32 keys take the
                    // columns of 16: they never reach scores that are still to be read.)
                    float most = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t raw[32];
                        tc_ld32(raw, ts + 32 * q);
                        tc_wait_ld();
                        const uint32_t bits = seen_bits(q);
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int n = 0; n < 32; ++n) top[n & 3] = fmaxf(top[n & 3], (bits >> n) & 1 ? __fmul_rn(__uint_as_float(raw[n]), c) : -INFINITY);
                        most = fmaxf(most, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
                    }
                    float f = 1.0f;
                    if (live && most > -INFINITY && (!seen || most - ref > W::kFar)) {
                        const float m = most - W::kTop;
                        if (seen) f = exp2_approx(ref - m);
                        ref = m;
                        seen = true;
                    }
                    if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
                        l2 = mul2(l2, pair(f, f));
                        if (j > rg.from) {
                            wait(&o_full[x][(tiles - 1) & 1], ((tiles - 1) >> 1) & 1);  // (O holds every tile before this one)
                            __syncwarp();
                            tc_after_sync();
#pragma unroll 1
                            for (int d = 0; d < D / 16; ++d) {
                                uint32_t o[16];
                                tc_ld16(o, to + 16 * d);
                                tc_wait_ld();
#pragma unroll
                                for (int n = 0; n < 16; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f);
                                tc_st16(to + 16 * d, o);
                            }
                        }
                    }
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t raw[32], w[16];
                        tc_ld32(raw, ts + 32 * q);
                        tc_wait_ld();
                        const uint32_t bits = seen_bits(q);
                        uint64_t sums[2] = {0, 0};
#pragma unroll
                        for (int n = 0; n < 32; n += 2) {
                            const float t0 = __fadd_rn(__fmul_rn(__uint_as_float(raw[n]), c), -ref), t1 = __fadd_rn(__fmul_rn(__uint_as_float(raw[n + 1]), c), -ref);
                            const float e0 = exp2_approx((bits >> n) & 1 ? t0 : -INFINITY), e1 = exp2_approx((bits >> (n + 1)) & 1 ? t1 : -INFINITY);
                            sums[n / 2 % 2] = add2(sums[n / 2 % 2], pair(e0, e1));
                            w[n / 2] = pack_two<T>(e0, e1);
                        }
                        l2 = add2(l2, add2(sums[0], sums[1]));
                        tc_st16(ts + 16 * q, w);
                    }
                }
                tc_wait_st();
                tc_before_sync();
                mbar_arrive(&p_full[x][tiles & 1]);
            }
            // Every row sees itself: one without a score above -inf has no softmax (its scores are -inf or NaN) and is NaN, as one with a score of inf or NaN is.
            const float2 lf = parts_of(l2);
            const float l = seen ? lf.x + lf.y : __int_as_float(0x7FC00000);
            const float inv = 1.0f / l;
            if (live && p.q.lse_dev != nullptr)
                p.q.lse_dev[static_cast<int64_t>(sg.first + i) * p.q.heads_q + a] = (ref + log2f(l)) * p.unscale;
            T* const out = static_cast<T*>(p.q.out_dev) + (sg.first + i) * p.q.out_token_stride + a * p.q.out_head_stride;
            wait(&o_full[x][(tiles - 1) & 1], ((tiles - 1) >> 1) & 1);
            __syncwarp();
            tc_after_sync();
            const bool odd = *static_cast<volatile int*>(&s_odd[it % S::kSegs]) != 0;
            uint32_t o[D / 32][32];
#pragma unroll
            for (int q = 0; q < D / 32; ++q) tc_ld32(o[q], to + 32 * q);
            tc_wait_ld();
            if (live) {
                // (32 bytes at a time are whole sectors: as fast as whole lines through shared memory, and 103 us against 110 with a window of 1000)
#pragma unroll
                for (int n = 0; n < D; n += 16) {
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[e] = pack_two<T>(__uint_as_float(o[n / 32][n % 32 + 2 * e]) * inv, __uint_as_float(o[n / 32][n % 32 + 2 * e + 1]) * inv);
                    if (p.out32) {
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + n), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]),
                                     "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                                     : "memory");
                    } else {
                        *reinterpret_cast<uint4*>(out + n) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(out + n + 8) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                }
            }
            if (odd && live) {
                // what was taken out of V, for the rows that see it
                const T* const v_rows = static_cast<const T*>(p.q.v_dev) + sg.group * p.sub / p.ratio * p.q.v_head_stride;
#pragma unroll 1
                for (int pos = max(see0, rg.from * S::kKeys); pos < see0 + static_cast<int>(see); ++pos) {
                    if (!all.masked(pos / S::kKeys)) continue;
#pragma unroll 1
                    for (int d = 0; d < D; ++d) {
                        const float f = to_f32(v_rows[(sg.first + pos) * p.q.v_token_stride + d]);
                        if (!(fabsf(f) < INFINITY)) out[d] = from_f32<T>(to_f32(out[d]) + f);
                    }
                }
            }
            tc_before_sync();  // (the next segment's first weights, which these threads hand over, come after this O)
            release(it);
        }
    } else {
        regs_dec<S::kRegsOther>();
        if (warp < 10) {
        // ---------------------------------------------------------------------------------------- products
        // A warp a row tile, which goes through the loop as a whole, with values that are the same in its lanes; one lane issues. They take turns: a
        // row tile's products of a key tile, O += P V and the next scores (of the next segment, at the end of one), are issued together, so that
        // the two row tiles stay half a period apart (without turns both were in their softmax and then both in their products: 3740 cycles a
        // key tile); and as one waits for what its turn needs while the other issues, the tensor cores get one's after the other's (with
        // one warp for both they stood still for 450 cycles a turn: 3370 cycles).
        const int x = warp - 8;
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), to = tm + S::kOCols + (S::kAhead ? 64 : 128) * x;
        const uint64_t q_desc = tc_desc(smem_addr(s_q) + x * S::kQBytes), k_desc = tc_desc(smem_addr(s_k));
        const uint64_t v_desc = tc_desc_v(smem_addr(s_v), S::kKeys * 128);
        constexpr uint32_t kScores = tc_idesc(S::kKeys) | tc_idesc_type<T>(), kOut = tc_idesc(D) | tc_idesc_type<T>() | (1u << 16);
        const auto hold = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            dead = __any_sync(0xFFFFFFFFu, dead);
        };
        uint32_t q_had = 0, s_had = 0, p_had = 0;
        PromptSegment sg = segment(0);
        PromptTiles t = prompt_tiles(p, sg);
        int it = 0, g = -1;  // segment; key tiles so far
#pragma unroll 1
        for (int j = t.first() - 1; sg.n >= 0; ++g) {
            // O += P V of key tile j (but before the first of all), and scores of the tile after it, of this segment or the next
            PromptSegment next_sg = sg;
            PromptTiles next = t;
            int next_j = j + 1;
            const bool cross = next_j == t.last();
            if (cross) {
                next_sg = segment(it + 1);
                next = prompt_tiles(p, next_sg);
                next_j = next.first();
            }
            const bool old_keys = t.has(x, j), new_keys = next_sg.n >= 0 && next.has(x, next_j);
            const int buf = g & 1, next_buf = buf ^ 1;
            const uint32_t parity = (g >> 1) & 1, next_parity = ((g + 1) >> 1) & 1;
            const uint64_t vd = v_desc + buf * (S::kKvBytes >> 4), kd = k_desc + next_buf * (S::kKvBytes >> 4);
            const bool add = j > t.from(x);
            const uint32_t from = tm + S::scores_at(g, x), ts = tm + S::scores_at(g + 1, x);
            const auto give_turn = [&]() {  // the other's products come after those issued so far
                tc_before_sync();
                mbar_arrive(&turn[x ^ 1]);
            };
            const auto outputs = [&]() {
                if (!old_keys) {
                    if (S::kAhead && lane == 0) give_turn();
                    return;
                }
                hold(&p_full[x][p_had & 1], (p_had >> 1) & 1);
                tc_after_sync();
                if (elect_one()) {
                    if (!dead) {
#pragma unroll
                        for (int kk = 0; kk < S::kKeys / 16; ++kk) tc_mma_ts(to, from + 8 * kk, vd + kk * (2048 >> 4), kOut, kk > 0 || add);
                    }
                    if (S::kAhead) give_turn();
                    tc_commit(&v_free[buf]);
                    tc_commit(&o_full[x][p_had & 1]);
                }
                ++p_had;
                __syncwarp();
            };
            const auto scores = [&]() {
                if (cross && next_sg.n >= 0) hold(&k_full[next_buf], next_parity);
                if (!new_keys) {
                    if (!S::kAhead && lane == 0) give_turn();
                    if (next_sg.n >= 0 && lane == 0) mbar_arrive(&k_free[next_buf]);
                    return;
                }
                if (next_j == next.from(x)) {
                    hold(&q_full[x], q_had++ & 1);
                    tc_after_sync();
                }
                if (elect_one()) {
                    if (!dead) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (kk / 4 * (128 * 128) + kk % 4 * 32) >> 4;
                            tc_mma_ss(ts, q_desc + off, kd + off, kScores, kk > 0);
                        }
                    }
                    if (!S::kAhead) give_turn();
                    tc_commit(&s_full[x][s_had & 1]);
                    tc_commit(&k_free[next_buf]);
                    if (next_j == next.to(x) - 1) tc_commit(&q_free[x]);
                }
                ++s_had;
                __syncwarp();
            };
            // (who does not have a tile lets it go all the same, once it is there: its buffers wait for both)
            if (g >= 0) hold(&v_ok[buf], parity);
            if (!cross) hold(&k_full[next_buf], next_parity);
            if (!old_keys && g >= 0 && lane == 0) mbar_arrive(&v_free[buf]);
            hold(&turn[x], (g + 1) & 1);
            tc_after_sync();
            // (products run in the order of their issue: the scores go over weights whose products come before)
            if constexpr (S::kAhead) {
                scores();
                outputs();
            } else {
                outputs();
                scores();
            }
            if (cross) release(it++);
            sg = next_sg, t = next, j = next_j;
        }
        // The last products arrive at barriers that nobody else waits for: none may be under way when the CTA's memory goes.
#pragma unroll 1
        for (int i = max(0, g - S::kBufs); i < g; ++i) {
            mbar_wait(&k_free[i % S::kBufs], (i / S::kBufs) & 1);
            mbar_wait(&v_free[i % S::kBufs], (i / S::kBufs) & 1);
        }
        } else if (warp == 10) {
        // ---------------------------------------------------------------------------------------- segments and copies
        int g = 0;
        uint32_t q_had[2] = {0, 0};
#pragma unroll 1
        for (int it = 0;; ++it) {
            if (it >= S::kSegs) wait(&seg_free[it % S::kSegs], (it / S::kSegs - 1) & 1);
            dead = __any_sync(0xFFFFFFFFu, dead);
            // Every other round of the list is dealt backwards, so that who has the longest of one has the shortest of the next.
            const int64_t want = static_cast<int64_t>(it) * gridDim.x + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            PromptSegment sg = {0, -1, 0, 0};
            if (want < total && !dead) {
                int x = -1;  // the last thread that starts at or before `want`
#pragma unroll 1
                for (int i = lane; i < min(p.q.n_req, S::kThreads); i += 32)
                    if (t_before[i] <= want) x = i;
                x = __reduce_max_sync(0xFFFFFFFFu, x);
                unsigned o = static_cast<unsigned>(want) - t_before[x];
                const unsigned groups = p.groups;
                PromptSpan s;
                unsigned block;
                if (run == 1) {
                    const unsigned width = by_block ? (x + 1) * groups : groups;
                    block = t_blocks[x] - 1 - o / width;
                    o %= width;
                    s = t_span[by_block ? o / groups : x];
                } else {
                    s = {0, 0}, block = 0;
#pragma unroll 1
                    for (int64_t req = static_cast<int64_t>(x) * run; req < min(static_cast<int64_t>(x + 1) * run, static_cast<int64_t>(p.q.n_req)); ++req) {
                        s = prompt_span(p, static_cast<int>(req));
                        const unsigned n = prompt_blocks(p, s.n) * groups;
                        if (o < n) {
                            block = n / groups - 1 - o / groups;
                            break;
                        }
                        o -= n;
                    }
                }
                if (s.n > 0) sg = {s.first, s.n, static_cast<int>(o % groups), static_cast<int>(block) * 2 * p.tokens};
            }
            if (lane == 0) {
                s_seg[it % S::kSegs] = sg;
                s_odd[it % S::kSegs] = 0;
                mbar_arrive(&seg_full[it % S::kSegs]);
            }
            __syncwarp();
            if (sg.n < 0) break;
            const PromptTiles t = prompt_tiles(p, sg);
            const int head = sg.group * p.sub / p.ratio;
            if (it > 0 && lane < 2 * S::kAtoms && t.to(lane & 1) > 0)  // (their place is not free for a while)
                tma_prefetch(&q_map, 64 * (lane >> 1), sg.group * p.sub, sg.first + sg.t0 + p.tokens * (lane & 1));
            __syncwarp();
#pragma unroll 1
            for (int j = t.first(); j < t.last() && !dead; ++j, ++g) {
                const int buf = g % S::kBufs, key = sg.first + j * S::kKeys;
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    uint64_t* const bar = v ? &v_full[buf] : &k_full[buf];
                    if (g >= S::kBufs) wait(v ? &v_free[buf] : &k_free[buf], (g / S::kBufs - 1) & 1);
                    dead = __any_sync(0xFFFFFFFFu, dead);
                    if (dead) {  // (what was asked for is waited for below)
                        if (v) mbar_wait(&k_full[buf], (g / S::kBufs) & 1);
                        break;
                    }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, S::kKvBytes);
                        uint8_t* const dst = (v ? s_v : s_k) + buf * S::kKvBytes;
#pragma unroll
                        for (int d = 0; d < S::kAtoms; ++d) tma_load(dst + d * (S::kKeys * 128), v ? &v_map : &k_map, 64 * d, head, key, bar);
                    }
                    __syncwarp();
                    if (v == 0 && j == t.first()) {
                        // the segment's queries, once the products are done with those of the one before
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (t.to(x) == 0) continue;
                            if (q_had[x] > 0) wait(&q_free[x], (q_had[x] - 1) & 1);
                            dead = __any_sync(0xFFFFFFFFu, dead);
                            if (dead) break;
                            ++q_had[x];
                            if (lane == 0) {
                                mbar_arrive_expect_tx(&q_full[x], p.tokens * p.sub * D * 2);
#pragma unroll
                                for (int d = 0; d < S::kAtoms; ++d)
                                    tma_load(s_q + x * S::kQBytes + d * (128 * 128), &q_map, 64 * d, sg.group * p.sub, sg.first + sg.t0 + p.tokens * x, &q_full[x]);
                            }
                            __syncwarp();
                        }
                    }
                }
                if (dead) break;
            }
        }
        // (all have landed, unless someone gave up)
#pragma unroll 1
        for (int i = max(0, g - S::kBufs); i < g; ++i) {
            mbar_wait(&k_full[i % S::kBufs], (i / S::kBufs) & 1);
            mbar_wait(&v_full[i % S::kBufs], (i / S::kBufs) & 1);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (q_had[x] > 0) mbar_wait(&q_full[x], (q_had[x] - 1) & 1);
        } else {
        // ---------------------------------------------------------------------------------------- V that is not seen
        int g = 0;
#pragma unroll 1
        for (int it = 0;; ++it) {
            const PromptSegment sg = segment(it);
            if (sg.n < 0) break;
            const PromptTiles t = prompt_tiles(p, sg);
            const int last = t.last();
#pragma unroll 1
            for (int j = t.first(); j < last; ++j, ++g) {
                const int buf = g % S::kBufs;
                wait(&v_full[buf], (g / S::kBufs) & 1);
                __syncwarp();
                // 0 times a number is 0: a look at the whole tile takes one instruction a word
                if (t.masked(j) && no_numbers<T>(s_v + buf * S::kKvBytes, S::kKvBytes, lane)) {
                    uint8_t* const tile = s_v + buf * S::kKvBytes;
                    const int keys = sg.n - j * S::kKeys;  // of the request
                    constexpr uint32_t kNot = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
                    bool odd = false;
#pragma unroll 1
                    for (int n = lane; n < S::kKvBytes / 16; n += 32) {
                        uint4* const at16 = reinterpret_cast<uint4*>(tile) + n;
                        uint4 w = *at16;
                        if (n / 8 % S::kKeys >= keys) {
                            *at16 = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint32_t bx = __vcmpeq2(w.x & kNot, kNot), by = __vcmpeq2(w.y & kNot, kNot), bz = __vcmpeq2(w.z & kNot, kNot),
                                       bw = __vcmpeq2(w.w & kNot, kNot);
                        if (bx | by | bz | bw) {
                            w.x &= ~bx, w.y &= ~by, w.z &= ~bz, w.w &= ~bw;
                            *at16 = w;
                            odd = true;
                        }
                    }
                    if (odd) *static_cast<volatile int*>(&s_odd[it % S::kSegs]) = 1;
                    __threadfence_block();
                    fence_async();
                }
                mbar_arrive(&v_ok[buf]);
            }
            release(it);
        }
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 8) tc_dealloc(tmem, S::kCols);
}

}  // namespace sgemv
