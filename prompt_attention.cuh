// Causal attention over packed prompts: softmax(scale q K^T) V of each request's own tokens, unquantised keys and values.
//
// Bound by the products, 4 D operations a (row, key), where prompts are long. Both go to the 5th-generation tensor cores with 128 x 128 x 16 and 128
// x D x 16 instructions. A row is a (token, query head) of one KV head, token after token, so that grouped heads share the keys they read and
// a tile's rows see about the same keys. A CTA has two 128-row tiles against the same 128-key tiles: while one is in its softmax the other's
// products run. Roles, by warp:
//   0-3, 4-7  softmax of the first and of the second row tile: a thread a row, scores from tensor memory, weights back over them
//   8         issues the products      9  issues the copies of K and V tiles (two buffers each)
//   10, 11    look through V tiles that are masked for some row (below)
// The softmax's reference m moves only when a tile's sum of weights passes 2^15 (and in a row's first tile), so that the largest score is
// looked for in few tiles and the output's sums are rarely rescaled.
//
// Roundings: scores are sums of exact products in 32 bits, scaled in 32 bits. Weights 2^(t - m) are rounded to the type of V, since the
// instruction takes one type for both (11 bits for fp16, whose end 2^16 the limit on m keeps away from; 8 for bf16).
//
// What a row does not see must not enter its sums whatever it holds, but 0 * NaN is NaN in the tensor cores. Scores are selected, so K needs
// nothing. In V tiles that some row does not see in full, rows past the request's end are cleared, and elements that are no numbers are
// taken out and remembered; if there were any, the rows that see them get them at their end.
#pragma once

#include <cuda.h>

#include "fp4_common.cuh"
#include "tcgen05.cuh"

namespace sgemv {
__device__ long long g_stamp[3*128*8];
#define STAMP(w,j,i) do { if (blockIdx.x==0 && lane==0 && (j)<128) g_stamp[((w)*128+(j))*8+(i)] = clock64(); } while(0)

struct PromptParams {
    sgemv_prompt_query q;
    int32_t* status;
    int ratio;
    float scale_log2;
};

template <int D>
struct PromptShape {
    static constexpr int kRows = 256, kTile = 128, kKeys = 128;
    static constexpr int kAtoms = D / 64;  // 128-byte columns of a row
    static constexpr int kBufs = 2;        // of K and of V
    static constexpr int kQBytes = kTile * D * 2, kKvBytes = kKeys * D * 2;
    static constexpr int kWarps = 12, kThreads = 32 * kWarps;
    static constexpr int kSmem = 1024 + 2 * kQBytes + 2 * kBufs * kKvBytes;
    static constexpr int kCols = 512;  // tensor memory: S of both row tiles (128 columns each), O of both
};

constexpr float kPromptTop = 6.0f, kPromptBig = 32768.0f;  // log2 of the largest weight when the reference is set; the limit of a tile's sum

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
__device__ __forceinline__ int64_t prompt_segments(const PromptParams& p, const PromptSpan& s, int rows) {
    return static_cast<int64_t>((static_cast<int64_t>(s.n) * p.ratio + rows - 1) / rows) * p.q.heads;
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_addr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
                 : "memory");
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

template <typename T, int D>
__global__ void __launch_bounds__(PromptShape<D>::kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptParams p) {
    using S = PromptShape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* const s_q = smem;
    uint8_t* const s_k = s_q + 2 * S::kQBytes;
    uint8_t* const s_v = s_k + S::kBufs * S::kKvBytes;
    __shared__ __align__(8) uint64_t k_full[S::kBufs], k_free[S::kBufs], v_full[S::kBufs], v_ok[S::kBufs], v_free[S::kBufs];
    __shared__ __align__(8) uint64_t q_full, s_full[2], p_full[2], o_full[2];
    __shared__ uint32_t s_tmem;
    __shared__ int64_t s_sum[S::kWarps];
    __shared__ int s_req, s_odd;
    __shared__ int64_t s_before;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&k_full[i], 1), mbar_init(&k_free[i], 1);
            mbar_init(&v_full[i], 1), mbar_init(&v_ok[i], 64), mbar_init(&v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 128), mbar_init(&o_full[i], 1);
        mbar_init(&q_full, 256);
        mbar_fence_init();
        s_req = -1, s_odd = 0;
    }
    pdl_launch_dependents();
    pdl_wait();

    // The request whose segment (two row tiles of a KV head) this CTA has. Thread x has requests [x * run, (x + 1) * run); where that is one
    // each, they are taken by descending length, so that the longest segments do not come last.
    const int run = (p.q.n_req + S::kThreads - 1) / S::kThreads;
    int64_t mine = 0;
    int* const t_len = reinterpret_cast<int*>(s_q);  // until the queries come
    int* const t_order = t_len + S::kThreads;
    int* const t_count = t_order + S::kThreads;
    if (run == 1) {
        int count = 0;
        if (tid < p.q.n_req) {
            const PromptSpan s = prompt_span(p, tid);
            count = static_cast<int>(prompt_segments(p, s, S::kRows));
            t_len[tid] = s.n;
        }
        __syncthreads();
        if (tid < p.q.n_req) {
            const int len = t_len[tid];
            int rank = 0;
            for (int r = 0; r < p.q.n_req; ++r) rank += t_len[r] > len || (t_len[r] == len && r < tid);
            t_order[rank] = tid;
            t_count[rank] = count;
        }
        __syncthreads();
        if (tid < p.q.n_req) mine = t_count[tid];
    } else {
        for (int64_t r = static_cast<int64_t>(tid) * run; r < min(static_cast<int64_t>(tid + 1) * run, static_cast<int64_t>(p.q.n_req)); ++r)
            mine += prompt_segments(p, prompt_span(p, static_cast<int>(r)), S::kRows);
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
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    if (blockIdx.x >= total) return;
    const int64_t want = blockIdx.x;
    if (want >= before && want < before + mine) {
        int r = run == 1 ? t_order[tid] : tid * run;
        for (; run > 1; ++r) {
            const int64_t n = prompt_segments(p, prompt_span(p, r), S::kRows);
            if (want < before + n) break;
            before += n;
        }
        s_req = r, s_before = before;
    }
    if (warp == 8) tc_alloc(&s_tmem, S::kCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = s_tmem;
    const PromptSpan sp = prompt_span(p, s_req);
    // within a request the last rows, which see the most keys, come first
    const int in_req = static_cast<int>(want - s_before), rows = sp.n * p.ratio;
    const int head = in_req % p.q.heads, row0 = ((rows + S::kRows - 1) / S::kRows - 1 - in_req / p.q.heads) * S::kRows;
    // Keys [lo, hi) that row tile x sees, in tiles [from, to); those with positions in [clear0, clear1) are seen in full by all its rows.
    struct Range {
        int from, to, clear0, clear1;
    };
    const auto range_of = [&](int x) {
        const int a = row0 + 128 * x;
        if (a >= rows) return Range{INT_MAX, 0, INT_MIN, INT_MAX};
        const int ia = a / p.ratio, ib = min(a + 127, rows - 1) / p.ratio;
        const int lo = p.q.window > 0 ? max(0, ia - p.q.window + 1) : 0, hi = p.q.causal ? ib + 1 : sp.n;
        return Range{lo / S::kKeys, (hi + S::kKeys - 1) / S::kKeys, p.q.window > 0 ? max(0, ib - p.q.window + 1) : 0, p.q.causal ? ia + 1 : sp.n};
    };
    const Range r0 = range_of(0), r1 = range_of(1);
    const int first = r0.from, last = max(r0.to, r1.to);  // tiles of the CTA
    bool dead = false;  // a wait gave up: nothing is waited for any more, and what comes out is reported as invalid
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || mbar_wait(bar, parity)) return;
        dead = true;
        report(p.status, SGEMV_ERR_TIMEOUT);
    };
    const auto masked = [&](int j) {  // for some row that has it
        const int pos0 = j * S::kKeys, pos1 = pos0 + S::kKeys;
        return (j >= r0.from && j < r0.to && (pos0 < r0.clear0 || pos1 > r0.clear1)) ||
               (j >= r1.from && j < r1.to && (pos0 < r1.clear0 || pos1 > r1.clear1));
    };

    if (warp < 8) {
        // ---------------------------------------------------------------------------------------- softmax
        const int x = warp >> 2, r = tid & 127, row = row0 + 128 * x + r;
        const bool live = row < rows;
        const Range rg = x == 0 ? r0 : r1;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + 128 * x;
        const int i = min(row, rows - 1) / p.ratio, a = head * p.ratio + min(row, rows - 1) % p.ratio;
        {
            const T* const src = static_cast<const T*>(p.q.q_dev) + (sp.first + i) * p.q.q_token_stride + a * p.q.q_head_stride;
            uint8_t* const dst = s_q + x * S::kQBytes + r * 128;
#pragma unroll
            for (int d = 0; d < D; d += 8) {
                const uint4 w = live ? *reinterpret_cast<const uint4*>(src + d) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(dst + d / 64 * (128 * 128) + (((d / 8) & 7) ^ (r & 7)) * 16) = w;
            }
            fence_async();
            mbar_arrive(&q_full);
        }
        // this row sees positions [see0, see0 + see)
        const int see0 = p.q.window > 0 ? max(0, i - p.q.window + 1) : 0;
        const uint32_t see = static_cast<uint32_t>((p.q.causal ? i + 1 : sp.n) - see0);
        const float c = p.scale_log2;
        float ref = 0.0f;   // the reference
        bool seen = false;  // whether it was set
        uint64_t l2 = 0;    // two sums
        for (int j = rg.from; j < rg.to; ++j) {
            const int pos0 = j * S::kKeys;
            wait(&s_full[x], (j - rg.from) & 1);  // (and all products issued before: O holds every tile before this one)
            __syncwarp();
            tc_after_sync();
            if ((warp&3)==0) STAMP(x,j,0);
            const bool plain = pos0 >= rg.clear0 && pos0 + S::kKeys <= rg.clear1;
            uint32_t w[64];
            uint64_t sum;
            // The weights of 32 keys. Past 2^26, scores are rounded before the reference comes off, so that the largest has a weight of about
            // 2^kPromptTop; else one rounding for both.
            const auto weights = [&](const uint32_t (&raw)[32], int q, bool select) {
                if (!select) {
                    const uint64_t cc = pair(c, c), mm = pair(-ref, -ref);
#pragma unroll
                    for (int n = 0; n < 32; n += 2) {
                        const float2 t = parts_of(fma2(pair(__uint_as_float(raw[n]), __uint_as_float(raw[n + 1])), cc, mm));
                        const float e0 = exp2_approx(t.x), e1 = exp2_approx(t.y);
                        sum = add2(sum, pair(e0, e1));
                        w[16 * q + n / 2] = pack_two<T>(e0, e1);
                    }
                } else {
                    const uint32_t at = static_cast<uint32_t>(pos0 + 32 * q - see0);
#pragma unroll
                    for (int n = 0; n < 32; n += 2) {
                        const float t0 = __fadd_rn(__fmul_rn(__uint_as_float(raw[n]), c), -ref), t1 = __fadd_rn(__fmul_rn(__uint_as_float(raw[n + 1]), c), -ref);
                        const float e0 = at + n < see ? exp2_approx(t0) : 0.0f, e1 = at + n + 1 < see ? exp2_approx(t1) : 0.0f;
                        sum = add2(sum, pair(e0, e1));
                        w[16 * q + n / 2] = pack_two<T>(e0, e1);
                    }
                }
            };
            bool need = !seen;
            for (int pass = 0;; ++pass) {
                if (__any_sync(0xFFFFFFFFu, need)) {
                    // the largest score that this row sees
                    float top = -INFINITY;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t raw[32];
                        tc_ld32(raw, ts + 32 * q);
                        tc_wait_ld();
                        const uint32_t at = static_cast<uint32_t>(pos0 + 32 * q - see0);
#pragma unroll
                        for (int n = 0; n < 32; ++n)
                            if (at + n < see) top = fmaxf(top, __fmul_rn(__uint_as_float(raw[n]), c));
                    }
                    float f = 1.0f;
                    if (need && top > -INFINITY) {
                        const float m = top - kPromptTop;
                        if (seen) f = exp2_approx(ref - m);
                        ref = m;
                        seen = true;
                    }
                    l2 = mul2(l2, pair(f, f));
                    if (j > rg.from && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
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
                sum = 0;
                const bool select = !plain || __any_sync(0xFFFFFFFFu, fabsf(ref) > 67108864.0f);
                uint32_t raw[2][32];
                tc_ld32(raw[0], ts);
                tc_wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q < 3) tc_ld32(raw[(q + 1) & 1], ts + 32 * (q + 1));
                    weights(raw[q & 1], q, select);
                    if (q < 3) tc_wait_ld();
                }
                const float2 both = parts_of(sum);
                need = both.x + both.y > kPromptBig;  // (not after the reference has moved)
                if (pass == 2 || !__any_sync(0xFFFFFFFFu, need)) break;
            }
            if ((warp&3)==0) STAMP(x,j,1);
            l2 = add2(l2, sum);
            tc_st32(ts, *reinterpret_cast<const uint32_t(*)[32]>(w));
            tc_st32(ts + 32, *reinterpret_cast<const uint32_t(*)[32]>(w + 32));
            tc_wait_st();
            tc_before_sync();
            mbar_arrive(&p_full[x]);
            if ((warp&3)==0) STAMP(x,j,2);
        }
        if (rg.from < rg.to) {
            wait(&o_full[x], 0);
            __syncwarp();
            tc_after_sync();
            const float2 lf = parts_of(l2);
            const float l = lf.x + lf.y;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            T* const out = static_cast<T*>(p.q.out_dev) + (sp.first + i) * p.q.out_token_stride + a * p.q.out_head_stride;
            const bool odd = *static_cast<volatile int*>(&s_odd) != 0;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tc_ld32(o, to + 32 * q);
                tc_wait_ld();
                if (!live) continue;
                if (odd) {
                    // what was taken out of V, for the rows that see it
                    for (int j = rg.from; j < rg.to; ++j) {
                        if (!masked(j)) continue;
                        for (int pos = max(see0, j * S::kKeys); pos < min(see0 + static_cast<int>(see), (j + 1) * S::kKeys); ++pos) {
                            const T* const v = static_cast<const T*>(p.q.v_dev) + (sp.first + pos) * p.q.v_token_stride + head * p.q.v_head_stride + 32 * q;
#pragma unroll
                            for (int n = 0; n < 32; ++n) {
                                const float f = to_f32(v[n]);
                                if (!(fabsf(f) < INFINITY)) o[n] = __float_as_uint(__uint_as_float(o[n]) + f);
                            }
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < 32; n += 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        h[e] = pack_two<T>(__uint_as_float(o[n + 2 * e]) * inv, __uint_as_float(o[n + 2 * e + 1]) * inv);
                    *reinterpret_cast<uint4*>(out + 32 * q + n) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
            if (live && p.q.lse_dev != nullptr)
                p.q.lse_dev[static_cast<int64_t>(sp.first + i) * p.q.heads_q + a] = seen ? (ref + log2f(l)) * 0.693147180559945309f : -INFINITY;
        }
    } else if (warp == 8) {
        // ---------------------------------------------------------------------------------------- products
        // The whole warp goes through the loop, with values that are the same in its lanes; one lane issues. A row tile's products of a key tile,
        // O += P V and the next scores, are issued together, so that the two row tiles stay half a period apart: with a warp for each, both
        // were in their softmax and then both in their products (3740 cycles a key tile).
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        const uint64_t q_desc = tc_desc(smem_addr(s_q)), k_desc = tc_desc(smem_addr(s_k));
        const uint64_t v_desc = tc_desc_v(smem_addr(s_v), S::kKeys * 128);
        constexpr uint32_t kScores = tc_idesc(S::kKeys) | tc_idesc_type<T>(), kOut = tc_idesc(D) | tc_idesc_type<T>() | (1u << 16);
        const auto hold = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            dead = __any_sync(0xFFFFFFFFu, dead);
            tc_after_sync();
        };
        const auto scores = [&](int x, int j, bool free_k) {
            const int at = j - first, buf = at % S::kBufs;
            hold(&k_full[buf], (at / S::kBufs) & 1);
            if (elect_one()) {
                const uint64_t kd = k_desc + buf * (S::kKvBytes >> 4), qd = q_desc + x * (S::kQBytes >> 4);
                if (!dead) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk / 4 * (128 * 128) + kk % 4 * 32) >> 4;
                        tc_mma_ss(tm + 128 * x, qd + off, kd + off, kScores, kk > 0);
                    }
                }
                tc_commit(&s_full[x]);
                if (free_k) tc_commit(&k_free[buf]);
            }
            __syncwarp();
        };
        // of a key tile, the last row tile that has it frees its buffers
        const auto last_user = [&](int x, int j) { return x == 1 || j < r1.from || j >= r1.to; };
        hold(&q_full, 0);
        for (int j = first - 1; j < last; ++j) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int from = x == 0 ? r0.from : r1.from, end = x == 0 ? r0.to : r1.to;
                if (j >= from && j < end) {
                    const int at = j - first, buf = at % S::kBufs;
                    hold(&v_ok[buf], (at / S::kBufs) & 1);
                    hold(&p_full[x], (j - from) & 1);
                    STAMP(x,j,3);
                    if (elect_one()) {
                        const uint64_t vd = v_desc + buf * (S::kKvBytes >> 4);
                        if (!dead) {
#pragma unroll
                            for (int kk = 0; kk < S::kKeys / 16; ++kk)
                                tc_mma_ts(tm + 256 + 128 * x, tm + 128 * x + 8 * kk, vd + kk * (2048 >> 4), kOut, j > from || kk > 0);
                        }
                        if (last_user(x, j)) tc_commit(&v_free[buf]);
                        if (j == end - 1) tc_commit(&o_full[x]);
                    }
                    __syncwarp();
                    STAMP(x,j,4);
                }
                // (over the weights just used: the products run in the order of their issue)
                if (j + 1 >= from && j + 1 < end) { scores(x, j + 1, last_user(x, j + 1)); if (j>=0) STAMP(x,j,5);}
            }
        }
        // The last products arrive at barriers that nobody else waits for: none may be under way when the CTA's memory goes.
        for (int at = max(0, last - first - S::kBufs); at < last - first; ++at) {
            mbar_wait(&k_free[at % S::kBufs], (at / S::kBufs) & 1);
            mbar_wait(&v_free[at % S::kBufs], (at / S::kBufs) & 1);
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------------------------------------- copies
        if (lane == 0) {
            int at = 0;
            for (; at < last - first; ++at) {
                const int buf = at % S::kBufs, key = sp.first + (first + at) * S::kKeys;
                for (int v = 0; v < 2; ++v) {
                    uint64_t* const bar = v ? &v_full[buf] : &k_full[buf];
                    if (at >= S::kBufs) wait(v ? &v_free[buf] : &k_free[buf], (at / S::kBufs - 1) & 1);
                    if (dead) break;
                    mbar_arrive_expect_tx(bar, S::kKvBytes);
                    uint8_t* const dst = (v ? s_v : s_k) + buf * S::kKvBytes;
#pragma unroll
                    for (int d = 0; d < S::kAtoms; ++d) tma_load(dst + d * (S::kKeys * 128), v ? &v_map : &k_map, 64 * d, head, key, bar);
                }
                if (dead) break;
            }
            for (int i = max(0, at - S::kBufs); i < min(at + 1, last - first); ++i) {  // (all have landed, unless someone gave up)
                mbar_wait(&k_full[i % S::kBufs], (i / S::kBufs) & 1);
                if (i < at) mbar_wait(&v_full[i % S::kBufs], (i / S::kBufs) & 1);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------------------------------- V that is not seen
        for (int at = 0; at < last - first; ++at) {
            const int buf = at % S::kBufs, j = first + at;
            wait(&v_full[buf], (at / S::kBufs) & 1);
            __syncwarp();
            if (masked(j)) {
                uint8_t* const tile = s_v + buf * S::kKvBytes;
                const int keys = sp.n - j * S::kKeys;  // of the request
                constexpr uint32_t kNot = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
                bool odd = false;
#pragma unroll 4
                for (int n = tid - 320; n < S::kKvBytes / 16; n += 64) {
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
                if (odd) *static_cast<volatile int*>(&s_odd) = 1;
                __threadfence_block();
                fence_async();
            }
            mbar_arrive(&v_ok[buf]);
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 8) tc_dealloc(tmem, S::kCols);
}

}  // namespace sgemv
