// Attention over the paged 4-bit KV cache: the decode kernel.
//
// With q the integers of a cached row, s its scale and z its zero point, k = s (q - z) and v the same:
//   t_j = log2(e) scale x . k_j = c s_j (sum_d x_d q_jd - z_j sum_d x_d)
//   out = sum_j 2^(t_j - m) s'_j (q'_j - z'_j) / sum_j 2^(t_j - m)
// for any reference m near the largest t_j. Integers and their scales never meet in a rounded product: the matrix
// instruction multiplies x by the integers (exact, 32-bit sums), and the second one the weights 2^(t - m) s', rounded
// once to 11 bits, by the integers of V; the zero points come off in 32 bits, from the same rounded weights.
//
// A nibble masked out of its word at bit 0 or 4 is the fp16 subnormal q 2^-24 or q 2^-20: one AND turns 4 bits into two
// operands, no conversion. The powers of two are taken up by x (odd dims are divided by 16, each row is scaled into
// fp16's middle by a power of two) and by the epilogue.
//
// Both products are computed transposed, S^T = K x^T and O^T = V^T P^T, so that the cache is the 16-row operand of
// mma.m16n8k16 and 8 rows of queries (query heads of a KV head x new tokens) the narrow one: with few rows this is half the
// tensor work of the usual orientation, and the weights become the second product's operand with one movmatrix per 8 x 8.
//
// Work: the 32-token tiles of all (request, row tile, head) segments form one list, split evenly over the CTAs and
// again over their warps, whatever the lengths. A warp copies its tiles (two 16-token subtiles, contiguous in the
// cache) into a ring of its own with the copy engine and keeps the softmax's reference, sum and O in registers. Segments
// that cross warps are joined in shared memory, those that cross CTAs through the workspace by the last CTA to arrive,
// always in the order of the keys: the same inputs give the same bits.
#pragma once

#include "kv_common.cuh"

namespace sgemv {

constexpr int kTileTok = 32;      // tokens of a tile
constexpr int kMaxLen = 1 << 30;  // positions past the end of a tile stay in 32 bits
constexpr float kWeightScale = 64.0f;   // weights go into fp16 times this
constexpr float kMaxGrowth = 8.0f;      // the reference m follows the maximum when it is passed by more than this (log2)

struct AttnParams {
    const uint8_t* cache;
    uint64_t sub_bytes, head_bytes, page_bytes;
    sgemv_kv_query q;
    int32_t* status;
    int heads, page, log2_page, n_pages, ratio;
    float scale_log2;  // scale * log2(e)
};

// The registers, shared memory and warps of one instance: T queries, dim D, group G, 8 NT rows.
template <int D, int G, int NT>
struct AttnShape {
    static constexpr int kPanel = D < 128 ? D : 128, kPanels = D / kPanel;
    static constexpr int kGroups = D / G;
    static constexpr bool kSplit = G < kPanel;       // a panel holds two groups
    static constexpr int kSubBytes = 16 * D + 128 * kGroups;
    static constexpr int kStageBytes = 2 * kSubBytes;
    static constexpr int kWarps = (D == 256 || NT > 1) ? 8 : 16;
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;             // floats of a partial row: 4 more so that two rows are 8 banks apart
    static constexpr int kPartial = kRows * kPitch + 2 * kRows;  // floats of a partial: O, then m, then l
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kJoin = kWarps * kPartial * 4;
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

// What request r asks for; n = 0 where there is nothing to do.
struct Span {
    int first, n, len;
};

__device__ __forceinline__ Span span_of(const AttnParams& p, int r) {
    const int a = p.q.q_start_dev[r], b = p.q.q_start_dev[r + 1], len = p.q.len_dev[r];
    Span s = {a, b - a, len};
    if (a < 0 || b < a || b > p.q.n_tokens || b - a > p.q.max_q || len < 0) {
        report(p.status, SGEMV_ERR_ARG);
        s.n = 0;
    } else if (len > kMaxLen || (len + p.page - 1) >> p.log2_page > p.q.table_cols) {
        report(p.status, SGEMV_ERR_SHAPE);
        s.n = 0;
    }
    return s;
}

// The keys of rows [row0, row0 + rows) of a request: the first one (a multiple of the tile) and the end.
struct Keys {
    int lo, hi, tiles;
};

__device__ __forceinline__ Keys keys_of(const AttnParams& p, const Span& s, int row0, int rows) {
    const int i0 = row0 / p.ratio, i1 = min(row0 + rows - 1, s.n * p.ratio - 1) / p.ratio;
    const int old = s.len - s.n;
    Keys k;
    k.hi = p.q.tree_dev != nullptr ? s.len : max(0, old + i1 + 1);
    k.lo = p.q.window > 0 ? max(0, old + i0 - p.q.window + 1) / kTileTok * kTileTok : 0;
    k.tiles = max(1, (k.hi - k.lo + kTileTok - 1) / kTileTok);  // rows that see nothing still have an owner
    return k;
}

// A (request, row tile, head) and its place in the list of tiles.
struct Segment {
    int r, row0, head;
    Span span;
    Keys keys;
    int64_t start;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

constexpr float kTwo24 = 16777216.0f, kTwo20 = 1048576.0f;

// Writes row R (of its request) of a finished segment: dims and logarithm of the sum.
template <typename T>
__device__ __forceinline__ T* out_row(const AttnParams& p, const Segment& s, int row, int& tok, int& a) {
    tok = s.span.first + row / p.ratio;
    a = s.head * p.ratio + row % p.ratio;
    return static_cast<T*>(p.q.out_dev) + tok * p.q.out_token_stride + a * p.q.out_head_stride;
}
__device__ __forceinline__ void write_lse(const AttnParams& p, int tok, int a, float m, float l) {
    if (p.q.lse_dev != nullptr)
        p.q.lse_dev[static_cast<int64_t>(tok) * p.q.heads_q + a] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// Joins partials part(0) .. part(n - 1) of a segment, in order, by the whole CTA, into the output (dst null) or a partial.
// val(i, x) is float x of partial i.
template <typename T, int D, int G, int NT, typename Val>
__device__ __forceinline__ void join(const AttnParams& p, const Segment& s, int n, Val val, float* dst) {
    using S = AttnShape<D, G, NT>;
    for (int e = threadIdx.x; e < S::kRows * D; e += S::kThreads) {
        const int row = e / D, d = e % D;
        if (s.row0 + row >= s.span.n * p.ratio) continue;
        float m = -INFINITY;
        for (int i = 0; i < n; ++i) m = fmaxf(m, val(i, S::kRows * S::kPitch + row));
        float o = 0.0f, l = 0.0f;
        for (int i = 0; i < n; ++i) {
            const float mi = val(i, S::kRows * S::kPitch + row), li = val(i, S::kRows * S::kPitch + S::kRows + row);
            const float f = mi == -INFINITY ? (li == 0.0f ? 0.0f : 1.0f) : exp2_approx(mi - m);
            o = fmaf(val(i, row * S::kPitch + d), f, o);
            l = fmaf(li, f, l);
        }
        if (dst != nullptr) {
            dst[row * S::kPitch + d] = o;
            if (d == 0) dst[S::kRows * S::kPitch + row] = m, dst[S::kRows * S::kPitch + S::kRows + row] = l;
        } else {
            int tok, a;
            T* out = out_row<T>(p, s, s.row0 + row, tok, a);
            out[d] = from_f32<T>(l == 0.0f ? 0.0f : o / l);
            if (d == 0) write_lse(p, tok, a, m, l);
        }
    }
}

template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(AttnShape<D, G, NT>::kThreads, 1) decode_kernel(const AttnParams p) {
    using S = AttnShape<D, G, NT>;
    constexpr int kWords = S::kPanel / 32;   // 32-bit words of a K row and panel a lane holds
    constexpr int kMt = D / 16;              // 16-dim tiles of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_before[S::kThreads];
    __shared__ int64_t s_warp[S::kWarps];
    __shared__ __align__(8) uint64_t s_bar[S::kWarps][S::kStages];
    __shared__ Segment s_seg[2 * S::kWarps];  // of each warp's first and last partial
    __shared__ int s_has[2 * S::kWarps];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(&s_bar[warp][i], 1);
        mbar_fence_init();
        s_has[2 * warp] = s_has[2 * warp + 1] = 0;
    }
    pdl_launch_dependents();
    pdl_wait();

    // Tiles of every request; thread x has requests [x * run, (x + 1) * run).
    const int run = (p.q.n_req + S::kThreads - 1) / S::kThreads;
    const auto tiles_of = [&](const Span& s) {
        int64_t n = 0;
        for (int row0 = 0; row0 < s.n * p.ratio; row0 += S::kRows) n += keys_of(p, s, row0, S::kRows).tiles;
        return n * p.heads;
    };
    int64_t mine = 0;
    for (int r = tid * run; r < min((tid + 1) * run, p.q.n_req); ++r) mine += tiles_of(span_of(p, r));
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t total = 0, before = incl - mine;
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    s_before[tid] = before;
    __syncthreads();
    // A CTA takes a tile a warp at least: with little work fewer CTAs have less to join.
    const int64_t ctas = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), (total + S::kWarps - 1) / S::kWarps));
    if (blockIdx.x >= ctas || total == 0) return;
    const int64_t cta0 = blockIdx.x * total / ctas, cta1 = (blockIdx.x + 1) * total / ctas;
    const int64_t begin = cta0 + warp * (cta1 - cta0) / S::kWarps, end = cta0 + (warp + 1) * (cta1 - cta0) / S::kWarps;

    float* const scratch = reinterpret_cast<float*>(static_cast<uint8_t*>(p.q.workspace_dev) + 4096);
    float* const slots = scratch + static_cast<int64_t>(gridDim.x) * S::kWarps * S::kPartial;  // two a CTA
    int* const arrived = static_cast<int*>(p.q.workspace_dev);

    uint8_t* const ring = smem + warp * S::kStages * S::kStageBytes;
    Segment seg;
    int at = 0;           // tile of the segment
    uint32_t turn = 0;    // tiles this warp has waited for
    bool dead = false;    // a copy never came
    if (begin < end) {
        int lo = 0, hi = min(S::kThreads, (p.q.n_req + run - 1) / run) - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_before[mid] <= begin) lo = mid; else hi = mid - 1;
        }
        seg.start = s_before[lo];
        seg.r = lo * run;
        for (;; ++seg.r) {
            seg.span = span_of(p, seg.r);
            const int64_t n = tiles_of(seg.span);
            if (begin < seg.start + n) break;
            seg.start += n;
        }
        for (seg.row0 = 0;; seg.row0 += S::kRows) {
            seg.keys = keys_of(p, seg.span, seg.row0, S::kRows);
            const int64_t n = static_cast<int64_t>(seg.keys.tiles) * p.heads;
            if (begin < seg.start + n) break;
            seg.start += n;
        }
        seg.head = static_cast<int>((begin - seg.start) / seg.keys.tiles);
        seg.start += static_cast<int64_t>(seg.head) * seg.keys.tiles;
        at = static_cast<int>(begin - seg.start);
    }

    for (int64_t tile = begin; tile < end;) {
        const int stop = static_cast<int>(min(static_cast<int64_t>(seg.keys.tiles), at + (end - tile)));
        const int old = seg.span.len - seg.span.n;
        const uint8_t* const base = p.cache + seg.head * p.head_bytes;
        const int32_t* const table = p.q.table_dev + seg.r * p.q.table_stride;

        // Page ids of the next 32 subtiles, one a lane; -1 past the keys, -2 for one outside the cache.
        int ids = -1, ids_at = at - 16;
        uint32_t bad = 0;  // two bits a stage: subtiles whose page is outside the cache
        const auto issue = [&](int k, uint32_t stage) {
            if (k >= ids_at + 16) {
                ids_at = k;
                const int pos = seg.keys.lo + 16 * (2 * k + lane);
                ids = -1;
                if (pos < seg.keys.hi) {
                    ids = table[pos >> p.log2_page];
                    if (ids < 0 || ids >= p.n_pages) {
                        report(p.status, SGEMV_ERR_ARG);
                        ids = -2;
                    }
                }
            }
            const int id = __shfl_sync(0xFFFFFFFFu, ids, 2 * (k - ids_at) + (lane & 1));
            const uint32_t want = __ballot_sync(0xFFFFFFFFu, lane < 2 && id >= 0);
            const uint32_t none = __ballot_sync(0xFFFFFFFFu, lane < 2 && id == -2);
            bad = (bad & ~(3u << (2 * stage))) | (none << (2 * stage));
            if (lane == 0) mbar_arrive_expect_tx(&s_bar[warp][stage], __popc(want) * S::kSubBytes);
            __syncwarp();
            if (lane < 2 && id >= 0) {
                const int pos = seg.keys.lo + 16 * (2 * k + lane);
                bulk_g2s(ring + stage * S::kStageBytes + lane * S::kSubBytes,
                         base + id * p.page_bytes + ((pos & (p.page - 1)) >> 4) * S::kSubBytes, S::kSubBytes, &s_bar[warp][stage]);
            }
        };
        for (int k = 0; k < S::kStages && at + k < stop && !dead; ++k) issue(at + k, (turn + k) % S::kStages);

        // Queries: lane (g, t) holds dims 32 t .. 32 t + 31 of each panel of row g (16 t .. where a panel has 64), scaled by a
        // power of two that brings the row's largest into [2^9, 2^10); xs = sums over a group's dims.
        uint32_t qb[NT][S::kPanels][2 * kWords][2];
        float c[NT][2], xs[S::kGroups][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = seg.row0 + 8 * nt + g;
            const bool live = row < seg.span.n * p.ratio;
            const T* x = static_cast<const T*>(p.q.q_dev);
            if (live) x += (seg.span.first + row / p.ratio) * p.q.q_token_stride + (seg.head * p.ratio + row % p.ratio) * p.q.q_head_stride;
            uint4 raw[S::kPanels][kWords];
            float big = 0.0f;
#pragma unroll
            for (int pn = 0; pn < S::kPanels; ++pn)
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    raw[pn][w] = live ? *reinterpret_cast<const uint4*>(x + pn * 128 + 8 * (kWords * t + w)) : make_uint4(0, 0, 0, 0);
                    const T* h = reinterpret_cast<const T*>(&raw[pn][w]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(to_f32(h[j])));
                }
            big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
            const int be = static_cast<int>(__float_as_uint(big) >> 23);  // biased exponent; 0 and infinity are left alone
            const int sh = be == 0 || be == 255 ? 0 : min(max(127 + 9 - be, -100), 100);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
            float sum[S::kPanels];
#pragma unroll
            for (int pn = 0; pn < S::kPanels; ++pn) {
                sum[pn] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const T* h = reinterpret_cast<const T*>(&raw[pn][w]);
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = to_f32(h[j]) * up;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t e = pack_half2(f[2 * j], f[2 * j + 4]);
                        const uint32_t o = pack_half2(f[2 * j + 1] * 0.0625f, f[2 * j + 5] * 0.0625f);
                        qb[nt][pn][2 * w + j][0] = e;
                        qb[nt][pn][2 * w + j][1] = o;
                        const float2 fe = unpack_half2(e), fo = unpack_half2(o);
                        sum[pn] += (fe.x + fe.y) + 16.0f * (fo.x + fo.y);
                    }
                }
                sum[pn] += __shfl_xor_sync(0xFFFFFFFFu, sum[pn], 1);
                if (!S::kSplit) sum[pn] += __shfl_xor_sync(0xFFFFFFFFu, sum[pn], 2);
                sum[pn] *= 1.0f / kTwo24;
            }
            // from rows (g) to the columns 2t, 2t + 1 of the products
            const float down = p.scale_log2 * kTwo24 / up;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                c[nt][j] = __shfl_sync(0xFFFFFFFFu, down, 4 * (2 * t + j));
#pragma unroll
                for (int pn = 0; pn < S::kPanels; ++pn) {
                    if constexpr (S::kSplit) {
                        xs[2 * pn][nt][j] = __shfl_sync(0xFFFFFFFFu, sum[pn], 4 * (2 * t + j));
                        xs[2 * pn + 1][nt][j] = __shfl_sync(0xFFFFFFFFu, sum[pn], 4 * (2 * t + j) + 2);
                    } else {
                        xs[pn][nt][j] = __shfl_sync(0xFFFFFFFFu, sum[pn], 4 * (2 * t + j));
                    }
                }
            }
        }

        float o[kMt][NT][4], l[NT][2], zp[S::kGroups][NT][2], m[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < kMt; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[nt][j] = 0.0f, m[nt][j] = -INFINITY;
#pragma unroll
                for (int gr = 0; gr < S::kGroups; ++gr) zp[gr][nt][j] = 0.0f;
            }
        }
        // positions that every row of the segment sees
        const int i0 = seg.row0 / p.ratio, i1 = min(seg.row0 + S::kRows - 1, seg.span.n * p.ratio - 1) / p.ratio;
        const int clear1 = p.q.tree_dev != nullptr ? old : old + i0 + 1;
        const int clear0 = p.q.window > 0 ? old + i1 - p.q.window + 1 : 0;
        const int ta = 4 * (g >> 1) + (g & 1);  // the token of row g of S^T; row g + 8 is token ta + 2

        for (int k = at; k < stop; ++k, ++turn) {
            const uint32_t stage = turn % S::kStages;
            if (!dead && !mbar_wait(&s_bar[warp][stage], (turn / S::kStages) & 1)) {
                report(p.status, SGEMV_ERR_TIMEOUT);
                dead = true;
            }
            dead = __any_sync(0xFFFFFFFFu, dead);
            const uint8_t* const buf = ring + stage * S::kStageBytes;
            const int pos0 = seg.keys.lo + k * kTileTok;
            const bool plain = pos0 >= clear0 && pos0 + kTileTok <= clear1 && ((bad >> (2 * stage)) & 3u) == 0;

            float sc[2][NT][4];   // scores: before c, then in log2
            float vs[2][S::kGroups][2], vz[2][S::kGroups][2];  // of the lane's tokens ta, ta + 2: scale x 64, zero point
            float ve[2][2];       // exponent of the largest scale of V
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* const sub = buf + u * S::kSubBytes;
                // a token past the keys, or in a page outside the cache, may hold anything: s = 1, z = 0 for it
                bool gone[2] = {false, false};
                if (!plain) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        gone[e] = pos0 + 16 * u + ta + 2 * e >= seg.keys.hi || ((bad >> (2 * stage + u)) & 1u);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ve[u][e] = -100.0f;
#pragma unroll
                    for (int gr = 0; gr < S::kGroups; ++gr) {
                        uint32_t w = *reinterpret_cast<const uint32_t*>(sub + 16 * D + 64 * S::kGroups + 64 * gr + 4 * (ta + 2 * e));
                        if (!plain && gone[e]) w = 0x00003C00u;
                        const float2 f = unpack_half2(w);
                        vs[u][gr][e] = f.x * kWeightScale;
                        vz[u][gr][e] = f.y;
                        ve[u][e] = fmaxf(ve[u][e], static_cast<float>(static_cast<int>((w & 0x7C00u) >> 10) - 15));
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[u][nt][j] = 0.0f;
#pragma unroll
                for (int pn = 0; pn < S::kPanels; ++pn) {
                    uint32_t ka[kWords], kb[kWords];
                    const uint8_t* const ra = sub + pn * 1024 + ta * (S::kPanel / 2) + 4 * kWords * t;
                    if constexpr (kWords == 4) {
                        *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(ra);
                        *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(ra + S::kPanel);
                    } else {
                        *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(ra);
                        *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(ra + S::kPanel);
                    }
                    constexpr int kSets = S::kSplit ? 2 : 1;
                    float acc[kSets][NT][4];
#pragma unroll
                    for (int h = 0; h < kSets; ++h)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[h][nt][j] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a = h ? ka[w] >> 8 : ka[w], b = h ? kb[w] >> 8 : kb[w];
                            const uint32_t a0 = a & 0x000F000Fu, a1 = b & 0x000F000Fu, a2 = a & 0x00F000F0u, a3 = b & 0x00F000F0u;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t b0 = qb[nt][pn][2 * w + h][0], b1 = qb[nt][pn][2 * w + h][1];
                                if constexpr (S::kSplit) {  // lanes t = 0, 1 hold the first group's dims, 2 and 3 the second's
                                    const uint32_t m0 = t < 2 ? 0xFFFFFFFFu : 0u;
                                    mma16816(acc[0][nt], a0, a1, a2, a3, b0 & m0, b1 & m0);
                                    mma16816(acc[1][nt], a0, a1, a2, a3, b0 & ~m0, b1 & ~m0);
                                } else {
                                    mma16816(acc[0][nt], a0, a1, a2, a3, b0, b1);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < kSets; ++h) {
                        const int gr = kSets * pn + h;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 f = unpack_half2(*reinterpret_cast<const uint32_t*>(sub + 16 * D + 64 * gr + 4 * (ta + 2 * e)));
                            const float sz = f.x * f.y;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    sc[u][nt][2 * e + j] += fmaf(f.x, acc[h][nt][2 * e + j], -sz * xs[gr][nt][j]);
                        }
                    }
                }
            }
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    top[nt][j] = -INFINITY;
                    const int row = seg.row0 + 8 * nt + 2 * t + j;
                    int last = 0, first = 0;
                    uint64_t tree = 0;
                    if (!plain) {
                        const int i = min(row, seg.span.n * p.ratio - 1) / p.ratio;
                        last = old + i;
                        if (p.q.window > 0) first = last - p.q.window + 1;
                        if (p.q.tree_dev != nullptr) tree = p.q.tree_dev[seg.span.first + i];
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& x = sc[u][nt][2 * e + j];
                            x *= c[nt][j];
                            if (!plain) {
                                const int pos = pos0 + 16 * u + ta + 2 * e;
                                bool see = pos < seg.keys.hi && !((bad >> (2 * stage + u)) & 1u);
                                if (p.q.tree_dev != nullptr) see = see && (pos < old || ((tree >> (pos - old)) & 1));
                                else see = see && pos >= first && pos <= last;
                                if (!see) x = -INFINITY;
                            }
                            top[nt][j] = fmaxf(top[nt][j], x + ve[u][e]);
                        }
                }
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) grow = grow || top[nt][j] > m[nt][j] + kMaxGrowth;
            if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = top[nt][j];
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                        x = fmaxf(x, m[nt][j]);
                        const float f = x == -INFINITY ? 1.0f : exp2_approx(m[nt][j] - x);
                        m[nt][j] = x;
                        l[nt][j] *= f;
#pragma unroll
                        for (int gr = 0; gr < S::kGroups; ++gr) zp[gr][nt][j] *= f;
#pragma unroll
                        for (int i = 0; i < kMt; ++i) o[i][nt][j] *= f, o[i][nt][2 + j] *= f;
                    }
            }
            // weights, rounded to fp16 per group of V, and the second product
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* const sub = buf + u * S::kSubBytes + 8 * D;
                uint32_t pb[S::kGroups][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float ref = m[nt][j] == -INFINITY ? 0.0f : m[nt][j];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& x = sc[u][nt][2 * e + j];
                            x = exp2_approx(x - ref);
                            l[nt][j] += x;
                        }
                    }
#pragma unroll
                    for (int gr = 0; gr < S::kGroups; ++gr)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t w = pack_half2(sc[u][nt][2 * e] * vs[u][gr][e], sc[u][nt][2 * e + 1] * vs[u][gr][e]);
                            const float2 f = unpack_half2(w);
                            zp[gr][nt][0] = fmaf(f.x, vz[u][gr][e], zp[gr][nt][0]);
                            zp[gr][nt][1] = fmaf(f.y, vz[u][gr][e], zp[gr][nt][1]);
                            pb[gr][nt][e] = transpose8x8(w);
                        }
                }
                uint32_t vw[D / 16];
#pragma unroll
                for (int r = 0; r < D / 64; ++r)
                    *reinterpret_cast<uint4*>(vw + 4 * r) = *reinterpret_cast<const uint4*>(sub + 512 * r + 16 * lane);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a = h ? vw[i] >> 8 : vw[i], b = h ? vw[D / 32 + i] >> 8 : vw[D / 32 + i];
                        const uint32_t a0 = a & 0x000F000Fu, a1 = a & 0x00F000F0u, a2 = b & 0x000F000Fu, a3 = b & 0x00F000F0u;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[2 * i + h][nt], a0, a1, a2, a3, pb[32 * i / G][nt][0], pb[32 * i / G][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (k + S::kStages < stop && !dead) issue(k + S::kStages, stage);
        }

        // the lanes' sums over their tokens
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], d);
#pragma unroll
                    for (int gr = 0; gr < S::kGroups; ++gr) zp[gr][nt][j] += __shfl_xor_sync(0xFFFFFFFFu, zp[gr][nt][j], d);
                }
            }
        const bool whole = at == 0 && stop == seg.keys.tiles;
        const bool to_first = !whole && stop == seg.keys.tiles && tile + (stop - at) < end;  // more segments follow
        float* const mine_p = to_first ? scratch + (static_cast<int64_t>(blockIdx.x) * S::kWarps + warp) * S::kPartial
                                       : reinterpret_cast<float*>(smem) + warp * S::kPartial;
        if (!whole && !to_first) named_bar_sync(1, S::kThreads);  // every warp is done with its ring: partials go there
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int n = 8 * nt + 2 * t + j, row = seg.row0 + n;
                const bool live = row < seg.span.n * p.ratio;
                int tok = 0, a = 0;
                T* out = nullptr;
                if (whole && live) out = out_row<T>(p, seg, row, tok, a);
                const float inv = l[nt][j] == 0.0f ? 0.0f : 1.0f / l[nt][j];
#pragma unroll
                for (int i = 0; i < kMt; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = 16 * i + 8 * e + g;
                        const float v = (o[i][nt][2 * e + j] * (e ? kTwo20 : kTwo24) - zp[16 * i / G][nt][j]) * (1.0f / kWeightScale);
                        if (!whole) mine_p[n * S::kPitch + d] = v;
                        else if (live) out[d] = from_f32<T>(v * inv);
                    }
                if (g == 0) {
                    if (!whole) mine_p[S::kRows * S::kPitch + n] = m[nt][j], mine_p[S::kRows * S::kPitch + S::kRows + n] = l[nt][j];
                    else if (live) write_lse(p, tok, a, m[nt][j], l[nt][j]);
                }
            }
        if (!whole && lane == 0) {
            const int slot = 2 * warp + (to_first ? 0 : 1);
            s_has[slot] = 1;
            s_seg[slot] = seg;
        }
        if (!whole && !to_first) break;  // the warp's last segment, and the barrier is behind it
        tile += stop - at;
        at = 0;
        if (tile < end) {
            seg.start += seg.keys.tiles;
            if (++seg.head == p.heads) {
                seg.head = 0;
                seg.row0 += S::kRows;
                while (seg.row0 >= seg.span.n * p.ratio) {
                    seg.span = span_of(p, ++seg.r);
                    seg.row0 = 0;
                }
                seg.keys = keys_of(p, seg.span, seg.row0, S::kRows);
            }
        } else {
            named_bar_sync(1, S::kThreads);  // the same barrier, for a warp that ends with a whole segment
        }
    }
    if (begin >= end) named_bar_sync(1, S::kThreads);  // and for one that had no tile
    __syncthreads();

    // Join the partials of each segment that this CTA's warps share, in the order of the warps.
    for (int i = 0; i < 2 * S::kWarps;) {
        if (!s_has[i]) {
            ++i;
            continue;
        }
        const Segment s = s_seg[i];
        int idx[2 * S::kWarps], n = 0;
        for (; i < 2 * S::kWarps && (!s_has[i] || s_seg[i].start == s.start); ++i)
            if (s_has[i]) idx[n++] = i;
        const auto part = [&](int x, int at) {
            const float* q = (idx[x] & 1) ? reinterpret_cast<const float*>(smem) + (idx[x] >> 1) * S::kPartial
                                          : scratch + (static_cast<int64_t>(blockIdx.x) * S::kWarps + (idx[x] >> 1)) * S::kPartial;
            return q[at];
        };
        const int64_t s_end = s.start + s.keys.tiles;
        if (s.start >= cta0 && s_end <= cta1) {
            join<T, D, G, NT>(p, s, n, part, nullptr);
            continue;
        }
        const auto slot = [&](int64_t cta, bool tail) { return slots + (2 * cta + (tail ? 1 : 0)) * S::kPartial; };
        join<T, D, G, NT>(p, s, n, part, slot(blockIdx.x, s.start >= cta0));
        __threadfence();
        __syncthreads();
        const int64_t from = ((s.start + 1) * ctas - 1) / total, to = (s_end * ctas - 1) / total;
        if (tid == 0) s_last = atomicAdd(&arrived[from], 1) == static_cast<int>(to - from);
        __syncthreads();
        if (s_last) {
            __threadfence();
            join<T, D, G, NT>(p, s, static_cast<int>(to - from + 1), [&](int x, int at) { return __ldcg(slot(from + x, x == 0) + at); }, nullptr);
            if (tid == 0) arrived[from] = 0;
        }
        __syncthreads();
    }
}

}  // namespace sgemv
