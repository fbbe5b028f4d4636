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
// operands, no conversion. The powers of two are taken up by x (odd dims are divided by 16, each row is scaled into fp16's range by a
// power of two of its own: exact but for elements below 2^-29 of the row's largest, 2^-25 in odd dims) and by the epilogue.
//
// Both products are computed transposed, S^T = K x^T and O^T = V^T P^T, so that the cache is the 16-row operand of
// mma.m16n8k16 and 8 rows of queries (query heads of a KV head x new tokens) the narrow one: with few rows this is half the
// tensor work of the usual orientation, and the weights become the second product's operand with one movmatrix per 8 x 8.
//
// out = 0 and lse = -inf where a row sees nothing; a masked key's weight is set to 0. What lies past the keys or in a page outside
// the cache may hold scales that are not numbers: they are replaced before a tile that reaches there is read.
//
// Work: the 32-token tiles of all (request, row tile, head) segments form one list, split evenly over the CTAs and
// again over their warps, whatever the lengths (a segment counts kSwitch tiles more than it has). A warp copies its
// tiles (two 16-token subtiles, contiguous in the cache) into a ring of its own with the copy engine, running ahead across
// segments, and keeps the softmax's reference, sum and O in registers. Segments that cross warps are joined in shared
// memory, those that cross CTAs through the workspace by the last CTA to arrive, always in the order of the keys: the
// same inputs give the same bits.
//
// Measured: a longer context costs its bytes at 6.9 TB/s (8 KV heads of 128; a plain copy has 6.7), and a call that gives every SM
// work 15 to 19 us besides: 7 us up to the first tile (lengths, the split, block tables, and then all SMs' rings fill at once, 20 MB),
// 5 to 8 us after the last (joins, an arrival, joins across CTAs). These are short steps that wait for one another and run once,
// so that their instructions come from L2 too: going through the join once beforehand, to have them near, cost more than it
// saved (single 9.3 -> 10.3 us). 64 requests of up to 16384 tokens (571 MB): 98 us; one of 262144 (285 MB): 60 us; one
// of 333 with 32 heads: 9.5 us; 24 trees of 12 tokens, 48 rows a head of 64: 23 us, half of it the products; the first of them
// with a window of 4096 (251 MB): 52 us.
#pragma once

#include "kv_common.cuh"

namespace sgemv {

constexpr int kTileTok = 32;      // tokens of a tile
constexpr int kMaxLen = 1 << 30;  // positions past the end of a tile stay in 32 bits
// Weights 2^(t - m) s' go into fp16: the largest is 2^kTop when the reference m is set, and m is set anew when one would pass
// 2^kLimit (fp16 ends at 2^16). Weights below 2^(kTop - 20) of the largest lose bits, as fp16 subnormals.
constexpr float kTop = 6.0f, kLimit = 15.0f;
constexpr int kSwitch = 4;  // what taking up a segment costs, in tiles: counted when the work is split (1: 114 us, 2: 107, 3: 104.3, 4: 104.7
                            // for a batch of 64 requests of 1 to 16384 keys; one request of 262144: 65.0 with 3, 64.1 with 4)
constexpr int kMaxCtas = 152; // CTAs that the workspace has room for
constexpr int kSpans = 256; // requests whose lengths are kept in shared memory

struct AttnParams {
    const uint8_t* cache;
    uint64_t sub_bytes, head_bytes, page_bytes;
    sgemv_kv_query q;
    int32_t* status;
    int heads, page, log2_page, n_pages, ratio;
    int log2_ratio;    // -1 where ratio is not a power of two
    int max_rows;      // requests with more rows a KV head are the chunk kernel's
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
    // 12 warps have 168 registers a thread: the 128 of 16 warps spilled (104.3 against 102.6 us for the batch of 64 requests).
    static constexpr int kWarps = (D == 256 || (NT > 1 && D > 64)) ? 8 : 12;
    static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;             // floats of a partial row: 4 more so that two rows are 8 banks apart
    static constexpr int kPartial = kRows * kPitch + 2 * kRows;  // floats of a partial: O, then m, then l
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kSmem = kRing + kWarps * kPartial * 4;  // the rings, then a partial a warp
    // With at most so many tiles in all, a CTA's part of the list starts where a segment starts, if that segment has at
    // most kShortSegment tiles: a join across CTAs costs more than it brings.
    static constexpr int kFewTiles = 2 * kWarps, kShortSegment = 2 * kWarps;
};

// Token of a row of a request, and its query head among those of the KV head.
__device__ __forceinline__ int token_of_row(const AttnParams& p, int row) {
    return p.log2_ratio >= 0 ? row >> p.log2_ratio : row / p.ratio;
}
__device__ __forceinline__ int head_of_row(const AttnParams& p, int row) { return row - token_of_row(p, row) * p.ratio; }

// a / b, a >= 0, b > 0; a 64-bit division costs several times a 32-bit one.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

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

// The same for the decode kernel.
__device__ __forceinline__ Span decode_span(const AttnParams& p, int r) {
    Span s = span_of(p, r);
    if (static_cast<int64_t>(s.n) * p.ratio > p.max_rows) s.n = 0;
    return s;
}

// The keys of rows [row0, row0 + rows) of a request: where the first tile starts, in the page of the first key that a row sees (pages
// before it may be free) and where a page's copies start, and the end.
struct Keys {
    int lo, hi, tiles;
};

template <int kTile>
__device__ __forceinline__ Keys keys_of(const AttnParams& p, const Span& s, int row0, int rows) {
    const int i0 = token_of_row(p, row0), i1 = token_of_row(p, min(row0 + rows - 1, s.n * p.ratio - 1));
    const int old = s.len - s.n;
    Keys k;
    k.hi = p.q.tree_dev != nullptr ? s.len : max(0, old + i1 + 1);
    k.lo = p.q.window > 0 ? max(0, old + i0 - p.q.window + 1) & -min(p.page, kTile) : 0;
    k.tiles = max(1, (k.hi - k.lo + kTile - 1) / kTile);  // rows that see nothing still have an owner
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
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

constexpr uint32_t kLeast = 1;  // scale 2^-24, zero point 0
constexpr float kTwo24 = 16777216.0f, kTwo20 = 1048576.0f;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }  // -126 <= e <= 127
// The power of two that brings a row's largest element into [2^15, 2^16), fp16's last binade, or as near as a binary32 factor can.
__device__ __forceinline__ int query_shift(float big) { return min(127 + 15 - static_cast<int>(__float_as_uint(big) >> 23), 126); }

// Writes row R (of its request) of a finished segment: dims and logarithm of the sum.
template <typename T>
__device__ __forceinline__ T* out_row(const AttnParams& p, const Segment& s, int row, int& tok, int& a) {
    tok = s.span.first + token_of_row(p, row);
    a = s.head * p.ratio + head_of_row(p, row);
    return static_cast<T*>(p.q.out_dev) + tok * p.q.out_token_stride + a * p.q.out_head_stride;
}
__device__ __forceinline__ void write_lse(const AttnParams& p, int tok, int a, float m, float l) {
    if (p.q.lse_dev != nullptr)
        p.q.lse_dev[static_cast<int64_t>(tok) * p.q.heads_q + a] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// Joining n partials of a row, in order: 4 dims a thread, which forms the reference and what each partial counts, 2^(its
// reference - the joint one), for itself. So a join is as long as its loads, and kFlight partials' are under way at once. (With the
// weights formed first, by a warp a row, the join across CTAs took 14000 to 20000 cycles, mostly waiting for one load after another.)
__device__ __forceinline__ float join_weight(float mi, float li, float m) {
    return mi == -INFINITY ? (li == 0.0f ? 0.0f : 1.0f) : exp2_approx(mi - m);  // (1: li is not a number, and shows)
}
// get(i, m, l, x): partial i's reference, sum and 4 dims.
template <int kFlight, typename Get>
__device__ __forceinline__ float4 join(int n, Get get, float& m, float& l) {
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kFlight) {
        float mi[kFlight], li[kFlight];
        float4 x[kFlight];
        float top = m;
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            mi[j] = -INFINITY, li[j] = 0.0f, x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i0 + j < n) get(i0 + j, mi[j], li[j], x[j]);
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j) top = fmaxf(top, mi[j]);
        const float before = join_weight(m, l, top);
        m = top;
        l *= before, o.x *= before, o.y *= before, o.z *= before, o.w *= before;
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const float f = join_weight(mi[j], li[j], top);
            l = fmaf(li[j], f, l);
            o.x = fmaf(x[j].x, f, o.x);
            o.y = fmaf(x[j].y, f, o.y);
            o.z = fmaf(x[j].z, f, o.z);
            o.w = fmaf(x[j].w, f, o.w);
        }
    }
    return o;
}
// 4 dims of a finished row of the output; the first of them writes the row's lse.
template <typename T>
__device__ __forceinline__ void write_quad(const AttnParams& p, T* out, int d, float4 o, float m, float l, int tok, int a) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const T h[4] = {from_f32<T>(o.x * inv), from_f32<T>(o.y * inv), from_f32<T>(o.z * inv), from_f32<T>(o.w * inv)};
    *reinterpret_cast<uint2*>(out + d) = *reinterpret_cast<const uint2*>(h);
    if (d == 0) write_lse(p, tok, a, m, l);
}
// The join of a decode row, into the output (dst null) or a partial.
template <typename T, int D, int G, int NT, int kFlight, typename Get>
__device__ __forceinline__ void join_quad(const AttnParams& p, const Segment& s, int row, int d, int n, Get get, float* dst) {
    using S = AttnShape<D, G, NT>;
    constexpr int kM = S::kRows * S::kPitch, kL = kM + S::kRows;
    float m, l;
    const float4 o = join<kFlight>(n, get, m, l);
    if (dst != nullptr) {
        *reinterpret_cast<float4*>(dst + row * S::kPitch + d) = o;
        if (d == 0) dst[kM + row] = m, dst[kL + row] = l;
    } else {
        int tok, a;
        T* const out = out_row<T>(p, s, s.row0 + row, tok, a);
        write_quad(p, out, d, o, m, l, tok, a);
    }
}

// Tiles of a request (all its segments), with what taking each up costs.
template <int kRows>
__device__ __forceinline__ int64_t units_of(const AttnParams& p, const Span& s) {
    int64_t n = 0;
    for (int row0 = 0; row0 < s.n * p.ratio; row0 += kRows) n += keys_of<kTileTok>(p, s, row0, kRows).tiles + kSwitch;
    return n * p.heads;
}

// The requests' lengths, from shared memory where they fit.
struct Spans {
    const AttnParams& p;
    const Span* cached;  // of every request, or null
    __device__ __forceinline__ Span operator[](int r) const { return cached != nullptr ? cached[r] : decode_span(p, r); }
};

// The segment after s (there is one).
template <int kRows>
__device__ __forceinline__ void next_segment(const AttnParams& p, const Spans& spans, Segment& s) {
    s.start += s.keys.tiles + kSwitch;
    if (++s.head < p.heads) return;
    s.head = 0;
    s.row0 += kRows;
    while (s.row0 >= s.span.n * p.ratio) {
        s.span = spans[++s.r];
        s.row0 = 0;
    }
    s.keys = keys_of<kTileTok>(p, s.span, s.row0, kRows);
}

// The segment that holds a unit. before: units before each thread's run of requests.
template <int kRows>
__device__ __forceinline__ Segment locate(const AttnParams& p, const Spans& spans, const int64_t* before, int runs, int run, int64_t unit) {
    int lo = 0, hi = runs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= unit) lo = mid; else hi = mid - 1;
    }
    Segment s;
    s.start = before[lo];
    for (s.r = lo * run;; ++s.r) {
        s.span = spans[s.r];
        if (run == 1) break;
        const int64_t n = units_of<kRows>(p, s.span);
        if (unit < s.start + n) break;
        s.start += n;
    }
    for (s.row0 = 0;; s.row0 += kRows) {
        s.keys = keys_of<kTileTok>(p, s.span, s.row0, kRows);
        const int64_t n = static_cast<int64_t>(s.keys.tiles + kSwitch) * p.heads;
        if (unit < s.start + n) break;
        s.start += n;
    }
    s.head = static_cast<int>(quotient(unit - s.start, s.keys.tiles + kSwitch));
    s.start += static_cast<int64_t>(s.head) * (s.keys.tiles + kSwitch);
    return s;
}

// The copies of one warp: a ring of stages, filled tile by tile along the warp's part of the list.
template <int D, int G, int NT>
struct Producer {
    using S = AttnShape<D, G, NT>;
    Segment* seg;          // shared memory, one a warp
    uint64_t* bar;
    uint8_t* ring;
    int k, to;             // next tile of the segment, and where the warp's part of it ends
    int at;                // first tile of the copies that the lanes hold
    const uint8_t* src;    // this lane's copy of those, its bytes, and what its tile's copies bring
    uint32_t bytes, tx;
    uint32_t wrong;        // lanes whose page is outside the cache
    uint32_t bad;          // two bits a stage: subtiles whose page is outside the cache
    bool done;

    // Copies the next tile into `stage`, by the whole warp: one copy where a page holds the tile's two subtiles, else two.
    __device__ __forceinline__ void issue(const AttnParams& p, const Spans& spans, uint32_t stage, int64_t end, int lane) {
        if (done) return;
        if (k >= to) {
            Segment s = *seg;
            if (end <= s.start + kSwitch + s.keys.tiles + kSwitch) {
                done = true;
                return;
            }
            next_segment<S::kRows>(p, spans, s);
            __syncwarp();
            if (lane == 0) *seg = s;
            __syncwarp();
            k = 0;
            to = static_cast<int>(min(static_cast<int64_t>(s.keys.tiles), end - s.start - kSwitch));
            at = -64;
        }
        const int two = p.page == kSub;  // a copy a subtile
        if (k >= at + (32 >> two)) {  // the next 32 copies, one a lane
            at = k;
            const int lo = seg->keys.lo, hi = seg->keys.hi;
            const int pos = lo + kTileTok * k + (kTileTok >> two) * lane;
            bytes = 0;
            bool out = false;
            if (pos < hi) {
                const int id = p.q.table_dev[seg->r * p.q.table_stride + (pos >> p.log2_page)];
                out = id < 0 || id >= p.n_pages;
                if (out) report(p.status, SGEMV_ERR_ARG);
                else bytes = !two && pos + kSub < hi ? S::kStageBytes : S::kSubBytes;
                src = p.cache + id * p.page_bytes + seg->head * p.head_bytes + ((pos & (p.page - 1)) >> 4) * S::kSubBytes;
            }
            const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, bytes, 1);
            tx = two ? bytes + next : bytes;
            wrong = __ballot_sync(0xFFFFFFFFu, out);
        }
        const int i = k - at;
        if ((lane >> two) == i) {
            if (!two || (lane & 1) == 0) mbar_arrive_expect_tx(bar + stage, tx);
            if (bytes) bulk_g2s(ring + stage * S::kStageBytes + (two ? (lane & 1) * S::kSubBytes : 0), src, bytes, bar + stage);
        }
        if (wrong | bad) {
            const uint32_t w = two ? (wrong >> (2 * i)) & 3u : ((wrong >> i) & 1u) * 3u;
            bad = (bad & ~(3u << (2 * stage))) | (w << (2 * stage));
        }
        ++k;
    }
};

// A V group of zeros is cached with s = 1, z = 0. The reference follows weight times scale, so that the weight of such a token would
// push what far smaller values weigh out of fp16's range, for a product that is 0. Before the reference moves for a tile, those
// of its tokens get s = 2^-24, which says the same, by a token a lane; whether one did. (Looked at in every tile: 102 us for the
// batch of 64 requests that takes 98.)
template <int D, int G>
__device__ __forceinline__ bool drop_empty_groups(uint8_t* tile, int lane) {
    uint8_t* const sub = tile + (lane >> 4) * (16 * D + 128 * (D / G));
    uint32_t* const sz = reinterpret_cast<uint32_t*>(sub + 16 * D + 64 * (D / G)) + (lane & 15);
    bool some = false;
#pragma unroll
    for (int gr = 0; gr < D / G; ++gr) some = some || sz[16 * gr] == 0x00003C00u;
    if (!__any_sync(0xFFFFFFFFu, some)) return false;
    some = false;
    const uint8_t* const v = sub + 8 * D + ((lane & 15) >> 2) * 16 + (lane & 1) * 2;
#pragma unroll 1
    for (int gr = 0; gr < D / G; ++gr) {
        uint32_t any = sz[16 * gr] ^ 0x00003C00u;
#pragma unroll 1
        for (int x = 0; x < G / 4; ++x) {  // 4 dims each
            const int i = ((lane >> 1) & 1) * (D / 32) + gr * (G / 32) + (x >> 3);
            any |= *reinterpret_cast<const uint16_t*>(v + (i >> 2) * 512 + (x & 7) * 64 + (i & 3) * 4);
        }
        if (any == 0) sz[16 * gr] = kLeast, some = true;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copy engine writes there next
    __syncwarp();
    return __any_sync(0xFFFFFFFFu, some);
}

template <typename T, int D, int G, int NT>
__global__ void __launch_bounds__(AttnShape<D, G, NT>::kThreads, 1) decode_kernel(const AttnParams p) {
    using S = AttnShape<D, G, NT>;
    constexpr int kWords = S::kPanel / 32;   // 32-bit words of a K row and panel a lane holds
    constexpr int kMt = D / 16;              // 16-dim tiles of O^T
    constexpr int kGr = S::kGroups;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_before[S::kThreads];
    __shared__ int64_t s_warp[S::kWarps];
    __shared__ __align__(8) uint64_t s_bar[S::kWarps][S::kStages];
    __shared__ Segment s_ahead[S::kWarps];    // where each warp's copies are
    __shared__ Segment s_seg[2 * S::kWarps];  // of each warp's first and last partial
    __shared__ int s_has[2 * S::kWarps], s_list[2 * S::kWarps + 1], s_first[2 * S::kWarps + 1], s_groups;
    __shared__ Span s_span[kSpans];
    __shared__ int s_parts[2], s_cta[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(&s_bar[warp][i], 1);
        mbar_fence_init();
        s_has[2 * warp] = s_has[2 * warp + 1] = 0;
    }
    pdl_launch_dependents();
    pdl_wait();

    // Units of every request; thread x has requests [x * run, (x + 1) * run).
    const int run = (p.q.n_req + S::kThreads - 1) / S::kThreads;
    int64_t mine = 0;
    for (int r = tid * run; r < min((tid + 1) * run, p.q.n_req); ++r) {
        const Span s = decode_span(p, r);
        if (r < kSpans) s_span[r] = s;
        mine += units_of<S::kRows>(p, s);
    }
    const Spans spans = {p, p.q.n_req <= kSpans ? s_span : nullptr};
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
    // With little work fewer CTAs have less to join: half a unit a warp at least, and whole segments.
    const bool few = total <= static_cast<int64_t>(S::kFewTiles) * gridDim.x;
    const int64_t ctas = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), (2 * total + S::kWarps - 1) / S::kWarps));
    if (blockIdx.x >= ctas || total == 0) return;
    const int runs = min(S::kThreads, (p.q.n_req + run - 1) / run);
    const int64_t each = quotient(total, ctas), rest = total - each * ctas;  // the first `rest` CTAs take a unit more
    const auto split = [&](int64_t cta) {  // first unit of a CTA
        int64_t u = cta * each + min(cta, rest);
        if (few && u > 0 && u < total) {
            const Segment s = locate<S::kRows>(p, spans, s_before, runs, run, u);
            if (s.keys.tiles <= S::kShortSegment) u = s.start;
        }
        return u;
    };
    const int64_t bound = split(blockIdx.x + (lane & 1));  // both ends at once
    const int64_t cta0 = __shfl_sync(0xFFFFFFFFu, bound, 0), cta1 = __shfl_sync(0xFFFFFFFFu, bound, 1);
    if (cta0 == cta1) return;
    const int64_t begin = cta0 + ((warp * (cta1 - cta0)) / S::kWarps), end = cta0 + (((warp + 1) * (cta1 - cta0)) / S::kWarps);

    float* const scratch = reinterpret_cast<float*>(static_cast<uint8_t*>(p.q.workspace_dev) + 4096);
    float* const slots = scratch + static_cast<int64_t>(gridDim.x) * S::kWarps * S::kPartial;  // two a CTA
    int* const arrived = static_cast<int*>(p.q.workspace_dev);

    Segment seg;
    int from = 0, to = 0;   // the warp's tiles of the segment
    if (begin < end) {
        seg = locate<S::kRows>(p, spans, s_before, runs, run, begin);
        from = static_cast<int>(max(static_cast<int64_t>(0), begin - seg.start - kSwitch));
        to = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(seg.keys.tiles), end - seg.start - kSwitch)));
    }
    bool more = from < to;
    // The queries of a segment, raw: row g of each 8, this lane's dims (see below).
    uint4 raw_q[NT][S::kPanels][kWords];
    const auto load_queries = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = seg.row0 + 8 * nt + g;
            const bool live = row < seg.span.n * p.ratio;
            const T* x = static_cast<const T*>(p.q.q_dev);
            if (live) x += (seg.span.first + token_of_row(p, row)) * p.q.q_token_stride + (seg.head * p.ratio + head_of_row(p, row)) * p.q.q_head_stride;
#pragma unroll
            for (int pn = 0; pn < S::kPanels; ++pn)
#pragma unroll
                for (int w = 0; w < kWords; ++w)
                    raw_q[nt][pn][w] = live ? *reinterpret_cast<const uint4*>(x + pn * 128 + 8 * (kWords * t + w)) : make_uint4(0, 0, 0, 0);
        }
    };
    bool dead = false;       // a copy never came
    uint32_t stage = 0, parity = 0;  // of the tile waited for next
    Producer<D, G, NT> ahead;
    if (more) {
        if (lane == 0) s_ahead[warp] = seg;
        __syncwarp();
        ahead.seg = &s_ahead[warp];
        ahead.bar = s_bar[warp];
        ahead.ring = smem + warp * S::kStages * S::kStageBytes;
        ahead.k = from, ahead.to = to;
        ahead.at = -64;
        ahead.src = nullptr, ahead.bytes = ahead.tx = 0;
        ahead.wrong = ahead.bad = 0;
        ahead.done = false;
        for (int i = 0; i < S::kStages; ++i) ahead.issue(p, spans, i, end, lane);
    }

    while (more) {
        const int old = seg.span.len - seg.span.n, rows = seg.span.n * p.ratio;
        load_queries();

        // Queries: lane (g, t) holds dims 32 t .. 32 t + 31 of each panel of row g (16 t .. where a panel has 64), scaled by a power of
        // two of the row's own that brings its largest into [2^15, 2^16): what a row gets depends on no other row. c: what that
        // leaves to the scores, per column (in binary32 up to rows of 2^120 or so, whose scores come near its end); nx = - sums over
        // a group's dims, per column.
        uint32_t qb[NT][S::kPanels][2 * kWords][2];
        uint64_t nx[kGr][NT], c[NT];  // pairs
        {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float big = 0.0f;
#pragma unroll
                for (int pn = 0; pn < S::kPanels; ++pn)
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        const T* h = reinterpret_cast<const T*>(&raw_q[nt][pn][w]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(to_f32(h[j])));
                    }
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                const int sh = query_shift(big);
                const float up = pow2(sh), down = pow2(-sh) * p.scale_log2;
                float sum[S::kPanels];
#pragma unroll
                for (int pn = 0; pn < S::kPanels; ++pn) {
                    sum[pn] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        const T* h = reinterpret_cast<const T*>(&raw_q[nt][pn][w]);
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
                    sum[pn] *= -1.0f / kTwo24;
                }
                // from rows (g) to the columns 2t, 2t + 1 of the products
                const auto of_column = [&](float x, int j) { return __shfl_sync(0xFFFFFFFFu, x, 8 * t + j); };
                c[nt] = pair(of_column(down, 0), of_column(down, 4));
#pragma unroll
                for (int gr = 0; gr < kGr; ++gr) {
                    const float x = sum[S::kSplit ? gr / 2 : gr];
                    const int half = S::kSplit ? 2 * (gr & 1) : 0;
                    nx[gr][nt] = pair(of_column(x, half), of_column(x, 4 + half));
                }
            }
        }

        // o: V's integers times weights. zs: V's zero points times weights. l: this lane's tokens' weights. ref: the
        // reference, and lim = ref + kLimit + what the scale adds, or -inf while nothing was seen.
        float o[kMt][NT][4], zs[kGr][NT][4], l[NT][2], ref[NT][2], lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int i = 0; i < kMt; ++i) o[i][nt][j] = 0.0f;
#pragma unroll
                for (int gr = 0; gr < kGr; ++gr) zs[gr][nt][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) l[nt][j] = 0.0f, ref[nt][j] = 0.0f, lim[nt][j] = -INFINITY;
        }
        // tiles [plain0, plain1) hold positions that every row of the segment sees
        int plain0 = 0, plain1;
        {
            const int i0 = token_of_row(p, seg.row0), i1 = token_of_row(p, min(seg.row0 + S::kRows - 1, rows - 1));
            if (p.q.window > 0) plain0 = (max(seg.keys.lo, old + i1 - p.q.window + 1) - seg.keys.lo + kTileTok - 1) / kTileTok;
            plain1 = (max(seg.keys.lo, p.q.tree_dev != nullptr ? old : old + i0 + 1) - seg.keys.lo) / kTileTok;
        }
        const int ta = 4 * (g >> 1) + (g & 1);  // the token of row g of S^T; row g + 8 is token ta + 2

        for (int k = from; k < to; ++k) {
            {
                const bool here = dead || mbar_try_wait(&s_bar[warp][stage], parity);
                if (!__all_sync(0xFFFFFFFFu, here)) {
                    const bool came = here || mbar_wait(&s_bar[warp][stage], parity);
                    if (!__all_sync(0xFFFFFFFFu, came)) {
                        report(p.status, SGEMV_ERR_TIMEOUT);
                        dead = true;
                        ahead.done = true;  // no more copies
                        // those under way land in the rings, which the joins write and the CTA leaves behind: wait for them too
#pragma unroll 1
                        for (uint32_t i = 0; i < S::kStages; ++i) {
                            const uint32_t next = stage + i;
                            mbar_wait(&s_bar[warp][next % S::kStages], parity ^ (next >= S::kStages ? 1u : 0u));
                        }
                    }
                }
            }
            const uint8_t* const buf = ahead.ring + stage * S::kStageBytes;
            const bool plain = k >= plain0 && k < plain1 && ahead.bad == 0;
            const int pos0 = seg.keys.lo + k * kTileTok;

            if (!plain) {
                // a token past the keys, or in a page outside the cache, may hold anything: s = 2^-24, z = 0 for it
                if (pos0 + lane >= seg.keys.hi || ((ahead.bad >> (2 * stage + (lane >> 4))) & 1u)) {
                    uint32_t* const w = reinterpret_cast<uint32_t*>(ahead.ring + stage * S::kStageBytes + (lane >> 4) * S::kSubBytes + 16 * D) + (lane & 15);
#pragma unroll
                    for (int gr = 0; gr < 2 * kGr; ++gr) w[16 * gr] = kLeast;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copy engine writes there next
                __syncwarp();
            }

            float sc[2][NT][4];    // t_j + log2 of the token's scale of V
            float iv[2][2];        // one over that scale, of the lane's tokens ta, ta + 2
            float fr[2][kGr][2];   // each group's scale of V over the token's largest
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* const sub = buf + u * S::kSubBytes;
                const uint8_t* const scales = sub + 16 * D + 4 * ta;
                uint32_t kw[kGr][2], vw[kGr][2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int gr = 0; gr < kGr; ++gr) {
                        kw[gr][e] = *reinterpret_cast<const uint32_t*>(scales + 64 * gr + 8 * e);
                        vw[gr][e] = *reinterpret_cast<const uint32_t*>(scales + 64 * (kGr + gr) + 8 * e);
                    }
                float lv[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = unpack_half2(vw[0][e]).x;
#pragma unroll
                    for (int gr = 1; gr < kGr; ++gr) v = fmaxf(v, unpack_half2(vw[gr][e]).x);
                    lv[e] = log2_approx(v);
                    iv[u][e] = exp2_approx(-lv[e]);
#pragma unroll
                    for (int gr = 0; gr < kGr; ++gr) fr[u][gr][e] = unpack_half2(vw[gr][e]).x * iv[u][e];
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[u][nt][j] = lv[j >> 1];
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
                            const float2 f = unpack_half2(kw[gr][e]);
                            const float ks = f.x * kTwo24;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float* const to = &sc[u][nt][2 * e];
                                // (the factor first: it need not wait for the product. With s_j (...) formed first and its factor last,
                                // the batch of 64 requests took 99.3 us where it takes 97.5, the long context 61.2 for 60)
                                const uint64_t kc = mul2(pair(ks, ks), c[nt]);
                                const uint64_t in = fma2(pair(f.y, f.y), nx[gr][nt], pair(acc[h][nt][2 * e], acc[h][nt][2 * e + 1]));
                                const float2 r = parts_of(fma2(kc, in, pair(to[0], to[1])));
                                to[0] = r.x, to[1] = r.y;
                            }
                        }
                    }
                }
            }
            if (!plain) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int i = token_of_row(p, min(seg.row0 + 8 * nt + 2 * t + j, rows - 1));
                        const int last = old + i, first = p.q.window > 0 ? last - p.q.window + 1 : 0;
                        const uint64_t tree = p.q.tree_dev != nullptr ? p.q.tree_dev[seg.span.first + i] : 0;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int pos = pos0 + 16 * u + ta + 2 * e;
                                bool see = pos < seg.keys.hi && !((ahead.bad >> (2 * stage + u)) & 1u);
                                if (p.q.tree_dev != nullptr) see = see && (pos < old || ((tree >> (pos - old)) & 1));
                                else see = see && pos >= first && pos <= last;
                                if (!see) sc[u][nt][2 * e + j] = -INFINITY;
                            }
                    }
            }
            float top[NT][2];
            const auto largest = [&] {  // of the lane's scores; whether a weight would pass the limit
                bool grow = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        top[nt][j] = fmaxf(fmaxf(fmaxf(sc[0][nt][j], sc[0][nt][2 + j]), sc[1][nt][j]), sc[1][nt][2 + j]);
                        grow = grow || top[nt][j] > lim[nt][j];
                    }
                return __any_sync(0xFFFFFFFFu, grow);
            };
            if (largest()) {
                if (drop_empty_groups<D, G>(ahead.ring + stage * S::kStageBytes, lane)) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint8_t* const at = buf + u * S::kSubBytes + 16 * D + 64 * kGr + 4 * ta + 8 * e;
                            float s[kGr], v = 0.0f;
#pragma unroll
                            for (int gr = 0; gr < kGr; ++gr) v = fmaxf(v, s[gr] = unpack_half2(*reinterpret_cast<const uint32_t*>(at + 64 * gr)).x);
                            if (fabsf(iv[u][e] - 1.0f) > 1e-4f || v >= 1.0f) continue;  // the token's largest scale was not 1, or is still
                            const float lv = log2_approx(v);
                            iv[u][e] = exp2_approx(-lv);
#pragma unroll
                            for (int gr = 0; gr < kGr; ++gr) fr[u][gr][e] = s[gr] * iv[u][e];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < 2; ++j) sc[u][nt][2 * e + j] += lv;
                        }
                    largest();
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = top[nt][j];
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                        if (x > lim[nt][j]) {  // the same in the 8 lanes of a column
                            const float f = lim[nt][j] == -INFINITY ? 1.0f : exp2_approx(ref[nt][j] - (x - kTop));
                            ref[nt][j] = x - kTop;
                            lim[nt][j] = x - kTop + kLimit;
                            l[nt][j] *= f;
#pragma unroll
                            for (int gr = 0; gr < kGr; ++gr) zs[gr][nt][j] *= f;
#pragma unroll
                            for (int i = 0; i < kMt; ++i) o[i][nt][j] *= f, o[i][nt][2 + j] *= f;
                        }
                    }
            }
            // weights, rounded to fp16 per group of V, and the second product
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* const sub = buf + u * S::kSubBytes;
                uint32_t pb[kGr][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = exp2_approx(sc[u][nt][2 * e] - ref[nt][0]), p1 = exp2_approx(sc[u][nt][2 * e + 1] - ref[nt][1]);
                        l[nt][0] = fmaf(p0, iv[u][e], l[nt][0]);
                        l[nt][1] = fmaf(p1, iv[u][e], l[nt][1]);
#pragma unroll
                        for (int gr = 0; gr < kGr; ++gr)
                            pb[gr][nt][e] = transpose8x8(kGr == 1 ? pack_half2(p0, p1) : pack_half2(p0 * fr[u][gr][e], p1 * fr[u][gr][e]));
                    }
                // zero points: every row of this product's first operand holds tokens 4t .. 4t + 3, so its sums need no joining
#pragma unroll
                for (int gr = 0; gr < kGr; ++gr) {
                    const uint4 w = *reinterpret_cast<const uint4*>(sub + 16 * D + 64 * (kGr + gr) + 16 * t);
                    const uint32_t a0 = __byte_perm(w.x, w.y, 0x7632), a2 = __byte_perm(w.z, w.w, 0x7632);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(zs[gr][nt], a0, 0, a2, 0, pb[gr][nt][0], pb[gr][nt][1]);
                }
                uint32_t vq[D / 16];
#pragma unroll
                for (int r = 0; r < D / 64; ++r)
                    *reinterpret_cast<uint4*>(vq + 4 * r) = *reinterpret_cast<const uint4*>(sub + 8 * D + 512 * r + 16 * lane);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a = h ? vq[i] >> 8 : vq[i], b = h ? vq[D / 32 + i] >> 8 : vq[D / 32 + i];
                        const uint32_t a0 = a & 0x000F000Fu, a1 = a & 0x00F000F0u, a2 = b & 0x000F000Fu, a3 = b & 0x00F000F0u;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[2 * i + h][nt], a0, a1, a2, a3, pb[32 * i / G][nt][0], pb[32 * i / G][nt][1]);
                    }
                }
            }
            __syncwarp();
            ahead.issue(p, spans, stage, end, lane);
            if (++stage == S::kStages) stage = 0, parity ^= 1;
        }

        // the lanes' sums over their tokens
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], d);
        const int64_t seg_end = seg.start + kSwitch + seg.keys.tiles;
        const bool whole = from == 0 && to == seg.keys.tiles;
        more = end > seg_end + kSwitch;  // a tile of the next segment is this warp's
        // A partial that more work follows goes to global memory, the warp's last one to its place in shared memory; rows that
        // are whole are turned there, so that they leave in full lines.
        float* const own = reinterpret_cast<float*>(smem + S::kRing) + warp * S::kPartial;
        float* const part = whole || !more ? own : scratch + (static_cast<int64_t>(blockIdx.x) * S::kWarps + warp) * S::kPartial;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int n = 8 * nt + 2 * t + j;
#pragma unroll
                for (int i = 0; i < kMt; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        part[n * S::kPitch + 16 * i + 8 * e + g] = fmaf(o[i][nt][2 * e + j], e ? kTwo20 : kTwo24, -zs[16 * i / G][nt][j]);
                if (g == 0) {
                    part[S::kRows * S::kPitch + n] = lim[nt][j] == -INFINITY ? -INFINITY : ref[nt][j];
                    part[S::kRows * S::kPitch + S::kRows + n] = l[nt][j];
                }
            }
        if (whole) {
            __syncwarp();
            constexpr int kLanes = D < 128 ? 16 : 32;  // lanes of a row
            for (int n = lane / kLanes; n < S::kRows && seg.row0 + n < rows; n += 32 / kLanes) {
                int tok, a;
                T* const out = out_row<T>(p, seg, seg.row0 + n, tok, a);
                const float sum = own[S::kRows * S::kPitch + S::kRows + n], inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int d = 4 * (lane % kLanes); d < D; d += 4 * kLanes) {
                    const float4 x = *reinterpret_cast<const float4*>(own + n * S::kPitch + d);
                    const T h[4] = {from_f32<T>(x.x * inv), from_f32<T>(x.y * inv), from_f32<T>(x.z * inv), from_f32<T>(x.w * inv)};
                    *reinterpret_cast<uint2*>(out + d) = *reinterpret_cast<const uint2*>(h);
                }
                if (lane % kLanes == 0) write_lse(p, tok, a, own[S::kRows * S::kPitch + n], sum);
            }
            __syncwarp();
        }
        if (!whole && lane == 0) {
            const int slot = 2 * warp + (more ? 0 : 1);
            s_has[slot] = 1;
            s_seg[slot] = seg;
        }
        __syncwarp();
        if (more) {
            next_segment<S::kRows>(p, spans, seg);
            from = 0;
            to = static_cast<int>(min(static_cast<int64_t>(seg.keys.tiles), end - seg.start - kSwitch));
        }
    }
    // A warp's first partial comes back from global memory into its ring, so that the joins read shared memory only.
    if (s_has[2 * warp]) {
        static_assert(S::kPartial * 4 <= S::kStages * S::kStageBytes, "a partial in a warp's ring");
        const float4* const src = reinterpret_cast<const float4*>(scratch + (static_cast<int64_t>(blockIdx.x) * S::kWarps + warp) * S::kPartial);
        float4* const dst = reinterpret_cast<float4*>(smem + warp * S::kStages * S::kStageBytes);
#pragma unroll 8
        for (int i = lane; i < S::kPartial / 4; i += 32) dst[i] = src[i];
    }
    __syncthreads();

    // Join the partials of each segment that this CTA's warps share, in the order of the warps: into the
    // output, or into a partial of this CTA where the segment goes on in another.
    const auto slot = [&](int64_t cta, bool tail) { return slots + (2 * cta + (tail ? 1 : 0)) * S::kPartial; };
    const auto owned = [&](const Segment& s) {  // tiles before this CTA (1), after it (2)
        return (s.start + kSwitch < cta0 ? 1 : 0) | (s.start + kSwitch + s.keys.tiles > cta1 ? 2 : 0);
    };
    if (warp == 0) {  // the partials in order, and where each segment's begin: lane x looks at slot x
        const bool has = lane < 2 * S::kWarps && s_has[lane];
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, has), below = all & ((1u << lane) - 1u);
        const bool head = has && (below == 0 || s_seg[31 - __clz(below)].start != s_seg[lane].start);
        const uint32_t heads = __ballot_sync(0xFFFFFFFFu, head);
        if (has) s_list[__popc(below)] = lane;
        if (head) s_first[__popc(heads & ((1u << lane) - 1u))] = __popc(below);
        if (lane == 0) s_groups = __popc(heads), s_first[__popc(heads)] = __popc(all);
    }
    __syncthreads();
    const int groups = s_groups;
    constexpr int kQuads = D / 4, kItems = S::kRows * kQuads, kM = S::kRows * S::kPitch, kL = kM + S::kRows;
    const auto partial = [&](int i) {  // i-th of the list
        const int x = s_list[i];
        return (x & 1) ? reinterpret_cast<const float*>(smem + S::kRing) + (x >> 1) * S::kPartial
                       : reinterpret_cast<const float*>(smem + (x >> 1) * S::kStages * S::kStageBytes);
    };
    for (int item = tid; item < groups * kItems; item += S::kThreads) {
        const int gr = item / kItems, row = item % kItems / kQuads, d = 4 * (item % kQuads), first = s_first[gr];
        const Segment& s = s_seg[s_list[first]];
        if (s.row0 + row >= s.span.n * p.ratio) continue;
        const int over = owned(s);
        join_quad<T, D, G, NT, 6>(
            p, s, row, d, s_first[gr + 1] - first,
            [&](int i, float& m, float& l, float4& x) {
                const float* const q = partial(first + i);
                m = q[kM + row], l = q[kL + row], x = *reinterpret_cast<const float4*>(q + row * S::kPitch + d);
            },
            over ? slot(blockIdx.x, !(over & 1)) : nullptr);
    }
    // Segments that other CTAs share (the first and the last one of this CTA's): the last CTA to arrive joins their partials.
    const Segment* cross[2] = {nullptr, nullptr};
    if (groups > 0) {
        const Segment* const a = &s_seg[s_list[0]];
        const Segment* const b = &s_seg[s_list[s_first[groups - 1]]];
        const int oa = owned(*a), ob = owned(*b);
        if (oa & 1) cross[0] = a;
        if (ob == 2) cross[1] = b;
    }
    if (cross[0] == nullptr && cross[1] == nullptr) return;
    __syncthreads();
    if (tid < 2) {
        s_parts[tid] = 0;
        if ((tid ? cross[1] : cross[0]) != nullptr) {
            const auto cta_of = [&](int64_t unit) {
                // the CTA whose part holds a unit of a segment that CTAs share: its bounds are not moved within such a segment
                return unit < rest * (each + 1) ? quotient(unit, each + 1) : rest + quotient(unit - rest * (each + 1), each);
            };
            const Segment& s = tid ? *cross[1] : *cross[0];
            const int c0 = static_cast<int>(cta_of(s.start + kSwitch)), c1 = static_cast<int>(cta_of(s.start + kSwitch + s.keys.tiles - 1));
            __threadfence();
            if (atomicAdd(&arrived[c0], 1) == c1 - c0) s_parts[tid] = c1 - c0 + 1, s_cta[tid] = c0;
            __threadfence();
        }
    }
    __syncthreads();
    const int n0 = s_parts[0], n1 = s_parts[1];
    for (int item = n0 ? tid : tid + kItems; item < (n1 ? 2 * kItems : kItems); item += S::kThreads) {
        const int x = item / kItems, row = item % kItems / kQuads, d = 4 * (item % kQuads);
        const Segment& s = x ? *cross[1] : *cross[0];
        if (s.row0 + row >= s.span.n * p.ratio) continue;
        const int c0 = s_cta[x];
        join_quad<T, D, G, NT, 10>(
            p, s, row, d, x ? n1 : n0,
            [&](int i, float& m, float& l, float4& v) {
                const float* const q = slot(c0 + i, i == 0);
                m = __ldcg(q + kM + row), l = __ldcg(q + kL + row), v = __ldcg(reinterpret_cast<const float4*>(q + row * S::kPitch + d));
            },
            nullptr);
    }
    if (tid < 2 && s_parts[tid] > 0) arrived[s_cta[tid]] = 0;
}

}  // namespace sgemv
