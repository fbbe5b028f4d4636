// Attention over the paged 4-bit KV cache: the kernel of prompt chunks (requests with many rows of queries).
//
// With many rows the products bound the work, not the cache's bytes: 4 D operations a (row, key) against D / 2 + 4 bytes a
// key. So they go to the 5th-generation tensor cores, S = x K^T with 128 x 64 x 16 and O += P V with 128 x D x 16 instructions, and
// one CTA holds two 128-row tiles of queries against each 64-key tile that it unpacks, which halves the unpacking a product
// needs. Roles, by warp:
//   0-3, 4-7  softmax of the first and of the second row tile: a thread a row, S from tensor memory, weights back to tensor
//             memory in fp16, over S
//   8-11      unpack K: raw subtiles -> the integers q - z [key][dim] in fp16, swizzled for the tensor cores, four buffers, and
//             the scales
//   12-15     unpack V [dim][key] likewise
//   16, 17    issue the products, a row tile each      18  issues the copies of raw subtiles (copy engine, 64 keys a stage)
// (with one warp a subtile for both K and V, unpacking was what a tile waited for: 2150 of 2850 cycles). Registers go from the
// other warps to the softmax's (setmaxnreg), whose rows' 64 scores stay in them.
// S has two buffers a row tile in tensor memory (2 x 2 x 64 columns beside 2 x D of O), so that the next tile's scores are there
// when a softmax is done with one: with 128-key tiles and one buffer each softmax waited 2100 of 6100 cycles a tile for its
// scores. (Where a key has two groups, each has sums of its own, and the two take the place of the two buffers.)
//
// Roundings: scores have none but the sums' in 32 bits: x is fp16, each row scaled by a power of two of its own
// (exact but for elements below 2^-29 of the row's largest), K's integers are exact, and the softmax multiplies a column by its
// scale. The weights are rounded to fp16, 11 bits, as in the decode kernel. V's values (q - z) s have up to 15 bits: they are formed
// as ((q - z) / 2) s, exact but for one rounding to 11 bits, in units of a power of two that follows from the segment's largest scale, so that no scale need be kept a column. The
// softmax's reference m moves only when a weight would pass 2^kLimit, so O is rarely rescaled.
//
// Bound by the softmax's chain and by shared memory: a 64-key tile takes 2450 cycles, of which the two row tiles' products need
// 1024 at the tensor cores' rate and 1500 as issued (64-column products read both operands from shared memory at more than
// its 128 bytes a cycle), and a softmax thread is busy for 1850. Two threads a row (16 softmax warps that agree on a reference
// tile by tile) took 3900 a tile: all roles contend for the same issue slots and shared memory. 3 requests of up to 2048 new tokens
// behind up to 8192 cached ones, 32 query heads, 8 KV heads of 128 (259 GFLOP): 337 us a call; 8 such requests:
// 624 us, 781 TFLOP/s (replayed from a graph over one set of inputs, the cache in L2: 331 and 620).
//
// Where there are fewer (row tile pair, head) segments than SMs, each is split over the keys; the softmax warps of the
// last CTA to arrive join.
#pragma once

#include "kv_decode.cuh"
#include "tcgen05.cuh"

namespace sgemv {

constexpr float kBig = 32768.0f; // 2^kLimit

template <int D, int G>
struct ChunkShape {
    static constexpr int kGroups = D / G;
    static constexpr int kSubBytes = 16 * D + 128 * kGroups;
    static constexpr int kRows = kChunkRows, kTile = 128;         // rows of a CTA and of a row tile
    static constexpr int kKeys = 64;                              // keys of a tile
    static constexpr int kSBufs = 2 / kGroups;                    // buffers of S
    static constexpr int kBufs = 4;                               // of K and V
    static constexpr int kRawSubs = 4, kRawStages = 3;            // subtiles of a raw stage
    static constexpr int kRawBytes = kRawSubs * kSubBytes;
    static constexpr int kAtoms = D / 64;                         // 128-byte columns of a row of x or K
    static constexpr int kQBytes = kTile * D * 2, kKBytes = kKeys * D * 2, kVBytes = D * kKeys * 2;
    static constexpr int kWarps = 20, kThreads = 32 * kWarps, kSoftmaxThreads = 256;
    // Registers a thread at launch, and after the split: 8 warps each, and 4. 8 kSoftmax + 8 kUnpack + 4 kOther = 20 kRegs. A warp
    // asks once: a second time is allowed only after its warpgroup has met, which the roles do not, so only softmax warps join.
    static constexpr int kRegs = 96, kRegsSoftmax = 128, kRegsUnpack = 80, kRegsOther = 64;
    static_assert(8 * kRegsSoftmax + 8 * kRegsUnpack + 4 * kRegsOther == kWarps * kRegs, "the split of the launch's registers");
    static constexpr int kSmem = 1024 + 2 * kQBytes + kBufs * (kKBytes + kVBytes) + kRawStages * kRawBytes;
    static constexpr int kPartial = kRows * (D + 2);              // floats of a partial: O, m, l
    static constexpr int kCols = 512;                             // tensor memory: S0, S1, O0, O1
};

// Segments (row tile pairs x heads) of a request that comes here.
template <int kRows>
__device__ __forceinline__ int64_t chunk_segments(const AttnParams& p, const Span& s) {
    const int rows = s.n * p.ratio;
    return rows > p.max_rows ? static_cast<int64_t>((rows + kRows - 1) / kRows) * p.heads : 0;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(ChunkShape<D, G>::kThreads, 1) chunk_kernel(const AttnParams p) {
    using S = ChunkShape<D, G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* const s_q = smem;
    uint8_t* const s_k = s_q + 2 * S::kQBytes;
    uint8_t* const s_v = s_k + S::kBufs * S::kKBytes;
    uint8_t* const s_raw = s_v + S::kBufs * S::kVBytes;
    __shared__ __align__(16) float s_scale[S::kBufs][S::kGroups][S::kKeys];  // of K's groups, times c
    __shared__ __align__(8) uint64_t raw_full[S::kRawStages], raw_free[S::kRawStages];
    __shared__ __align__(8) uint64_t k_full[S::kBufs], k_free[S::kBufs], v_full[S::kBufs], v_free[S::kBufs];
    __shared__ __align__(8) uint64_t q_full, s_full[2][2], p_full[2][2], o_full[2][2];
    __shared__ uint32_t s_tmem;
    __shared__ int64_t s_sum[S::kWarps];
    __shared__ int s_req, s_bad, s_last, s_vmax;
    __shared__ int64_t s_before;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S::kRawStages; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_free[i], 256);
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&k_full[i], 128), mbar_init(&k_free[i], 2);
            mbar_init(&v_full[i], 128), mbar_init(&v_free[i], 2);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(&s_full[i >> 1][i & 1], 1), mbar_init(&p_full[i >> 1][i & 1], 128), mbar_init(&o_full[i >> 1][i & 1], 1);
        mbar_init(&q_full, 256);
        mbar_fence_init();
        s_req = -1, s_bad = 0, s_vmax = 0;
    }
    pdl_launch_dependents();
    pdl_wait();

    // The request whose segment this CTA has. Thread x has requests [x * run, (x + 1) * run); where that is one each, they are taken
    // by descending length, so that the longest segments do not come last (3 requests of up to 2048 new tokens: 381 us in
    // index order, 335 so).
    const int run = (p.q.n_req + S::kThreads - 1) / S::kThreads;
    int64_t mine = 0;
    int* const s_len = reinterpret_cast<int*>(s_q);  // until the queries come
    int* const s_order = s_len + S::kThreads;
    int* const s_count = s_order + S::kThreads;
    if (run == 1) {
        int count = 0;
        if (tid < p.q.n_req) {
            const Span s = span_of(p, tid);
            count = static_cast<int>(chunk_segments<S::kRows>(p, s));
            s_len[tid] = count > 0 ? s.len : -1;
        }
        __syncthreads();
        if (tid < p.q.n_req) {
            const int len = s_len[tid];
            int rank = 0;
            for (int r = 0; r < p.q.n_req; ++r) rank += s_len[r] > len || (s_len[r] == len && r < tid);
            s_order[rank] = tid;
            s_count[rank] = count;
        }
        __syncthreads();
        if (tid < p.q.n_req) mine = s_count[tid];
    } else {
        for (int r = tid * run; r < min((tid + 1) * run, p.q.n_req); ++r) mine += chunk_segments<S::kRows>(p, span_of(p, r));
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
    // fewer segments than SMs are split over the keys (the workspace has a partial for each of kMaxCtas CTAs)
    const int splits = total == 0 || total * 2 > kMaxCtas ? 1 : static_cast<int>(kMaxCtas / total);
    if (blockIdx.x >= total * splits) return;
    const int64_t want = blockIdx.x / splits;
    const int part = blockIdx.x % splits;
    if (want >= before && want < before + mine) {
        int r = run == 1 ? s_order[tid] : tid * run;
        for (; run > 1; ++r) {
            const int64_t n = chunk_segments<S::kRows>(p, span_of(p, r));
            if (want < before + n) break;
            before += n;
        }
        s_req = r, s_before = before;
    }
    __syncthreads();
    const int req = s_req;
    const Span sp = span_of(p, req);
    const int in_req = static_cast<int>(want - s_before);
    // within a request the last rows, which see the most keys, come first
    const int rows = sp.n * p.ratio, old = sp.len - sp.n;
    const int head = in_req % p.heads, row0 = ((rows + S::kRows - 1) / S::kRows - 1 - in_req / p.heads) * S::kRows;
    const Keys keys = keys_of<S::kKeys>(p, sp, row0, S::kRows);
    const int all_tiles = keys.tiles;
    const int parts = min(splits, max(1, all_tiles / 4));  // a few tiles a split at least
    if (part >= parts) return;
    const int tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * part / parts);
    const int tiles = static_cast<int>(static_cast<int64_t>(all_tiles) * (part + 1) / parts) - tile0;
    const int key0 = keys.lo + tile0 * S::kKeys;
    const int32_t* const table = p.q.table_dev + req * p.q.table_stride;
    // Beforehand: page ids outside the cache, and the largest of V's scales (1% of the time of a long segment).
    {
        int big = 0;
        const int end = min(keys.hi, key0 + tiles * S::kKeys);
#pragma unroll 4
        for (int pos = key0 + tid; pos < end; pos += S::kThreads) {
            const int id = table[pos >> p.log2_page];
            if (id < 0 || id >= p.n_pages) {
                report(p.status, SGEMV_ERR_ARG);
                s_bad = 1;
                continue;
            }
            const uint8_t* const at = p.cache + id * p.page_bytes + head * p.head_bytes + ((pos & (p.page - 1)) / kSub) * S::kSubBytes +
                                      16 * D + 64 * S::kGroups + 4 * (pos % kSub);
#pragma unroll
            for (int gr = 0; gr < S::kGroups; ++gr) {
                const int bits = *reinterpret_cast<const unsigned short*>(at + 64 * gr);
                if (bits < 0x7C00) big = max(big, bits);  // (what a masked position holds need not be a number)
            }
        }
        big = __reduce_max_sync(0xFFFFFFFFu, big);
        if (lane == 0 && big != 0) atomicMax(&s_vmax, big);
    }
    if (warp == 16) tc_alloc(&s_tmem, S::kCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = s_tmem;
    const bool any_bad = s_bad != 0;
    // V's values are held in units of 2^vexp, which brings the largest scale to 2^11 .. 2^12: 15 s / 2 stays below fp16's end
    // whatever the scale, and small ones are not lost to subnormals.
    const int vexp = max(-14, min(4, (s_vmax >> 10) - 15 - 11));
    const auto lost = [&](int pos) {  // the page of a position is outside the cache
        const int id = table[pos >> p.log2_page];
        return id < 0 || id >= p.n_pages;
    };
    bool dead = false;  // a wait gave up: nothing is waited for any more, and what comes out is reported as invalid
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (dead || mbar_wait(bar, parity)) return;
        dead = true;
        report(p.status, SGEMV_ERR_TIMEOUT);
    };

    if (warp < 8) {
        regs_inc<S::kRegsSoftmax>();
        // ---------------------------------------------------------------------------------------- softmax
        const int x = warp >> 2, r = tid & 127, row = row0 + 128 * x + r;
        const bool live = row < rows;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + 256 + 128 * x;
        const int i = min(row, rows - 1) / p.ratio;
        // x: this thread's row, to shared memory, times a power of two of its own (with the sign of the scale) that brings its largest
        // element into [2^15, 2^16); what that leaves to the row's scores is `down`. Dims in the order 0 4 1 5 2 6 3 7 of each 8, as
        // K's nibbles come out.
        float down;
        {
            const T* src = static_cast<const T*>(p.q.q_dev) + (sp.first + i) * p.q.q_token_stride +
                           (head * p.ratio + min(row, rows - 1) % p.ratio) * p.q.q_head_stride;
            float big = 0.0f;
#pragma unroll 4
            for (int d = 0; d < D; d += 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(src + d);
                const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
                for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(to_f32(h[j])));
            }
            const int sh = query_shift(big);
            down = pow2(-sh);
            // (a row with an infinite element has no number for a score)
            const float up = big < INFINITY ? copysignf(pow2(sh), p.scale_log2) : __int_as_float(0x7FC00000);
            uint8_t* const dst = s_q + x * S::kQBytes + r * 128;
#pragma unroll 4
            for (int d = 0; d < D; d += 8) {
                uint4 w = live ? *reinterpret_cast<const uint4*>(src + d) : make_uint4(0, 0, 0, 0);
                const T* h = reinterpret_cast<const T*>(&w);
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = to_f32(h[j]) * up;
                const uint4 o = make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]), pack_half2(f[2], f[6]), pack_half2(f[3], f[7]));
                *reinterpret_cast<uint4*>(dst + d / 64 * (128 * 128) + (((d / 8) & 7) ^ (r & 7)) * 16) = o;
            }
            fence_async();
            mbar_arrive(&q_full);
        }
        const int last = old + i, first = p.q.window > 0 ? last - p.q.window + 1 : 0;
        const uint64_t tree = p.q.tree_dev != nullptr ? p.q.tree_dev[sp.first + i] : 0;
        // positions [clear0, clear1) are seen by every row of this row tile
        const int ia = min(row0 + 128 * x, rows - 1) / p.ratio, ib = min(row0 + 128 * x + 127, rows - 1) / p.ratio;
        const int clear1 = any_bad ? 0 : (p.q.tree_dev != nullptr ? old : old + ia + 1);
        const int clear0 = p.q.window > 0 ? old + ib - p.q.window + 1 : 0;
        float ref = 0.0f;   // the reference
        bool seen = false;  // whether it was set
        uint64_t l2 = 0;    // two sums
        for (int j = 0; j < tiles; ++j) {
            const int pos0 = key0 + j * S::kKeys, b = j % S::kSBufs;
            const uint32_t ts = tmem + lanes + 128 * x + 64 * b;
            wait(&s_full[x][b], (j / S::kSBufs) & 1);  // (the products waited for K, its scales with it)
            __syncwarp();
            tc_after_sync();
            const bool plain = pos0 >= clear0 && pos0 + S::kKeys <= clear1;
            // this row's scores but for `down`: sums times scales, -inf where masked
            float s[64];
            {
                const float* const scale = &s_scale[j % S::kBufs][0][0];
                if constexpr (S::kGroups == 1) {
                    uint32_t raw[2][32];
                    tc_ld32(raw[0], ts);
                    tc_ld32(raw[1], ts + 32);
                    tc_wait_ld();
#pragma unroll
                    for (int n = 0; n < 64; n += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(scale + n);
                        const uint32_t* const r4 = &raw[n / 32][n % 32];
                        const float2 t0 = parts_of(mul2(pair(__uint_as_float(r4[0]), __uint_as_float(r4[1])), pair(f.x, f.y)));
                        const float2 t1 = parts_of(mul2(pair(__uint_as_float(r4[2]), __uint_as_float(r4[3])), pair(f.z, f.w)));
                        s[n] = t0.x, s[n + 1] = t0.y, s[n + 2] = t1.x, s[n + 3] = t1.y;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t raw[2][32];
                        tc_ld32(raw[0], ts + 32 * q);
                        tc_ld32(raw[1], ts + 64 + 32 * q);
                        tc_wait_ld();
#pragma unroll
                        for (int n = 0; n < 32; n += 2) {
                            const float2 f = *reinterpret_cast<const float2*>(scale + 32 * q + n);
                            const float2 g = *reinterpret_cast<const float2*>(scale + S::kKeys + 32 * q + n);
                            const uint64_t a = mul2(pair(__uint_as_float(raw[0][n]), __uint_as_float(raw[0][n + 1])), pair(f.x, f.y));
                            const float2 t = parts_of(fma2(pair(__uint_as_float(raw[1][n]), __uint_as_float(raw[1][n + 1])), pair(g.x, g.y), a));
                            s[32 * q + n] = t.x, s[32 * q + n + 1] = t.y;
                        }
                    }
                }
            }
            if (!plain) {
                uint64_t see = 0;
#pragma unroll 1
                for (int n = 0; n < 64; ++n) {
                    const int pos = pos0 + n;
                    bool ok = pos < keys.hi;
                    if (p.q.tree_dev != nullptr) ok = ok && (pos < old || ((tree >> (pos - old)) & 1));
                    else ok = ok && pos >= first && pos <= last;
                    if (any_bad) ok = ok && !lost(pos);
                    see |= ok ? 1ull << n : 0ull;
                }
#pragma unroll
                for (int n = 0; n < 64; ++n)
                    if (!((see >> n) & 1u)) s[n] = -INFINITY;
            }
            // The weights. Whether a row's reference has to move shows in their sum, so that the largest score is looked for only in
            // the rare tile that moves one (and until a row has one). What a row does depends on nothing in other rows.
            uint32_t w[32];
            uint64_t sum;
            bool need = !seen;
            for (int pass = 0;; ++pass) {
                if (__any_sync(0xFFFFFFFFu, need)) {
                    float top = fmaxf(s[0], s[63]), top1 = s[1];
#pragma unroll
                    for (int n = 2; n < 62; n += 4) top = fmaxf(fmaxf(top, s[n]), s[n + 1]), top1 = fmaxf(fmaxf(top1, s[n + 2]), s[n + 3]);
                    top = fmaxf(fmaxf(top, top1), s[62]);
                    float f = 1.0f;
                    if (need && top > -INFINITY) {
                        const float at = fmaf(top, down, -kTop);
                        if (seen) f = exp2_approx(ref - at);
                        ref = at;
                        seen = true;
                    }
                    l2 = mul2(l2, pair(f, f));
                    if (j > 0 && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
                        // O holds every tile before this one. (The tile before that is known to be in: this one's scores came after it.)
                        wait(&o_full[x][(j - 1) % S::kSBufs], ((j - 1) / S::kSBufs) & 1);
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
                // (`down` is a power of two, so this is the difference of two rounded numbers: a score far past 2^24 still has a weight of
                // about 1 where it is the largest)
                sum = 0;
                const uint64_t rr = pair(-ref, -ref), dd = pair(down, down);
#pragma unroll
                for (int n = 0; n < 32; ++n) {
                    const float2 t = parts_of(fma2(pair(s[2 * n], s[2 * n + 1]), dd, rr));
                    const float a = exp2_approx(t.x), e = exp2_approx(t.y);
                    sum = add2(sum, pair(a, e));
                    w[n] = pack_half2(a, e);
                }
                const float2 both = parts_of(sum);
                need = both.x + both.y > kBig;  // (not after the reference has moved)
                if (pass == 2 || !__any_sync(0xFFFFFFFFu, need)) break;
            }
            l2 = add2(l2, sum);
            tc_st32(ts, w);
            tc_wait_st();
            tc_before_sync();
            mbar_arrive(&p_full[x][b]);
        }
        wait(&o_full[x][(tiles - 1) % S::kSBufs], ((tiles - 1) / S::kSBufs) & 1);
        __syncwarp();
        tc_after_sync();
        const float2 lf = parts_of(l2);
        const float m = seen ? ref : -INFINITY, l = lf.x + lf.y;
        float* const slot = parts > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(p.q.workspace_dev) + 4096) +
                                             static_cast<int64_t>(blockIdx.x) * S::kPartial : nullptr;
        int tok = 0, a = 0;
        T* out = nullptr;
        if (live) {
            tok = sp.first + row / p.ratio, a = head * p.ratio + row % p.ratio;
            out = static_cast<T*>(p.q.out_dev) + tok * p.q.out_token_stride + a * p.q.out_head_stride;
        }
        const float unit = __uint_as_float(static_cast<uint32_t>(127 + vexp + 1) << 23);  // and halved
        const float inv = l == 0.0f ? 0.0f : unit / l;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tc_ld32(o, to + 32 * q);
            tc_wait_ld();
            if (!live) continue;
#pragma unroll
            for (int n = 0; n < 32; n += 8) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[n + e]);
                if (slot != nullptr) {
                    float* const d = slot + (128 * x + r) * D + 32 * q + n;
                    *reinterpret_cast<float4*>(d) = make_float4(unit * f[0], unit * f[1], unit * f[2], unit * f[3]);
                    *reinterpret_cast<float4*>(d + 4) = make_float4(unit * f[4], unit * f[5], unit * f[6], unit * f[7]);
                } else {
                    T h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = from_f32<T>(f[e] * inv);
                    *reinterpret_cast<uint4*>(out + 32 * q + n) = *reinterpret_cast<const uint4*>(h);
                }
            }
        }
        if (slot != nullptr) {
            slot[S::kRows * D + 128 * x + r] = m;
            slot[S::kRows * (D + 1) + 128 * x + r] = l;
        } else if (live) {
            write_lse(p, tok, a, m, l);
        }
        __syncwarp();
        tc_before_sync();
        __syncthreads();  // (the other roles' at their ends)
        if (parts == 1) return;

        // Join the splits of the segment: the last CTA to arrive, 4 dims of a row a thread, in the order of the keys.
        int* const arrived = static_cast<int*>(p.q.workspace_dev);
        const int64_t seg = blockIdx.x / splits;
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(&arrived[seg], 1) == parts - 1;
            __threadfence();
        }
        named_bar_sync(1, S::kSoftmaxThreads);
        if (!s_last) return;
        const float* const slots = reinterpret_cast<const float*>(static_cast<uint8_t*>(p.q.workspace_dev) + 4096) + seg * splits * S::kPartial;
        constexpr int kQuads = D / 4;
        for (int item = tid; item < min(S::kRows, rows - row0) * kQuads; item += S::kSoftmaxThreads) {
            const int rr = item / kQuads, d = 4 * (item % kQuads), at = row0 + rr, t = sp.first + at / p.ratio, ah = head * p.ratio + at % p.ratio;
            float mj, lj;
            const float4 o = join<8>(parts, [&](int n, float& mi, float& li, float4& v) {
                const float* const q = slots + n * S::kPartial;
                mi = __ldcg(q + S::kRows * D + rr), li = __ldcg(q + S::kRows * (D + 1) + rr), v = __ldcg(reinterpret_cast<const float4*>(q + rr * D + d));
            }, mj, lj);
            write_quad(p, static_cast<T*>(p.q.out_dev) + t * p.q.out_token_stride + ah * p.q.out_head_stride, d, o, mj, lj, t, ah);
        }
        if (tid == 0) arrived[seg] = 0;
        return;
    }
    if (warp < 16) {
        regs_dec<S::kRegsUnpack>();
        // ---------------------------------------------------------------------------------------- unpack
        const bool keys_not_values = warp < 12;
        const int w = warp & 3, g = lane >> 2, t = lane & 3;
        const __half2 half2_half = __floats2half2_rn(0.5f, 0.5f), half2_32nd = __floats2half2_rn(0.03125f, 0.03125f);
        const __half2 up = __float2half2_rn(__uint_as_float(static_cast<uint32_t>(127 - vexp) << 23));
        const __half2 half2_16th = __floats2half2_rn(0.0625f, 0.0625f);
        // (nibble - zero) / 2 of bits 0 (hi false) or 4 of each half of a word, exactly; then times s, for V the scale
        const auto value = [&](uint32_t a, bool hi, __half2 zero, __half2 s) {
            const uint32_t m = hi ? 0x00F000F0u : 0x000F000Fu;
            const uint32_t b = (a & m) | 0x64006400u;  // 1024 + q, or 1024 + 16 q
            const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&b), hi ? half2_32nd : half2_half, zero);
            const __half2 f = __hmul2(v, s);
            return *reinterpret_cast<const uint32_t*>(&f);
        };
        // nibble - zero of the same bits, exactly
        const auto whole = [&](uint32_t a, bool hi, __half2 zero) {
            const uint32_t b = (a & (hi ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
            const __half2 n = *reinterpret_cast<const __half2*>(&b);
            const __half2 f = hi ? __hfma2(n, half2_16th, zero) : __hadd2(n, zero);
            return *reinterpret_cast<const uint32_t*>(&f);
        };
        const float c = fabsf(p.scale_log2);
        for (int j = 0; j < tiles; ++j) {
            const int stage = j % S::kRawStages, buf = j % S::kBufs;
            const int pos = key0 + S::kKeys * j + 16 * w;  // this warp's subtile
            wait(&raw_full[stage], (j / S::kRawStages) & 1);
            if (j >= S::kBufs) {  // after the tile that had the buffers; for K's scales, after its softmax too
                if (keys_not_values) wait(&k_free[buf], (j / S::kBufs - 1) & 1);
                wait(&v_free[buf], (j / S::kBufs - 1) & 1);
            }
            __syncwarp();
            const uint8_t* const sub = s_raw + stage * S::kRawBytes + w * S::kSubBytes;
            const bool odd = pos + kSub > keys.hi || any_bad;
            const auto scales = [&](const uint8_t* at, int token) {  // a token that there is not: 0
                uint32_t sz = *reinterpret_cast<const uint32_t*>(at + 4 * token);
                if (odd && (pos + token >= keys.hi || (any_bad && lost(pos + token)))) sz = 0;
                return sz;
            };
            const int col = 16 * w;  // key of the tile
            // K: 8 lanes a token and atom, each a word of 8 dims
            if (keys_not_values) {
                uint8_t* const dst = s_k + buf * S::kKBytes;
#pragma unroll
                for (int n = 0; n < 4 * S::kAtoms; ++n) {
                    const int token = 4 * (n % 4) + (lane >> 3), atom = n / 4, wd = lane & 7;
                    const int d = 64 * atom + 8 * wd;
                    constexpr int P = D < 128 ? D : 128;
                    const uint32_t a = *reinterpret_cast<const uint32_t*>(sub + d / P * 8 * P + token * (P / 2) + d % P / 2);
                    const uint32_t sz = scales(sub + 16 * D + 64 * (64 * atom / G), token);
                    const __half2 z = __half2half2(__ushort_as_half(static_cast<unsigned short>(sz >> 16)));
                    const __half2 z0 = __hsub2(__floats2half2_rn(-1024.0f, -1024.0f), z), z1 = __hsub2(__floats2half2_rn(-64.0f, -64.0f), z);
                    const uint4 o = make_uint4(whole(a, false, z0), whole(a, true, z1), whole(a >> 8, false, z0), whole(a >> 8, true, z1));
                    const int row = col + token;
                    *reinterpret_cast<uint4*>(dst + atom * (S::kKeys * 128) + row * 128 + ((wd ^ (row & 7)) * 16)) = o;
                    if (wd == 0 && 64 * atom % G == 0)
                        s_scale[buf][64 * atom / G][row] = __half2float(__ushort_as_half(static_cast<unsigned short>(sz & 0xFFFFu))) * c;
                }
                fence_async();
                mbar_arrive(&k_full[buf]);
            }
            // V: lane (g, t) has tokens 4t .. 4t + 3 of dims g + 8n + 32i
            if (!keys_not_values) {
                uint8_t* const dst = s_v + buf * S::kVBytes;
                uint32_t vq[D / 16];
#pragma unroll
                for (int r = 0; r < D / 64; ++r)
                    *reinterpret_cast<uint4*>(vq + 4 * r) = *reinterpret_cast<const uint4*>(sub + 8 * D + 512 * r + 16 * lane);
#pragma unroll
                for (int gr = 0; gr < S::kGroups; ++gr) {
                    __half2 s[2], z0[2], z1[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t a = scales(sub + 16 * D + 64 * (S::kGroups + gr), 4 * t + 2 * e);
                        const uint32_t b = scales(sub + 16 * D + 64 * (S::kGroups + gr), 4 * t + 2 * e + 1);
                        const uint32_t sw = __byte_perm(a, b, 0x5410), zw = __byte_perm(a, b, 0x7632);
                        s[e] = __hmul2(*reinterpret_cast<const __half2*>(&sw), up);
                        const __half2 z = *reinterpret_cast<const __half2*>(&zw);
                        z0[e] = __hfma2(z, __floats2half2_rn(-0.5f, -0.5f), __floats2half2_rn(-512.0f, -512.0f));
                        z1[e] = __hfma2(z, __floats2half2_rn(-0.5f, -0.5f), __floats2half2_rn(-32.0f, -32.0f));
                    }
#pragma unroll
                    for (int ii = 0; ii < G / 32; ++ii) {
                        const int i = gr * (G / 32) + ii;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const uint32_t a = n < 2 ? vq[i] : vq[i] >> 8, b = n < 2 ? vq[D / 32 + i] : vq[D / 32 + i] >> 8;
                            const uint2 o = make_uint2(value(a, n & 1, (n & 1) ? z1[0] : z0[0], s[0]), value(b, n & 1, (n & 1) ? z1[1] : z0[1], s[1]));
                            const int d = 32 * i + 8 * n + g, k = col + 4 * t;  // row and key
                            *reinterpret_cast<uint2*>(dst + k / 64 * (D * 128) + d * 128 + ((((k % 64) / 8) ^ (d & 7)) * 16) + (k % 8) * 2) = o;
                        }
                    }
                }
                fence_async();
                mbar_arrive(&v_full[buf]);
            }
            mbar_arrive(&raw_free[stage]);
        }
    } else {
        regs_dec<S::kRegsOther>();
        if (warp < 18) {
        // ---------------------------------------------------------------------------------------- products
        // A warp a row tile. The whole warp goes through the loop, with values that the compiler can see are the same in its lanes
        // (they end up in uniform registers, which the instruction reads); one lane issues. Issued from a branch of one lane, with
        // descriptors formed anew, an instruction took 115 cycles to issue, more than it takes to run; with one warp for both row
        // tiles, 80.
        const int x = __shfl_sync(0xFFFFFFFFu, warp - 16, 0);
        const int n_tiles = __shfl_sync(0xFFFFFFFFu, tiles, 0);
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0) + 128 * x;
        const uint64_t q_desc = tc_desc(smem_addr(s_q) + x * S::kQBytes), k_desc = tc_desc(smem_addr(s_k)), v_desc = tc_desc(smem_addr(s_v));
        const auto hold = [&](uint64_t* bar, uint32_t parity) {
            wait(bar, parity);
            dead = __any_sync(0xFFFFFFFFu, dead);
            tc_after_sync();
        };
        const auto scores = [&](int j) {  // of tile j, once its K is there
            const int buf = j % S::kBufs, b = j % S::kSBufs;
            if (elect_one()) {
                const uint64_t kd = k_desc + buf * (S::kKBytes >> 4);
                const uint32_t to = tm + 64 * b;
                if (!dead) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma_ss(to + 64 * (kk / (G / 16)), q_desc + ((kk / 4 * (128 * 128) + kk % 4 * 32) >> 4),
                                  kd + ((kk / 4 * (S::kKeys * 128) + kk % 4 * 32) >> 4), tc_idesc(S::kKeys), kk % (G / 16) > 0);
                }
                tc_commit(&s_full[x][b]);
                tc_commit(&k_free[buf]);
            }
            __syncwarp();
        };
        hold(&q_full, 0);
        for (int j = 0; j < min(S::kSBufs, n_tiles); ++j) {
            hold(&k_full[j], 0);
            scores(j);
        }
        for (int j = 0; j < n_tiles; ++j) {
            const int buf = j % S::kBufs, b = j % S::kSBufs, next = j + S::kSBufs;
            hold(&v_full[buf], (j / S::kBufs) & 1);
            if (next < n_tiles) hold(&k_full[next % S::kBufs], (next / S::kBufs) & 1);
            hold(&p_full[x][b], (j / S::kSBufs) & 1);
            if (elect_one()) {
                const uint64_t vd = v_desc + buf * (S::kVBytes >> 4);
                const uint32_t to = tm + 256, from = tm + 64 * b;
                if (!dead) {
                    tc_mma_ts(to, from, vd, tc_idesc(D), j > 0);
#pragma unroll
                    for (int kk = 1; kk < S::kKeys / 16; ++kk) tc_mma_ts(to, from + 8 * kk, vd + (kk * 32 >> 4), tc_idesc(D), true);
                }
                tc_commit(&o_full[x][b]);
                tc_commit(&v_free[buf]);
            }
            __syncwarp();
            if (next < n_tiles) scores(next);  // over the weights just used: the products run in the order of their issue
        }
        // The last products arrive at barriers that nobody else waits for: none may be under way when the CTA leaves and its tensor
        // memory goes, whether or not another role gave up.
        for (int j = max(0, n_tiles - S::kBufs); j < n_tiles; ++j) {
            mbar_wait(&k_free[j % S::kBufs], (j / S::kBufs) & 1);
            mbar_wait(&v_free[j % S::kBufs], (j / S::kBufs) & 1);
        }
        } else if (warp == 18) {
        // ---------------------------------------------------------------------------------------- copies
        const int per = min(p.page, 64);  // keys of a copy
        const uint8_t* const base = p.cache + head * p.head_bytes;
        int j = 0;
        for (; j < tiles; ++j) {
            const int stage = j % S::kRawStages;
            if (j >= S::kRawStages) wait(&raw_free[stage], (j / S::kRawStages - 1) & 1);
            const int pos = key0 + S::kKeys * j + lane * per;  // of this lane's copy
            uint32_t bytes = 0;
            const uint8_t* src = nullptr;
            if (lane * per < 64 && pos < keys.hi) {
                const int id = table[pos >> p.log2_page];
                if (id >= 0 && id < p.n_pages) {
                    bytes = ((min(keys.hi, pos + per) - pos + kSub - 1) / kSub) * S::kSubBytes;
                    src = base + id * p.page_bytes + ((pos & (p.page - 1)) / kSub) * S::kSubBytes;
                }
            }
            uint32_t sum = bytes;
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            dead = __any_sync(0xFFFFFFFFu, dead);
            if (dead) break;
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[stage], sum);
            __syncwarp();
            if (bytes) bulk_g2s(s_raw + stage * S::kRawBytes + lane * (per / kSub) * S::kSubBytes, src, bytes, &raw_full[stage]);
        }
        // (all have landed when the unpack warps are done, unless one of them gave up)
        for (int i = max(0, j - S::kRawStages); i < j; ++i) mbar_wait(&raw_full[i % S::kRawStages], (i / S::kRawStages) & 1);
        }
    }
    __syncwarp();
    __syncthreads();
    tc_after_sync();
    if (warp == 16) tc_dealloc(tmem, S::kCols);
}

}  // namespace sgemv
