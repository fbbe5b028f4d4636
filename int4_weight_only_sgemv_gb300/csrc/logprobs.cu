// Log-probabilities of rows of logits: lse = m + ln S, lp = (x - m) - ln S, entropy = ln S - E / S with
// S = sum e^(x-m), E = sum e^(x-m) (x-m), m the row's maximum, all in 32 bits; and the best `top` tokens of each row.
//
// The work is one read of the logits. A row is a CTA's, or a cluster's of up to 8 that share it where rows are few or long. A
// thread goes over its vectors of 16 bytes once, four loads under way, with sums about a reference of its own that follows the
// largest value only when that is more than kLag above (binary32 has room for far more), and keeps its maximum and where it
// is. At the end the sums are moved to the row's maximum. An element costs about 10 instructions, and what a warp does once a row
// about 500 (counted at two vocabularies), so CTAs are small where rows are many, and six of 256 threads share an SM (four: 106 us,
// five: 98, six: 94.5 for 4096 rows of 50001 bf16 logits, 64% of the measured HBM rate; the instructions bound it).
//
// The best tokens: each warp gives the ceil(top / warps)-th of its threads' maxima; the lowest of these is a bound that at least
// `top` elements reach. The vectors of the threads whose maximum reaches it, spread over all threads, are read again (from L2)
// for the elements that do, a little over `top`, which go into a list. An element's rank in the list is the number of larger
// ones; ties rank by the lower token, so keys are unique. If the list overflows (a row made so that a few threads hold
// most of the large values), its own `top`-th entry is a better bound and the search is run again. The CTAs of a cluster write
// their sums to each other, and their best to the first one, through distributed shared memory, before the one barrier that
// they share.
//
// x - m is formed before it is scaled to log2 (two packed operations for two elements, where one multiply-add by a rounded
// log2(e) m would do): a maximum's own weight is 1 exactly, so a row with all its weight on one token has lp 0 and entropy 0.
//
// Two passes over rows staged in shared memory by the copy engine, the next row's copies under way, were bound by two CTAs an
// SM (100 KB a row) waiting for each other: 145 us for 4096 rows of 50001 bf16 logits.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "kv_common.cuh"

namespace sgemv {

namespace {

namespace cg = cooperative_groups;

constexpr int kList = 1024;       // candidates
constexpr int kMaxTop = 64;
constexpr int kMaxCluster = 8;
constexpr float kLag = 8.0f;      // how far a thread's reference may be below its largest value
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

struct LogprobParams {
    const void* logits;
    int64_t stride;
    const int32_t* tokens;
    float* tok_logp;
    float* lse;
    float* entropy;
    int32_t* top_tok;
    float* top_logp;
    float* logp;
    int32_t* status;
    int rows, vocab, n_tok, top;
};

// What a CTA of a cluster tells the others: its maximum, the sums about it, and how many candidates it has.
struct Slice {
    float m, s, e;
    int n;
};

// Larger for a larger value, -0 as +0, NaN (as max_nan gives it) above +inf; never 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) == 0) u = 0;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t u) { return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u); }
// Larger for a larger logit; equal logits by the lower token. Never 0 for a real element.
__device__ __forceinline__ uint64_t key_of(float x, int tok) {
    return (static_cast<uint64_t>(order_of(x)) << 32) | static_cast<uint32_t>(~tok);
}
__device__ __forceinline__ float value_of(uint64_t key) { return of_order(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int token_of(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How many of the n keys are larger than k (key n is read too: 0).
__device__ __forceinline__ int count_larger(const uint64_t* keys, int n, uint64_t k) {
    int larger = 0;
#pragma unroll 8
    for (int j = 0; j < n; j += 2) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(keys + j);
        larger += (w.x > k) + (w.y > k);
    }
    return larger;
}
// The same for kMaxTop keys in descending order.
__device__ __forceinline__ int count_larger_sorted(const uint64_t* keys, uint64_t k) {
    int at = 0;
#pragma unroll
    for (int step = kMaxTop / 2; step > 0; step >>= 1)
        if (keys[at + step - 1] > k) at += step;
    return at + (keys[at] > k);
}

// 16 bytes of logits.
template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    uint4 w;
    __device__ __forceinline__ float at(int i) const { return to_f32(reinterpret_cast<const T*>(&w)[i]); }
    // Elements 2i and 2i + 1, what is below kLow (-inf among it) set to kLow: where the reference is far above, both have weight 0.
    static constexpr float kLow = std::is_same<T, __half>::value ? -65504.0f : -1e30f;
    __device__ __forceinline__ float2 two(int i) const {
        if constexpr (sizeof(T) == 2) {
            using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            const T low = from_f32<T>(kLow);
            const T2 h = __hmax2(reinterpret_cast<const T2*>(&w)[i], T2(low, low));
            return make_float2(to_f32(h.x), to_f32(h.y));
        } else {
            return make_float2(fmaxf(at(2 * i), kLow), fmaxf(at(2 * i + 1), kLow));
        }
    }
    __device__ __forceinline__ float max() const {  // NaN if one is
        if constexpr (sizeof(T) == 2) {
            using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            const T2* h = reinterpret_cast<const T2*>(&w);
            const T2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
            return max_nan(to_f32(m.x), to_f32(m.y));
        } else {
            return max_nan(max_nan(at(0), at(1)), max_nan(at(2), at(3)));
        }
    }
};

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 1536 / kThreads) logprobs_kernel(const LogprobParams p) {
    constexpr int kWarps = kThreads / 32, kN = Vec<T>::kN, kFlight = 4;
    __shared__ __align__(16) uint64_t s_list[kList + 2];
    __shared__ __align__(16) uint64_t s_best[kMaxCluster * kMaxTop];  // of each slice, highest first (in the first CTA)
    __shared__ Slice s_slice[kMaxCluster];
    __shared__ float s_f[2][kWarps];
    __shared__ uint32_t s_most[kWarps];
    __shared__ uint64_t s_key[kWarps];
    __shared__ uint16_t s_hot[kThreads];
    __shared__ int s_count, s_nhot;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / parts;
    if (tid == 0) s_count = s_nhot = 0;
    __syncwarp();
    if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // every CTA has started: see below
    pdl_launch_dependents();
    pdl_wait();

    // The row in vectors of 16 aligned bytes: vector v holds tokens kN v - head .. ; this CTA has [v0, v1), and [f0, f1) are whole.
    const T* const x = static_cast<const T*>(p.logits) + row * p.stride;
    const int head = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int nv = (head + p.vocab + kN - 1) / kN;
    const int v0 = parts == 1 ? 0 : static_cast<int>(static_cast<int64_t>(nv) * part / parts);
    const int v1 = parts == 1 ? nv : static_cast<int>(static_cast<int64_t>(nv) * (part + 1) / parts);
    const int f0 = max(v0, head > 0 ? 1 : 0), f1 = max(f0, min(v1, (head + p.vocab) / kN));
    const T* const xv = x - head;  // aligned: vector v is at xv + kN v
    const auto whole = [&](int v) {
        Vec<T> r;
        r.w = __ldg(reinterpret_cast<const uint4*>(xv + static_cast<int64_t>(v) * kN));
        return r;
    };
    const auto edge_of = [&](int v) {  // one that is not whole: -inf where there is no token
        Vec<T> r;
        T* h = reinterpret_cast<T*>(&r.w);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int tok = v * kN - head + i;
            h[i] = tok >= 0 && tok < p.vocab ? x[tok] : from_f32<T>(-INFINITY);
        }
        return r;
    };
    // a token asked for, a thread: its logit is needed at the end
    int given = -1;
    if (part == 0 && tid < p.n_tok) given = p.tokens[static_cast<int64_t>(row) * p.n_tok + tid];

    // this thread's maximum and the vector that has it; sums s of 2^a and e of 2^a a, a = (x - ref) log2(e), two of each
    float tm = -INFINITY, ref = 0.0f, lim = -INFINITY;
    int tv = -1;
    uint64_t s2 = 0, e2 = 0;
    const auto take = [&](const Vec<T>& y, int v) {
        const float vm = y.max();
        if (vm > tm || tv < 0) tv = v;
        tm = max_nan(tm, vm);
        if (vm > lim) {  // the first finite value, or one far above
            if (lim != -INFINITY) {
                const float d = (ref - vm) * kLog2e, f = exp2_approx(d);
                e2 = mul2(f == 0.0f ? 0 : fma2(s2, pair(d, d), e2), pair(f, f));
                s2 = mul2(s2, pair(f, f));
            }
            ref = vm, lim = vm + kLag;
        }
        if (vm == -INFINITY) return;
        if (ref > 0.5f * Vec<T>::kLow && ref < 1e30f) {  // kLow is far below, and kLow - ref finite
            const uint64_t scale = pair(kLog2e, kLog2e), minus = pair(-ref, -ref);
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) {
                const float2 f = y.two(i);
                const uint64_t a = mul2(add2(pair(f.x, f.y), minus), scale);
                const float2 af = parts_of(a);
                const uint64_t w = pair(exp2_approx(af.x), exp2_approx(af.y));
                s2 = add2(s2, w);
                e2 = fma2(w, a, e2);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const float a = fmaxf(y.at(i) - ref, -1e30f) * kLog2e, w = exp2_approx(a);
                s2 = add2(s2, pair(w, 0.0f));
                e2 = fma2(pair(w, 0.0f), pair(a, 0.0f), e2);
            }
        }
    };
    int v = f0 + tid;
    for (; v + (kFlight - 1) * kThreads < f1; v += kFlight * kThreads) {
        Vec<T> y[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) y[i] = whole(v + i * kThreads);
#pragma unroll
        for (int i = 0; i < kFlight; ++i) take(y[i], v + i * kThreads);
    }
    for (; v < f1; v += kThreads) take(whole(v), v);
    // the first and the last vector, where they are not whole
    const int edge = tid == 32 && v0 < f0 ? v0 : (tid == 33 && f1 < v1 ? v1 - 1 : -1);
    if (edge >= 0) take(edge_of(edge), edge);
    T given_x = from_f32<T>(0.0f);
    if (given >= 0 && given < p.vocab) given_x = x[given];
    // a thread's maximum is at least this key; 0 for a thread without a vector
    uint64_t key = tv >= 0 && tm == tm ? key_of(tm, tv * kN - head + kN - 1) : 0;
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, order_of(tm));
    if (lane == 0) s_most[warp] = most;
    if (p.top > 0) {
        // the warp's r-th largest: the largest is taken out r - 1 times
        uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key), h = 0, l = 0;
        for (int r = (p.top + kWarps - 1) / kWarps; r > 0; --r) {
            h = __reduce_max_sync(0xFFFFFFFFu, hi);
            l = __reduce_max_sync(0xFFFFFFFFu, hi == h ? lo : 0u);
            if (hi == h && lo == l) hi = lo = 0;
        }
        if (lane == 0) s_key[warp] = static_cast<uint64_t>(h) << 32 | l;
    }
    __syncthreads();
    // (a warp's lanes read all warps' and reduce them again)
    const float m = of_order(__reduce_max_sync(0xFFFFFFFFu, s_most[lane % kWarps]));
    uint64_t bound = ~0ull;
    if (p.top > 0) {
        const uint64_t k = s_key[lane % kWarps];
        const uint32_t hi = static_cast<uint32_t>(k >> 32), h = __reduce_min_sync(0xFFFFFFFFu, hi);
        const uint32_t l = __reduce_min_sync(0xFFFFFFFFu, hi == h ? static_cast<uint32_t>(k) : 0xFFFFFFFFu);
        bound = static_cast<uint64_t>(h) << 32 | l;
    }
    const bool usable = m < INFINITY;  // neither NaN nor +inf

    if (usable) {
        if (p.top > 0 && tv >= 0 && tm >= (bound == 0 ? -INFINITY : value_of(bound))) s_hot[atomicAdd(&s_nhot, 1)] = static_cast<uint16_t>(tid);
        // the sums about the slice's maximum, in natural units
        const float2 sf = parts_of(s2), ef = parts_of(e2);
        float s = sf.x + sf.y, e = ef.x + ef.y;
        const float d = lim == -INFINITY ? 0.0f : (ref - m) * kLog2e, f = exp2_approx(d);
        e = f == 0.0f ? 0.0f : kLn2 * fmaf(s, d, e) * f;
        s *= f;
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) {
            s += __shfl_xor_sync(0xFFFFFFFFu, s, j);
            e += __shfl_xor_sync(0xFFFFFFFFu, e, j);
        }
        if (lane == 0) s_f[0][warp] = s, s_f[1][warp] = e;
        __syncthreads();
        // candidates: vector i of hot thread j, and the edges
        const int hot = s_nhot, each = (f1 - f0 + kThreads - 1) / kThreads;  // vectors a thread has
        const int lg = 32 - __clz(max(each, 1) - 1);                         // and the next power of two
        while (p.top > 0) {
            const float bv = bound == 0 ? -INFINITY : value_of(bound);
            for (int i = tid; i < ((hot + 2) << lg); i += kThreads) {
                const int j0 = i >> lg, at = i & ((1 << lg) - 1);
                int v = -1;
                if (j0 < hot) {
                    v = f0 + s_hot[j0] + at * kThreads;
                    if (at >= each || v >= f1) v = -1;
                } else if (at == 0) {
                    v = j0 == hot ? (v0 < f0 ? v0 : -1) : (f1 < v1 ? v1 - 1 : -1);
                }
                if (v < 0) continue;
                const Vec<T> y = v >= f0 && v < f1 ? whole(v) : edge_of(v);
                uint32_t which = 0;
#pragma unroll
                for (int j = 0; j < kN; ++j) which |= y.at(j) >= bv ? 1u << j : 0u;
                for (; which != 0; which &= which - 1) {
                    const int j = __ffs(which) - 1, tok = v * kN - head + j;
                    if (tok < 0 || tok >= p.vocab) continue;
                    const uint64_t k = key_of(to_f32(x[tok]), tok);
                    if (k >= bound) {
                        const int at = atomicAdd(&s_count, 1);
                        if (at < kList) s_list[at] = k;
                    }
                }
            }
            __syncthreads();
            if (s_count <= kList) break;
            // too many: the list's own top-th key is a higher bound
            for (int i = tid; i < kList; i += kThreads) {
                const uint64_t k = s_list[i];
                if (count_larger(s_list, kList, k) == p.top - 1) s_key[0] = k;
            }
            __syncthreads();
            bound = s_key[0];
            if (tid == 0) s_count = 0;
            __syncthreads();
        }
    }
    if (tid == 0 && usable) s_list[s_count] = 0;
    __syncthreads();
    if (parts > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the others' shared memory may be written
    const int cand = usable ? s_count : 0;
    if (tid < parts) {
        Slice o = {m, 0.0f, 0.0f, min(cand, p.top)};
        if (usable) {
            for (int w = 0; w < kWarps; ++w) o.s += s_f[0][w], o.e += s_f[1][w];
        }
        *cluster.map_shared_rank(&s_slice[part], tid) = o;
    }
    uint64_t* const best = cluster.map_shared_rank(&s_best[part * kMaxTop], 0);
    for (int i = tid; i < cand; i += kThreads) {
        const uint64_t k = s_list[i];
        const int larger = count_larger(s_list, cand, k);
        if (larger < p.top) best[larger] = k;
    }
    if (tid >= min(cand, p.top) && tid < kMaxTop) best[tid] = 0;
    if (parts > 1) cluster.sync();
    else __syncthreads();

    // The whole row's, in every CTA of its cluster that writes something.
    const int writers = p.logp != nullptr ? kThreads : (part == 0 ? max(max(1, p.n_tok), parts * p.top) : 0);
    if ((tid & ~31) >= writers) return;
    float rm = s_slice[0].m, sum = 0.0f, ent = 0.0f;
    for (int i = 1; i < parts; ++i) rm = max_nan(rm, s_slice[i].m);
    const bool bad = !(rm < INFINITY), none = rm == -INFINITY;
    if (!bad && !none)
        for (int i = 0; i < parts; ++i) {
            const Slice o = s_slice[i];
            if (o.m == -INFINITY) continue;
            const float t = o.m - rm, f = exp2_approx(t * kLog2e), si = o.s * f;  // sums about o.m, moved to rm
            sum += si;
            ent += si == 0.0f ? 0.0f : fmaf(si, t, o.e * f);
        }
    const float kNan = __int_as_float(0x7FC00000), log_s = logf(sum);
    const auto lp = [&](float f) { return bad ? kNan : (none ? -INFINITY : (f - rm) - log_s); };
    if (part == 0) {
        if (tid == 0) {
            if (bad) report(p.status, SGEMV_ERR_NONFINITE);
            if (p.lse != nullptr) p.lse[row] = bad ? kNan : (none ? -INFINITY : rm + log_s);
            if (p.entropy != nullptr) p.entropy[row] = bad ? kNan : (none ? 0.0f : log_s - ent / sum);
        }
        if (tid < p.n_tok) {
            float v = 0.0f;
            if (given >= 0 && given < p.vocab) v = lp(to_f32(given_x));
            else if (given != -1) {
                v = kNan;
                report(p.status, SGEMV_ERR_ARG);
            }
            p.tok_logp[static_cast<int64_t>(row) * p.n_tok + tid] = v;
        }
        int found = 0;  // entries of all lists
        for (int i = 0; i < parts; ++i) found += s_slice[i].n;
        if (bad) found = 0;
        const int64_t o = static_cast<int64_t>(row) * p.top;
        for (int i = tid; i < parts * p.top && found > 0; i += kThreads) {
            int rank = i % p.top;
            const uint64_t k = s_best[i / p.top * kMaxTop + rank];
            if (k == 0) continue;
            if (parts > 1) {
                rank = 0;
#pragma unroll 4
                for (int j = 0; j < parts; ++j) rank += count_larger_sorted(s_best + j * kMaxTop, k);
            }
            if (rank < p.top) p.top_tok[o + rank] = token_of(k), p.top_logp[o + rank] = lp(value_of(k));
        }
        for (int j = found + tid; j < p.top; j += kThreads) p.top_tok[o + j] = -1, p.top_logp[o + j] = bad ? kNan : -INFINITY;
    }
    if (p.logp != nullptr) {
        float* const out = p.logp + static_cast<int64_t>(row) * p.vocab;
        const int t0 = max(0, v0 * kN - head), t1 = min(p.vocab, v1 * kN - head);
        int t = t0 + tid;
        for (; t + 7 * kThreads < t1; t += 8 * kThreads) {  // eight loads under way
            T y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[t + i * kThreads];
#pragma unroll
            for (int i = 0; i < 8; ++i) out[t + i * kThreads] = lp(to_f32(y[i]));
        }
        for (; t < t1; t += kThreads) out[t] = lp(to_f32(x[t]));
    }
}

template <typename T, int kThreads>
cudaError_t launch_rows(const LogprobParams& p, int parts, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * parts);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kThreads>, p);
}

template <typename T>
cudaError_t launch_logprobs(const LogprobParams& p, int sms, cudaStream_t s) {
    const int64_t nv = (static_cast<int64_t>(p.vocab) + 2 * Vec<T>::kN - 2) / Vec<T>::kN;  // with any alignment
    // One CTA a row; more where rows are too few to fill the GPU, in slices of 8 KB at least.
    int parts = 1;
    while (parts < kMaxCluster && static_cast<int64_t>(p.rows) * parts * 2 <= sms && nv > 512 * parts) parts *= 2;
    if (static_cast<int64_t>(p.rows) * parts > INT_MAX) return cudaErrorInvalidValue;
    const int64_t slice = (nv + parts - 1) / parts * 16;
    // As many threads as have a vector each (where some have none, every element is a candidate, and the list holds those of 128
    // vectors): 512 where rows are few, so that a row takes the least time, 256 where they fill the GPU.
    const bool few = static_cast<int64_t>(p.rows) * parts <= 2 * sms;
    if (slice >= 8 * 1024 && few) return launch_rows<T, 512>(p, parts, s);
    return slice >= 16 * 1024 ? launch_rows<T, 256>(p, parts, s) : launch_rows<T, 128>(p, parts, s);
}

}  // namespace

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_logprobs(const void* logits_dev, int dtype, int rows, int vocab, int64_t stride,
                              const int32_t* tokens_dev, int n_tok, int top, float* tok_logp_dev, float* lse_dev,
                              float* entropy_dev, int32_t* top_tok_dev, float* top_logp_dev, float* logp_dev,
                              int32_t* status_dev, void* stream) {
    if (dtype < SGEMV_F16 || dtype > SGEMV_F32 || rows < 0 || n_tok < 0 || n_tok > 64 || top < 0 || top > 64)
        return SGEMV_ERR_ARG;
    if (vocab < 1 || vocab > (1 << 24)) return SGEMV_ERR_SHAPE;
    if (stride < vocab) return SGEMV_ERR_ARG;
    if (rows == 0) return SGEMV_OK;
    if (logits_dev == nullptr || (n_tok > 0 && (tokens_dev == nullptr || tok_logp_dev == nullptr)) ||
        (top > 0 && (top_tok_dev == nullptr || top_logp_dev == nullptr)))
        return SGEMV_ERR_ARG;
    const void* words[] = {tokens_dev, tok_logp_dev, lse_dev, entropy_dev, top_tok_dev, top_logp_dev, logp_dev, status_dev};
    for (const void* q : words)
        if (!is_aligned(q, 4)) return SGEMV_ERR_ALIGN;
    if (!is_aligned(logits_dev, dtype == SGEMV_F32 ? 4 : 2)) return SGEMV_ERR_ALIGN;
    const uint64_t size = dtype == SGEMV_F32 ? 4 : 2, n = rows;
    const Bytes full(logp_dev, 4 * n * vocab), row(logits_dev, size * vocab);
    const Bytes written[] = {full, {tok_logp_dev, 4 * n * n_tok}, {lse_dev, 4 * n}, {entropy_dev, 4 * n}, {top_tok_dev, 4 * n * top},
                             {top_logp_dev, 4 * n * top}, {status_dev, 4}};
    const Bytes read[] = {{tokens_dev, 4 * n * n_tok}};
    if (!apart(written, read)) return SGEMV_ERR_ARG;
    for (int i = 0; i < 7; ++i)  // (a thread that writes a full row's element is the last to read it: logp may be logits)
        if (rows_meet(row, n, size * stride, written[i]) && (i > 0 || logp_dev != logits_dev || size != 4 || stride != vocab))
            return SGEMV_ERR_ARG;
    LogprobParams p = {};
    p.logits = logits_dev;
    p.stride = stride;
    p.tokens = tokens_dev;
    p.tok_logp = tok_logp_dev;
    p.lse = lse_dev;
    p.entropy = entropy_dev;
    p.top_tok = top_tok_dev;
    p.top_logp = top_logp_dev;
    p.logp = logp_dev;
    p.status = status_dev;
    p.rows = rows;
    p.vocab = vocab;
    p.n_tok = n_tok;
    p.top = top;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceInfo di;
    const int rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    const cudaError_t e = dtype == SGEMV_F16    ? launch_logprobs<__half>(p, di.sm_count, s)
                          : dtype == SGEMV_BF16 ? launch_logprobs<__nv_bfloat16>(p, di.sm_count, s)
                                                : launch_logprobs<float>(p, di.sm_count, s);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
