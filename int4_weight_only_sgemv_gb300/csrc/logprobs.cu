// Log-probabilities of rows of logits: lse = m + ln S, lp = (x - m) - ln S, entropy = ln S - E / S with
// S = sum e^(x-m), E = sum e^(x-m) (x-m), m the row's maximum, all in 32 bits; and the best `top` tokens of each row.
//
// The work is one read of the logits, so a row is read from global memory once: by one CTA, or by a cluster of up to 8 that
// share it where rows are few or long, into shared memory (copy engine, several chunks in flight). Two passes over
// shared memory follow:
//  A  each thread's maximum and where it is, as the chunks arrive; from these the row's (or slice's) maximum, and a bound that
//     at least `top` elements reach: each warp sorts its 32 maxima and gives its ceil(top / warps)-th; the bound is the lowest.
//  B  the sums, and the elements that reach the bound (a little over `top` of them) into a list.
// An element's rank in the list is the number of larger ones; ties rank by the lower token, so keys are unique. If the list
// overflows (a row made so that a few threads hold most of the large values), its own `top`-th entry is a better bound and
// the pass is run again. Clusters hand their lists and sums to the first CTA through distributed shared memory.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "kv_common.cuh"

namespace sgemv {

namespace {

namespace cg = cooperative_groups;

constexpr int kList = 2048;       // candidates
constexpr int kMaxTop = 64;
constexpr int kMaxCluster = 8;
constexpr int kChunks = 8;        // copies a slice is fetched with
constexpr float kLog2e = 1.44269504088896340736f;

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
    int staged;   // the slices fit in shared memory
};

// What a CTA of a cluster tells the first one.
struct Slice {
    float m, s, e;
    int n;                   // entries of best
    uint64_t best[kMaxTop];  // keys, highest first
};

// Larger for a larger logit; equal logits by the lower token. -0 counts as +0. Never 0 for a real element.
__device__ __forceinline__ uint64_t key_of(float x, int tok) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) == 0) u = 0;
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<uint64_t>(u) << 32) | static_cast<uint32_t>(~tok);
}
__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
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

// 16 bytes of logits.
template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    uint4 w;
    __device__ __forceinline__ float at(int i) const { return to_f32(reinterpret_cast<const T*>(&w)[i]); }
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
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobParams p) {
    constexpr int kWarps = kThreads / 32, kN = Vec<T>::kN;
    extern __shared__ __align__(16) uint8_t s_data[];  // the slice
    __shared__ uint64_t s_list[kList];
    __shared__ Slice s_slice;
    __shared__ float s_f[3][kWarps];
    __shared__ uint64_t s_key[kWarps];
    __shared__ int s_count;
    __shared__ __align__(8) uint64_t s_bar[kChunks];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / parts;
    if (tid < kChunks) mbar_init(&s_bar[tid], 1);
    if (tid == 0) mbar_fence_init();
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // The row in vectors of 16 aligned bytes: vector v holds tokens kN v - head .. ; this CTA has [v0, v1).
    const T* const x = static_cast<const T*>(p.logits) + row * p.stride;
    const int head = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    const int nv = (head + p.vocab + kN - 1) / kN;
    const int v0 = static_cast<int>(static_cast<int64_t>(nv) * part / parts), v1 = static_cast<int>(static_cast<int64_t>(nv) * (part + 1) / parts);
    const int f0 = max(v0, head > 0 ? 1 : 0), f1 = max(f0, min(v1, (head + p.vocab) / kN));  // whole ones
    const auto fetch = [&](int v) {  // from global memory; -inf where there is no token
        Vec<T> r;
        if (v >= f0 && v < f1) {
            r.w = *reinterpret_cast<const uint4*>(x + (static_cast<int64_t>(v) * kN - head));
        } else {
            T* h = reinterpret_cast<T*>(&r.w);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int tok = v * kN - head + i;
                h[i] = tok >= 0 && tok < p.vocab ? x[tok] : from_f32<T>(-INFINITY);
            }
        }
        return r;
    };
    Vec<T>* const data = reinterpret_cast<Vec<T>*>(s_data);
    const auto get = [&](int v) { return p.staged ? data[v - v0] : fetch(v); };
    // chunk c of the whole vectors; every thread waits for it before it reads one
    const auto chunk_at = [&](int c) { return f0 + static_cast<int>(static_cast<int64_t>(f1 - f0) * c / kChunks); };
    if (p.staged) {
        if (tid < kChunks) {
            const int a = chunk_at(tid), b = chunk_at(tid + 1);
            mbar_arrive_expect_tx(&s_bar[tid], static_cast<uint32_t>(b - a) * 16);
            if (b > a) bulk_g2s(&data[a - v0], x + (static_cast<int64_t>(a) * kN - head), static_cast<uint32_t>(b - a) * 16, &s_bar[tid]);
        }
        if (tid >= 32 && tid < 34) {  // the first and the last vector, where they are not whole
            const int v = tid == 32 ? v0 : v1 - 1;
            if (v >= v0 && v < v1 && !(v >= f0 && v < f1)) data[v - v0] = fetch(v);
        }
        __syncthreads();
    }

    // A: maxima
    float tm = -INFINITY;
    int tv = -1;
    const auto look = [&](int v) {
        const float vm = get(v).max();
        if (vm > tm || tv < 0) tv = v;
        tm = max_nan(tm, vm);
    };
    bool came = true;
    if (p.staged) {
        for (int c = 0; c < kChunks; ++c) {
            came = came && mbar_wait(&s_bar[c], 0);
            const int b = c == kChunks - 1 ? v1 : chunk_at(c + 1);
            for (int v = (c == 0 ? v0 : chunk_at(c)) + tid; v < b; v += kThreads) look(v);
        }
        if (!came) report(p.status, SGEMV_ERR_TIMEOUT);
    } else {
        for (int v = v0 + tid; v < v1; v += kThreads) look(v);
    }
    // a thread's maximum is at least this key; 0 for a thread without a vector
    uint64_t key = tv >= 0 && tm == tm ? key_of(tm, tv * kN - head + kN - 1) : 0;
    float m = tm;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (lane == 0) s_f[0][warp] = m;
    if (p.top > 0) {
        // the warp's maxima, descending over the lanes
#pragma unroll
        for (int len = 2; len <= 32; len <<= 1)
#pragma unroll
            for (int j = len >> 1; j > 0; j >>= 1) {
                const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, key, j);
                const bool keep_max = ((lane & j) == 0) == ((lane & len) == 0);
                key = keep_max ? (key > o ? key : o) : (key < o ? key : o);
            }
        const int r = (p.top + kWarps - 1) / kWarps - 1;
        if (lane == r) s_key[warp] = key;
    }
    if (tid == 0) s_count = 0;
    __syncthreads();
    m = s_f[0][0];
    uint64_t bound = p.top > 0 ? s_key[0] : ~0ull;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        m = max_nan(m, s_f[0][w]);
        if (p.top > 0) bound = min(bound, s_key[w]);
    }
    const bool usable = m < INFINITY;  // neither NaN nor +inf

    // B: sums and candidates. A slice of banned tokens alone (m = -inf) has sums of 0.
    float s = 0.0f, e = 0.0f;
    if (usable) {
        for (bool again = false;; again = true) {
            const float bv = bound == 0 ? -INFINITY : (p.top > 0 ? value_of(bound) : INFINITY);
            for (int v = v0 + tid; v < v1; v += kThreads) {
                const Vec<T> r = get(v);
                if (!again && m > -INFINITY) {
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        const float t = fmaxf(r.at(i) - m, -1e30f);
                        const float w = exp2_approx(t * kLog2e);
                        s += w;
                        e = fmaf(w, t, e);
                    }
                }
                if (p.top > 0 && r.max() >= bv) {
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        const int tok = v * kN - head + i;
                        const uint64_t k = key_of(r.at(i), tok);
                        if (k >= bound && tok >= 0 && tok < p.vocab) {
                            const int at = atomicAdd(&s_count, 1);
                            if (at < kList) s_list[at] = k;
                        }
                    }
                }
            }
            __syncthreads();
            if (s_count <= kList) break;
            // too many: the list's own top-th key is a higher bound
            for (int i = tid; i < kList; i += kThreads) {
                const uint64_t k = s_list[i];
                int larger = 0;
                for (int j = 0; j < kList; ++j) larger += s_list[j] > k;
                if (larger == p.top - 1) s_key[0] = k;
            }
            __syncthreads();
            bound = s_key[0];
            if (tid == 0) s_count = 0;
            __syncthreads();
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
            e += __shfl_xor_sync(0xFFFFFFFFu, e, d);
        }
        if (lane == 0) s_f[1][warp] = s, s_f[2][warp] = e;
    }
    __syncthreads();
    const int cand = usable ? s_count : 0;
    s = 0.0f, e = 0.0f;
    if (usable)
        for (int w = 0; w < kWarps; ++w) s += s_f[1][w], e += s_f[2][w];
    for (int i = tid; i < cand; i += kThreads) {
        const uint64_t k = s_list[i];
        int larger = 0;
        for (int j = 0; j < cand; ++j) larger += s_list[j] > k;
        if (larger < p.top) s_slice.best[larger] = k;
    }
    if (tid == 0) s_slice.m = m, s_slice.s = s, s_slice.e = e, s_slice.n = min(cand, p.top);

    // The whole row's, in every CTA of its cluster.
    float lse_m = m, sum = s, ent = e;
    if (parts > 1) {
        cluster.sync();
        float pm[kMaxCluster];
        for (int i = 0; i < parts; ++i) {
            pm[i] = cluster.map_shared_rank(&s_slice, i)->m;
            lse_m = i == 0 ? pm[0] : max_nan(lse_m, pm[i]);
        }
        sum = 0.0f, ent = 0.0f;
        if (lse_m < INFINITY && lse_m > -INFINITY)
            for (int i = 0; i < parts; ++i) {
                if (pm[i] == -INFINITY) continue;
                const Slice* o = cluster.map_shared_rank(&s_slice, i);
                // sums about pm[i], moved to lse_m
                const float d = pm[i] - lse_m, f = exp2_approx(d * kLog2e), si = o->s * f;
                sum += si;
                ent += si == 0.0f ? 0.0f : fmaf(si, d, o->e * f);
            }
        // the first CTA's list becomes all slices' best
        if (part == 0) {
            for (int i = tid; i < parts * p.top; i += kThreads) {
                const Slice* o = cluster.map_shared_rank(&s_slice, i / p.top);
                s_list[i] = i % p.top < o->n ? o->best[i % p.top] : 0;
            }
        }
    } else {
        __syncthreads();
    }
    const bool bad = !(lse_m < INFINITY), none = lse_m == -INFINITY;
    const float kNan = __int_as_float(0x7FC00000), log_s = logf(sum);
    const auto lp = [&](float f) { return bad ? kNan : (none ? -INFINITY : (f - lse_m) - log_s); };
    if (part == 0) {
        if (parts > 1) __syncthreads();
        if (tid == 0) {
            if (bad) report(p.status, SGEMV_ERR_NONFINITE);
            if (p.lse != nullptr) p.lse[row] = bad ? kNan : (none ? -INFINITY : lse_m + log_s);
            if (p.entropy != nullptr) p.entropy[row] = bad ? kNan : (none ? 0.0f : log_s - ent / sum);
        }
        for (int j = tid; j < p.n_tok; j += kThreads) {
            const int t = p.tokens[static_cast<int64_t>(row) * p.n_tok + j];
            float v = 0.0f;
            if (t >= 0 && t < p.vocab) v = lp(to_f32(x[t]));
            else if (t != -1) {
                v = kNan;
                report(p.status, SGEMV_ERR_ARG);
            }
            p.tok_logp[static_cast<int64_t>(row) * p.n_tok + j] = v;
        }
        const int64_t o = static_cast<int64_t>(row) * p.top;
        const auto put = [&](int rank, uint64_t k) {
            p.top_tok[o + rank] = bad || k == 0 ? -1 : token_of(k);
            p.top_logp[o + rank] = bad ? kNan : (k == 0 ? -INFINITY : lp(value_of(k)));
        };
        if (parts == 1) {
            for (int j = tid; j < p.top; j += kThreads) put(j, !bad && j < s_slice.n ? s_slice.best[j] : 0);
        } else {
            const int n = parts * p.top;
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t k = s_list[i];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += s_list[j] > k || (s_list[j] == k && j < i);  // only the empty ones are equal
                if (rank < p.top) put(rank, bad ? 0 : k);
            }
        }
    }
    if (p.logp != nullptr) {
        float* const out = p.logp + static_cast<int64_t>(row) * p.vocab;
        const int t0 = max(0, v0 * kN - head), t1 = min(p.vocab, v1 * kN - head);
        if (p.staged) {
            const T* const h = reinterpret_cast<const T*>(s_data) + (head - v0 * kN);
            for (int t = t0 + tid; t < t1; t += kThreads) out[t] = lp(to_f32(h[t]));
        } else {
            for (int t = t0 + tid; t < t1; t += kThreads) out[t] = lp(to_f32(x[t]));
        }
    }
    if (parts > 1) cluster.sync();  // the first CTA has read the others' shared memory
}

template <typename T, int kThreads>
cudaError_t launch_rows(const LogprobParams& p, int parts, uint32_t smem, cudaStream_t s) {
    auto kern = logprobs_kernel<T, kThreads>;
    static std::atomic<int> attr_smem[64];  // per device: dynamic shared memory already enabled
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (attr_smem[dev].load() < static_cast<int>(smem)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        attr_smem[dev].store(static_cast<int>(smem));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T>
cudaError_t launch_logprobs(LogprobParams p, int sms, cudaStream_t s) {
    const int64_t nv = (static_cast<int64_t>(p.vocab) + 2 * Vec<T>::kN - 2) / Vec<T>::kN;  // with any alignment
    // One CTA a row while two fit an SM; more where slices are longer, or rows too few to fill the GPU with slices of 4 KB.
    int parts = 1;
    while (parts < kMaxCluster && (nv * 16 > 92 * 1024 * static_cast<int64_t>(parts) ||
                                   (static_cast<int64_t>(p.rows) * parts * 2 <= sms && nv > 512 * parts)))
        parts *= 2;
    const int64_t slice = (nv + parts - 1) / parts * 16;
    p.staged = slice <= 196 * 1024;  // else the passes read global memory
    const uint32_t smem = p.staged ? static_cast<uint32_t>(slice) : 0;
    if (static_cast<int64_t>(p.rows) * parts > INT_MAX) return cudaErrorInvalidValue;
    // four warps where a slice gives 16 no more than a vector a thread (then every element fits the list)
    return slice >= 16 * 1024 ? launch_rows<T, 512>(p, parts, smem, s) : launch_rows<T, 128>(p, parts, smem, s);
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
