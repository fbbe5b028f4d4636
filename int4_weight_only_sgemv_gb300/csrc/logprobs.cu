// Log-probabilities of rows of logits: lse = m + ln sum exp(x - m), lp = x - lse, entropy = lse - sum p x
// = ln S - sum e^(x-m) (x-m) / S with S = sum e^(x-m), and the best `top` tokens of each row.
//
// One CTA a row; the row is read once for the statistics, once for every alternative and once for the full row.
#include <cstdint>

#include "kv_common.cuh"

namespace sgemv {

namespace {

constexpr int kRowThreads = 512;

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

// Larger for a larger logit; equal logits by the lower token. -0 counts as +0.
__device__ __forceinline__ uint64_t key_of(float x, int tok) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) == 0) u = 0;
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return (static_cast<uint64_t>(u) << 32) | static_cast<uint32_t>(~tok);
}

template <typename F, typename V>
__device__ __forceinline__ V block_reduce(V v, V* s_red, F f) {
    for (int d = 16; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s_red[0];
    for (int w = 1; w < kRowThreads / 32; ++w) v = f(v, s_red[w]);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) logprobs_kernel(const LogprobParams p) {
    __shared__ float s_f[kRowThreads / 32];
    __shared__ uint64_t s_k[kRowThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x, tid = threadIdx.x;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    const auto fmax2 = [](float a, float b) { return fmaxf(a, b); };
    const auto fadd2 = [](float a, float b) { return a + b; };
    const auto kmax = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
    float m = -INFINITY, bad = 0.0f;
    for (int i = tid; i < p.vocab; i += kRowThreads) {
        const float f = to_f32(x[i]);
        m = fmaxf(m, f);
        if (!(f < INFINITY)) bad = 1.0f;
    }
    m = block_reduce(m, s_f, fmax2);
    bad = block_reduce(bad, s_f, fmax2);
    const bool none = m == -INFINITY;  // every token is banned
    float s = 0.0f, e = 0.0f;
    if (!none && bad == 0.0f) {
        for (int i = tid; i < p.vocab; i += kRowThreads) {
            const float t = to_f32(x[i]) - m;
            const float w = expf(t);
            s += w;
            if (w > 0.0f) e += w * t;
        }
    }
    s = block_reduce(s, s_f, fadd2);
    e = block_reduce(e, s_f, fadd2);
    const float log_s = logf(s);
    const float kNan = __int_as_float(0x7FC00000);
    const float lse = bad != 0.0f ? kNan : (none ? -INFINITY : m + log_s);
    const auto lp = [&](float f) { return bad != 0.0f ? kNan : (none ? -INFINITY : (f - m) - log_s); };
    if (tid == 0) {
        if (bad != 0.0f) report(p.status, SGEMV_ERR_NONFINITE);
        if (p.lse != nullptr) p.lse[row] = lse;
        if (p.entropy != nullptr) p.entropy[row] = bad != 0.0f ? kNan : (none ? 0.0f : log_s - e / s);
    }
    for (int j = tid; j < p.n_tok; j += kRowThreads) {
        const int t = p.tokens[static_cast<int64_t>(row) * p.n_tok + j];
        float v = 0.0f;
        if (t >= 0 && t < p.vocab) v = lp(to_f32(x[t]));
        else if (t != -1) {
            v = kNan;
            report(p.status, SGEMV_ERR_ARG);
        }
        p.tok_logp[static_cast<int64_t>(row) * p.n_tok + j] = v;
    }
    if (p.logp != nullptr)
        for (int i = tid; i < p.vocab; i += kRowThreads) p.logp[static_cast<int64_t>(row) * p.vocab + i] = lp(to_f32(x[i]));
    uint64_t last = ~0ull;
    for (int j = 0; j < p.top; ++j) {
        uint64_t best = 0;
        if (bad == 0.0f) {
            for (int i = tid; i < p.vocab; i += kRowThreads) {
                const uint64_t k = key_of(to_f32(x[i]), i);
                if (k < last && k > best) best = k;
            }
        }
        best = block_reduce(best, s_k, kmax);
        last = best;
        if (tid == 0) {
            const int64_t o = static_cast<int64_t>(row) * p.top + j;
            const int t = best != 0 ? static_cast<int>(~static_cast<uint32_t>(best)) : -1;
            p.top_tok[o] = t;
            p.top_logp[o] = bad != 0.0f ? kNan : (t < 0 ? -INFINITY : lp(to_f32(x[t])));
        }
    }
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
    LogprobParams p;
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
    const dim3 grid(rows), block(kRowThreads);
    const cudaError_t e = dtype == SGEMV_F16    ? launch_pdl(logprobs_kernel<__half>, grid, block, 0, s, p)
                          : dtype == SGEMV_BF16 ? launch_pdl(logprobs_kernel<__nv_bfloat16>, grid, block, 0, s, p)
                                                : launch_pdl(logprobs_kernel<float>, grid, block, 0, s, p);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
