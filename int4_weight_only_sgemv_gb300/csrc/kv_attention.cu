// Attention over the paged 4-bit KV cache.
//
// With q the quantised row's integers, s its scale and z its zero point, k = s (q - z) and v the same:
//   score_j = scale * x . k_j,  out = sum_j e^(score_j - m) v_j / sum_j e^(score_j - m),  m = max_j score_j,
// with the maximum and the sum kept while the keys go by.
//
// One warp a (token, query head): 32 keys at a time, one a lane for the scores, then all lanes over the dims.
#include <algorithm>
#include <climits>

#include "kv_common.cuh"

namespace sgemv {

namespace {

constexpr int kAttnThreads = 128;

struct AttnParams {
    const uint8_t* cache;
    uint64_t sub_bytes, head_bytes, page_bytes;
    sgemv_kv_query q;
    int32_t* status;
    int heads, group, page, n_pages, ratio;
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
    } else if ((static_cast<int64_t>(len) + p.page - 1) / p.page > p.q.table_cols) {
        report(p.status, SGEMV_ERR_SHAPE);
        s.n = 0;
    }
    return s;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kAttnThreads) attention_kernel(const AttnParams p) {
    __shared__ float s_x[kAttnThreads / 32][D];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAttnThreads / 32) + warp;
    if (unit >= static_cast<int64_t>(p.q.n_tokens) * p.q.heads_q) return;
    const int tok = static_cast<int>(unit / p.q.heads_q), a = static_cast<int>(unit % p.q.heads_q);
    // the request of this token: the last one that starts at or before it
    int lo = 0, hi = p.q.n_req - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.q.q_start_dev[mid] <= tok) lo = mid; else hi = mid - 1;
    }
    const Span sp = span_of(p, lo);
    const int i = tok - sp.first;
    if (i < 0 || i >= sp.n) return;
    const int old = sp.len - sp.n;  // positions before the new tokens (negative where len < n)
    const int at = old + i;
    const uint64_t tree = p.q.tree_dev != nullptr ? p.q.tree_dev[tok] : 0;
    const bool has_tree = p.q.tree_dev != nullptr;
    const int end = has_tree ? sp.len : at + 1;
    const int begin = p.q.window > 0 ? max(0, at - p.q.window + 1) : 0;
    const T* x = static_cast<const T*>(p.q.q_dev) + tok * p.q.q_token_stride + a * p.q.q_head_stride;
    for (int d = lane; d < D; d += 32) s_x[warp][d] = to_f32(x[d]) * p.q.scale;
    __syncwarp();
    const int32_t* row = p.q.table_dev + lo * p.q.table_stride;
    const int head = a / p.ratio;
    constexpr int kWords = D / 128 > 0 ? D / 128 : 1;  // 16-bit words of V a lane has (half the lanes where D is 64)
    float m = -INFINITY, l = 0.0f, acc[kWords][4] = {};
    for (int j0 = begin & ~31; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        bool see = j >= begin && j < end;
        if (has_tree && j >= old) see = see && ((tree >> (j - old)) & 1);
        int id = see ? row[j / p.page] : 0;
        if (id < 0 || id >= p.n_pages) {
            report(p.status, SGEMV_ERR_ARG);
            see = false;
        }
        const uint8_t* sub = nullptr;
        float score = -INFINITY;
        const int tau = j % kSub;
        if (see) {
            sub = p.cache + id * p.page_bytes + head * p.head_bytes + (j % p.page) / kSub * p.sub_bytes;
            score = 0.0f;
            for (int g = 0; g < D / G; ++g) {
                float dot = 0.0f, sum = 0.0f;
                for (int d = g * G; d < (g + 1) * G; d += 8) {
                    constexpr int P = D < 128 ? D : 128;
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(sub + d / P * 8 * P + tau * (P / 2) + d % P / 2);
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float f = s_x[warp][d + n];
                        dot += f * static_cast<float>((w >> (4 * n)) & 15u);
                        sum += f;
                    }
                }
                const __half2 sz = *reinterpret_cast<const __half2*>(sub + 16 * D + 64 * g + 4 * tau);
                score += __low2float(sz) * (dot - __high2float(sz) * sum);
            }
        }
        float top = score;
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if (top == -INFINITY) continue;
        const float next = fmaxf(m, top);
        const float fade = expf(m - next);
        m = next;
        const float w = see ? expf(score - m) : 0.0f;
        float total = w;
        for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
        l = l * fade + total;
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            for (int n = 0; n < 4; ++n) acc[k][n] *= fade;
        for (int t = 0; t < 32; ++t) {
            const float wt = __shfl_sync(0xFFFFFFFFu, w, t);
            const uint8_t* st = reinterpret_cast<const uint8_t*>(
                __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(sub), t));
            if (st == nullptr) continue;
            const int c = lane & 7;
            const int tt = (j0 + t) % kSub;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                const int blk = (lane >> 3) + 4 * k;  // block of 32 dims
                if (blk >= D / 32) continue;
                const int w_ = ((tt >> 1) & 1) * (D / 32) + blk;
                const uint32_t v = *reinterpret_cast<const uint16_t*>(st + 8 * D + (w_ >> 2) * 512 +
                                                                      (4 * c + (tt >> 2)) * 16 + (w_ & 3) * 4 + (tt & 1) * 2);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int g = (c + 8 * n + 32 * blk) / G;
                    const __half2 sz = *reinterpret_cast<const __half2*>(st + 16 * D + 64 * (D / G) + 64 * g + 4 * tt);
                    acc[k][n] += wt * __low2float(sz) * (static_cast<float>((v >> (4 * n)) & 15u) - __high2float(sz));
                }
            }
        }
    }
    T* o = static_cast<T*>(p.q.out_dev) + tok * p.q.out_token_stride + a * p.q.out_head_stride;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const int blk = (lane >> 3) + 4 * k;
        if (blk >= D / 32) continue;
#pragma unroll
        for (int n = 0; n < 4; ++n) o[(lane & 7) + 8 * n + 32 * blk] = from_f32<T>(acc[k][n] * inv);
    }
    if (p.q.lse_dev != nullptr && lane == 0) p.q.lse_dev[static_cast<int64_t>(tok) * p.q.heads_q + a] = m + logf(l);
}

template <typename T>
cudaError_t launch_attention(const sgemv_kv_layout& L, const AttnParams& p, cudaStream_t s) {
    const int64_t units = static_cast<int64_t>(p.q.n_tokens) * p.q.heads_q;
    const int64_t blocks = (units + kAttnThreads / 32 - 1) / (kAttnThreads / 32);
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kAttnThreads);
#define SGEMV_KV_CASE(D, G) \
    if (L.dim == D && L.group == G) return launch_pdl(attention_kernel<T, D, G>, grid, block, 0, s, p);
    SGEMV_KV_CASE(64, 64)
    SGEMV_KV_CASE(128, 64)
    SGEMV_KV_CASE(128, 128)
    SGEMV_KV_CASE(256, 64)
    SGEMV_KV_CASE(256, 128)
#undef SGEMV_KV_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_kv_attention(const sgemv_kv_layout* layout, const void* cache_dev, const sgemv_kv_query* query,
                                  int32_t* status_dev, void* stream) {
    int rc = check_kv_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if (query == nullptr) return SGEMV_ERR_ARG;
    const sgemv_kv_query& q = *query;
    if ((q.dtype != SGEMV_F16 && q.dtype != SGEMV_BF16) || q.n_req < 0 || q.n_tokens < 0 || q.max_q < 0 ||
        q.window < 0 || q.table_cols < 1 || q.table_stride < q.table_cols || !(q.scale == q.scale))
        return SGEMV_ERR_ARG;
    if (q.heads_q < 1 || q.heads_q % layout->heads != 0 || q.heads_q > 16384) return SGEMV_ERR_SHAPE;
    if (q.tree_dev != nullptr && (q.window != 0 || q.max_q > 64)) return SGEMV_ERR_ARG;
    if (q.n_req == 0 || q.n_tokens == 0 || q.max_q == 0) return SGEMV_OK;
    const void* must[] = {cache_dev, q.q_dev, q.q_start_dev, q.len_dev, q.table_dev, q.out_dev, q.workspace_dev};
    for (const void* x : must)
        if (x == nullptr) return SGEMV_ERR_ARG;
    if (q.workspace_bytes < SGEMV_KV_WORKSPACE) return SGEMV_ERR_ARG;
    const void* lines[] = {cache_dev, q.q_dev, q.out_dev, q.workspace_dev};
    for (const void* x : lines)
        if (!is_aligned(x, 16)) return SGEMV_ERR_ALIGN;
    const void* words[] = {q.q_start_dev, q.len_dev, q.table_dev, q.lse_dev, status_dev};
    for (const void* x : words)
        if (!is_aligned(x, 4)) return SGEMV_ERR_ALIGN;
    if (!is_aligned(q.tree_dev, 8) || q.q_token_stride % 8 || q.q_head_stride % 8 || q.out_token_stride % 8 ||
        q.out_head_stride % 8)
        return SGEMV_ERR_ALIGN;
    AttnParams p;
    p.cache = static_cast<const uint8_t*>(cache_dev);
    p.sub_bytes = layout->sub_bytes;
    p.head_bytes = layout->head_bytes;
    p.page_bytes = layout->page_bytes;
    p.q = q;
    p.status = status_dev;
    p.heads = layout->heads;
    p.group = layout->group;
    p.page = layout->page;
    p.n_pages = layout->n_pages;
    p.ratio = q.heads_q / layout->heads;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = q.dtype == SGEMV_F16 ? launch_attention<__half>(*layout, p, s)
                                               : launch_attention<__nv_bfloat16>(*layout, p, s);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
