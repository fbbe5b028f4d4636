// Causal attention over packed prompts: the entry point (argument checks, tensor maps, launch).
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "prompt_attention.cuh"
#include "tensor_map.cuh"

namespace sgemv {

namespace {

constexpr float kLog2E = 1.44269504088896340736f;

// Tiles of `tokens` tokens of `heads` neighbouring heads, 64 dims of a row at a time, swizzled for the tensor cores. (A stride of an axis of
// length 1 is not used.)
bool map_rows(CUtensorMap* map, const void* base, const sgemv_prompt_query& q, int all_heads, int64_t token_stride, int64_t head_stride, int tokens,
              int heads) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(q.dim), static_cast<cuuint64_t>(all_heads), static_cast<cuuint64_t>(q.n_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(all_heads > 1 ? head_stride : q.dim) * 2,
                                   static_cast<cuuint64_t>(q.n_tokens > 1 ? token_stride : static_cast<int64_t>(all_heads) * q.dim) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
    return encode_map(map, q.dtype == SGEMV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int D>
cudaError_t launch_prompt(const CUtensorMap& qm, const CUtensorMap& k, const CUtensorMap& v, const PromptParams& p, unsigned grid, cudaStream_t s) {
    using S = PromptShape<D>;
    auto kern = prompt_kernel<T, D>;
    static std::atomic<int> attr_set[64];  // per device: dynamic shared memory already enabled
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (attr_set[dev].load() == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, kern);
        if (e != cudaSuccess) return e;
        if (a.numRegs != S::kRegs) return cudaErrorInvalidKernelImage;  // the roles' split would wait for registers for ever
        attr_set[dev].store(1);
    }
    return launch_pdl(kern, dim3(grid), dim3(S::kThreads), S::kSmem, s, qm, k, v, p);
}

}  // namespace

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_prompt_attention(const sgemv_prompt_query* query, int32_t* status_dev, void* stream) {
    if (query == nullptr) return SGEMV_ERR_ARG;
    const sgemv_prompt_query& q = *query;
    if ((q.dtype != SGEMV_F16 && q.dtype != SGEMV_BF16) || q.n_req < 0 || q.n_tokens < 0 || q.window < 0 || (q.causal != 0 && q.causal != 1) ||
        (q.window > 0 && q.causal == 0) || !(std::fabs(q.scale * kLog2E) < INFINITY))
        return SGEMV_ERR_ARG;
    if (q.dim != 64 && q.dim != 128) return SGEMV_ERR_SHAPE;
    if (q.heads < 1 || q.heads_q < q.heads || q.heads_q % q.heads != 0 || q.heads_q > 16384) return SGEMV_ERR_SHAPE;
    // (A CTA looks for a segment among n_req / 384 requests, some 80 ns each, while others wait for it with a limit of 200 ms: 14 ms at 2^26.)
    if (static_cast<int64_t>(q.n_tokens) * q.heads_q > (1 << 30) || q.n_req > (1 << 26)) return SGEMV_ERR_SHAPE;
    if (q.n_req == 0 || q.n_tokens == 0) return SGEMV_OK;
    const void* must[] = {q.q_dev, q.k_dev, q.v_dev, q.start_dev, q.out_dev};
    for (const void* x : must)
        if (x == nullptr) return SGEMV_ERR_ARG;
    const void* lines[] = {q.q_dev, q.k_dev, q.v_dev, q.out_dev};
    for (const void* x : lines)
        if (!is_aligned(x, 16)) return SGEMV_ERR_ALIGN;
    const void* words[] = {q.start_dev, q.length_dev, q.lse_dev, status_dev};
    for (const void* x : words)
        if (!is_aligned(x, 4)) return SGEMV_ERR_ALIGN;
    if (!strides_aligned(q.n_tokens, q.q_token_stride, q.heads_q, q.q_head_stride) ||
        !strides_aligned(q.n_tokens, q.out_token_stride, q.heads_q, q.out_head_stride) ||
        !strides_aligned(q.n_tokens, q.k_token_stride, q.heads, q.k_head_stride) ||
        !strides_aligned(q.n_tokens, q.v_token_stride, q.heads, q.v_head_stride))
        return SGEMV_ERR_ALIGN;
    constexpr int64_t kFar = 1ll << 38;  // a tensor map's strides are below 2^40 bytes
    const int64_t strides[][2] = {{q.n_tokens, q.q_token_stride}, {q.heads_q, q.q_head_stride}, {q.n_tokens, q.k_token_stride}, {q.heads, q.k_head_stride},
                                  {q.n_tokens, q.v_token_stride}, {q.heads, q.v_head_stride}, {q.n_tokens, q.out_token_stride},
                                  {q.heads_q, q.out_head_stride}};
    for (const auto& s : strides)
        if (s[0] > 1 && (s[1] < 1 || s[1] > kFar)) return SGEMV_ERR_SHAPE;
    // out's rows do not overlap
    if (q.n_tokens > 1 || q.heads_q > 1) {
        const bool heads_inside = q.heads_q > 1 && (q.n_tokens < 2 || q.out_head_stride <= q.out_token_stride);
        const int64_t inner = heads_inside ? q.out_head_stride : q.out_token_stride, n_inner = heads_inside ? q.heads_q : q.n_tokens;
        const int64_t outer = heads_inside ? q.out_token_stride : q.out_head_stride, n_outer = heads_inside ? q.n_tokens : q.heads_q;
        if (inner < q.dim || (n_outer > 1 && outer < (n_inner - 1) * inner + q.dim)) return SGEMV_ERR_ARG;
    }
    // (rows between others, as those of a fused projection, may be out's: what lies from its first to its last byte is looked at only where
    // nothing else has a place there)
    const uint64_t all = 2ull * q.n_tokens * q.heads_q * q.dim;
    const auto span = [&](const void* p, int64_t ts, int heads, int64_t hs) {
        return span_bytes(p, q.n_tokens, q.n_tokens > 1 ? ts : 0, heads, heads > 1 ? hs : 0, q.dim);
    };
    const Bytes out = span(q.out_dev, q.out_token_stride, q.heads_q, q.out_head_stride), qs = span(q.q_dev, q.q_token_stride, q.heads_q, q.q_head_stride);
    const Bytes ks = span(q.k_dev, q.k_token_stride, q.heads, q.k_head_stride), vs = span(q.v_dev, q.v_token_stride, q.heads, q.v_head_stride);
    const uint64_t kv_all = 2ull * q.n_tokens * q.heads * q.dim;
    const Bytes lse(q.lse_dev, 4ull * q.n_tokens * q.heads_q), status(status_dev, 4);
    const Bytes start(q.start_dev, 4ull * q.n_req + 4), length(q.length_dev, 4ull * q.n_req);
    const Bytes written[] = {lse, status}, read[] = {start, length};
    if (!apart(written, read)) return SGEMV_ERR_ARG;
    for (const Bytes& b : {lse, status, start, length}) {
        if (out.size == all && meet(out, b)) return SGEMV_ERR_ARG;
        if ((b.at == lse.at || b.at == status.at) && ((qs.size == all && meet(qs, b)) || (ks.size == kv_all && meet(ks, b)) || (vs.size == kv_all && meet(vs, b))))
            return SGEMV_ERR_ARG;
    }
    if (q.out_dev != q.q_dev && out.size == all && qs.size == all && meet(out, qs)) return SGEMV_ERR_ARG;
    if (q.out_dev == q.q_dev && ((q.n_tokens > 1 && q.q_token_stride != q.out_token_stride) || (q.heads_q > 1 && q.q_head_stride != q.out_head_stride)))
        return SGEMV_ERR_ARG;
    if (out.size == all && ((ks.size == kv_all && meet(out, ks)) || (vs.size == kv_all && meet(out, vs)))) return SGEMV_ERR_ARG;
    PromptParams p;
    p.q = q;
    // A window that no request reaches hides nothing, and without it positions minus the window stay in 32 bits.
    if (q.window >= q.n_tokens) p.q.window = 0;
    p.status = status_dev;
    p.ratio = q.heads_q / q.heads;
    p.out32 = is_aligned(q.out_dev, 32) && (q.n_tokens < 2 || q.out_token_stride % 16 == 0) && (q.heads_q < 2 || q.out_head_stride % 16 == 0);
    p.scale_log2 = q.scale * kLog2E;
    p.unscale = p.scale_log2 == 0.0f ? 0.693147180559945309f : static_cast<float>(static_cast<double>(q.scale) / p.scale_log2);
    p.sub = std::min(p.ratio, 128);
    while (p.ratio % p.sub != 0) --p.sub;
    p.tokens = 128 / p.sub;
    p.groups = q.heads_q / p.sub;
    // at most so many segments: every request's last may be short
    const int64_t most = (static_cast<int64_t>(q.n_tokens) / (2 * p.tokens) + q.n_req) * p.groups;
    if (most > INT_MAX) return SGEMV_ERR_SHAPE;
    p.most = static_cast<int>(most);
    CUtensorMap q_map, k_map, v_map;
    if (!map_rows(&q_map, q.q_dev, q, q.heads_q, q.q_token_stride, q.q_head_stride, p.tokens, p.sub) ||
        !map_rows(&k_map, q.k_dev, q, q.heads, q.k_token_stride, q.k_head_stride, 128, 1) ||
        !map_rows(&v_map, q.v_dev, q, q.heads, q.v_token_stride, q.v_head_stride, 128, 1))
        return SGEMV_ERR_CUDA;
    DeviceInfo di;
    const int rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(most, di.sm_count));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool half = q.dtype == SGEMV_F16;
    const cudaError_t e = q.dim == 64 ? (half ? launch_prompt<__half, 64>(q_map, k_map, v_map, p, grid, s) : launch_prompt<__nv_bfloat16, 64>(q_map, k_map, v_map, p, grid, s))
                                      : (half ? launch_prompt<__half, 128>(q_map, k_map, v_map, p, grid, s) : launch_prompt<__nv_bfloat16, 128>(q_map, k_map, v_map, p, grid, s));
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
