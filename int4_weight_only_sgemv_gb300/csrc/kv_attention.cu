// Attention over the paged 4-bit KV cache: the entry point (argument checks, choice of the kernel).
#include <climits>

#include "kv_chunk.cuh"

namespace sgemv {
cudaError_t launch_decode_f16(int dim, int group, const AttnParams& p, int sms, cudaStream_t s);
cudaError_t launch_decode_bf16(int dim, int group, const AttnParams& p, int sms, cudaStream_t s);
cudaError_t launch_chunk(int dtype, int dim, int group, const AttnParams& p, cudaStream_t s);
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
    if (static_cast<int64_t>(q.n_tokens) * (q.heads_q / layout->heads) > (1 << 30)) return SGEMV_ERR_SHAPE;  // rows in 32 bits
    if (q.n_req > (1 << 30)) return SGEMV_ERR_SHAPE;  // and the runs of requests that threads look after
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
    if (!is_aligned(q.tree_dev, 8) || !strides_aligned(q.n_tokens, q.q_token_stride, q.heads_q, q.q_head_stride) ||
        !strides_aligned(q.n_tokens, q.out_token_stride, q.heads_q, q.out_head_stride))
        return SGEMV_ERR_ALIGN;
    // (rows between others, as those of a fused projection, may be out's: what lies from its first to its last byte is looked at
    // only where nothing else has a place there)
    const Bytes out = span_bytes(q.out_dev, q.n_tokens, q.out_token_stride, q.heads_q, q.out_head_stride, layout->dim);
    const Bytes qs = span_bytes(q.q_dev, q.n_tokens, q.q_token_stride, q.heads_q, q.q_head_stride, layout->dim);
    const Bytes cache(cache_dev, layout->total_bytes), ws(q.workspace_dev, SGEMV_KV_WORKSPACE);
    const Bytes lse(q.lse_dev, 4ull * q.n_tokens * q.heads_q);
    const Bytes written[] = {ws, lse, {status_dev, 4}};
    const Bytes read[] = {cache, {q.q_start_dev, 4ull * q.n_req + 4}, {q.len_dev, 4ull * q.n_req}, {q.tree_dev, 8ull * q.n_tokens}};
    if (!apart(written, read) || meet(out, cache) || meet(out, ws) || meet(qs, ws)) return SGEMV_ERR_ARG;
    const uint64_t all = 2ull * q.n_tokens * q.heads_q * layout->dim;
    if (q.out_dev != q.q_dev && out.size == all && qs.size == all && meet(out, qs)) return SGEMV_ERR_ARG;
    AttnParams p;
    p.cache = static_cast<const uint8_t*>(cache_dev);
    p.sub_bytes = layout->sub_bytes;
    p.head_bytes = layout->head_bytes;
    p.page_bytes = layout->page_bytes;
    p.q = q;
    // A window that no length reaches hides nothing, and without it positions minus the window stay in 32 bits.
    if (q.window >= kMaxLen) p.q.window = 0;
    p.status = status_dev;
    p.heads = layout->heads;
    p.page = layout->page;
    p.log2_page = 0;
    while ((1 << p.log2_page) < layout->page) ++p.log2_page;
    p.n_pages = layout->n_pages;
    p.ratio = q.heads_q / layout->heads;
    p.log2_ratio = 0;
    while ((1 << p.log2_ratio) < p.ratio) ++p.log2_ratio;
    if ((1 << p.log2_ratio) != p.ratio) p.log2_ratio = -1;
    p.scale_log2 = q.scale * 1.44269504088896340736f;
    DeviceInfo di;
    rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.max_rows = chunk_threshold(layout->dim, layout->heads, p.ratio, q.n_req, q.n_tokens, q.max_q, di.sm_count);
    cudaError_t e = q.dtype == SGEMV_F16 ? launch_decode_f16(layout->dim, layout->group, p, di.sm_count, s)
                                         : launch_decode_bf16(layout->dim, layout->group, p, di.sm_count, s);
    if (e == cudaSuccess && p.max_rows < INT_MAX) e = launch_chunk(q.dtype, layout->dim, layout->group, p, s);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
