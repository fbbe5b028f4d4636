// The paged 4-bit KV cache: its layout, writing K and V rows into it, and reading them back.
//
// Work unit of both kernels: one panel of min(dim, 128) dims of one (token, head), by width / 4 lanes: a warp, or
// a half warp where dim is 64. Lane l holds dims 4l .. 4l+3 of the panel, so a quantisation group of 64 or 128
// is 16 or 32 neighbouring lanes and its range is a few shuffles.
#include <climits>

#include "kv_common.cuh"

namespace sgemv {

namespace {

constexpr int kCacheThreads = 256;

struct CacheParams {
    uint8_t* cache;
    const int64_t* slots;
    int32_t* status;
    const void* k;
    const void* v;
    int64_t k_token, k_head, v_token, v_head;
    void* k_out;
    void* v_out;
    uint64_t sub_bytes, head_bytes, page_bytes;
    int64_t n_slots;  // slots of the cache
    int64_t units;
    int heads, page, n_tokens;
};

// Quantises the 4 values of this lane with the group of `lanes` neighbouring lanes: nibbles (first dim lowest),
// scale and zero point. Binary32, no fused multiply-add, division rounded to nearest.
__device__ __forceinline__ uint32_t quantise(const float (&x)[4], int lanes, __half& s16, float& z, bool& bad) {
    float mn = fminf(fminf(fminf(x[0], x[1]), fminf(x[2], x[3])), 0.0f);
    float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), 0.0f);
    // fminf and fmaxf drop NaN: it is looked for by itself
    int nan = (x[0] != x[0]) | (x[1] != x[1]) | (x[2] != x[2]) | (x[3] != x[3]);
    for (int d = 1; d < lanes; d <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
        nan |= __shfl_xor_sync(0xFFFFFFFFu, nan, d);
    }
    s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
    bad = nan || __hisinf(s16) || isinf(mn) || isinf(mx);
    if (bad || __half2float(s16) == 0.0f) s16 = __float2half_rn(1.0f);
    const float s = __half2float(s16);
    if (bad) {
        z = 0.0f;
        return 0;
    }
    z = fminf(fmaxf(rintf(__fdiv_rn(-mn, s)), 0.0f), 15.0f) + 0.0f;  // + 0: never -0
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float f = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(x[j], s)), z), 0.0f), 15.0f);
        q |= static_cast<uint32_t>(f) << (4 * j);
    }
    return q;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = to_f32(h[j]);
}

// Byte offset in a subtile of the 16-bit word of V with dims c + 8n + 32i (n = 0..3) of token tau.
template <int D>
__device__ __forceinline__ uint32_t v_word(int tau, int c, int i) {
    const int w = ((tau >> 1) & 1) * (D / 32) + i;
    return 8 * D + (w >> 2) * 512 + (4 * c + (tau >> 2)) * 16 + (w & 3) * 4 + (tau & 1) * 2;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kCacheThreads) append_kernel(const CacheParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kPanel = D < 128 ? D : 128, kPanels = D / kPanel, kLanes = kPanel / 4;
    const int lane = threadIdx.x % kLanes;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x) / kLanes;
    const bool in = unit < p.units;  // a half warp may be past the end: it still takes part in the shuffles
    const int panel = static_cast<int>(unit % kPanels);
    const int head = static_cast<int>(unit / kPanels % p.heads);
    const int64_t tok = unit / kPanels / p.heads;
    int64_t slot = in ? p.slots[tok] : -1;
    if (slot >= p.n_slots) {
        report(p.status, SGEMV_ERR_ARG);
        slot = -1;
    }
    float x[4] = {}, y[4] = {};
    if (slot >= 0) {
        load4(static_cast<const T*>(p.k) + tok * p.k_token + head * p.k_head + panel * kPanel + 4 * lane, x);
        load4(static_cast<const T*>(p.v) + tok * p.v_token + head * p.v_head + panel * kPanel + 4 * lane, y);
    }
    __half ks, vs;
    float kz, vz;
    bool kbad, vbad;
    const uint32_t kq = quantise(x, G / 4, ks, kz, kbad);
    const uint32_t vq = quantise(y, G / 4, vs, vz, vbad);
    // V's word (i, c) takes the nibbles c + 8n + 32i: lane 8i + 2n + c / 4 of the panel, place c % 4
    const int c = lane & 7, i = lane >> 3;
    const int first = (threadIdx.x & 31) - lane + 8 * i + (c >> 2);
    uint32_t vw = 0;
#pragma unroll
    for (int n = 0; n < 4; ++n)
        vw |= ((__shfl_sync(0xFFFFFFFFu, vq, first + 2 * n) >> (4 * (c & 3))) & 15u) << (4 * n);
    if (slot < 0) return;
    if (kbad || vbad) report(p.status, SGEMV_ERR_NONFINITE);
    const int at = static_cast<int>(slot % p.page);
    uint8_t* sub = p.cache + static_cast<uint64_t>(slot / p.page) * p.page_bytes + head * p.head_bytes +
                   (at / kSub) * p.sub_bytes;
    const int tau = at % kSub;
    *reinterpret_cast<uint16_t*>(sub + panel * 8 * kPanel + tau * (kPanel / 2) + 2 * lane) = static_cast<uint16_t>(kq);
    *reinterpret_cast<uint16_t*>(sub + v_word<D>(tau, c, i + 4 * panel)) = static_cast<uint16_t>(vw);
    if (lane % (G / 4) == 0) {
        const int grp = panel * (kPanel / G) + lane / (G / 4);
        const __half2 k2 = __halves2half2(ks, __float2half_rn(kz)), v2 = __halves2half2(vs, __float2half_rn(vz));
        *reinterpret_cast<__half2*>(sub + 16 * D + 64 * grp + 4 * tau) = k2;
        *reinterpret_cast<__half2*>(sub + 16 * D + 64 * (D / G) + 64 * grp + 4 * tau) = v2;
    }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]) {
    T h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = from_f32<T>(x[j]);
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
    else *reinterpret_cast<float4*>(p) = make_float4(h[0], h[1], h[2], h[3]);
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const CacheParams p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kPanel = D < 128 ? D : 128, kPanels = D / kPanel, kLanes = kPanel / 4;
    const int lane = threadIdx.x % kLanes;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x) / kLanes;
    const bool in = unit < p.units;
    const int panel = static_cast<int>(unit % kPanels);
    const int head = static_cast<int>(unit / kPanels % p.heads);
    const int64_t tok = unit / kPanels / p.heads;
    int64_t slot = in ? p.slots[tok] : -1;
    if (slot >= p.n_slots) {
        report(p.status, SGEMV_ERR_ARG);
        slot = -1;
    }
    uint32_t kq = 0, vw = 0;
    float ks = 0.0f, kz = 0.0f, vs = 0.0f, vz = 0.0f;
    const int c = lane & 7, i = lane >> 3;
    if (slot >= 0) {
        const int at = static_cast<int>(slot % p.page);
        const uint8_t* sub = p.cache + static_cast<uint64_t>(slot / p.page) * p.page_bytes + head * p.head_bytes +
                             (at / kSub) * p.sub_bytes;
        const int tau = at % kSub;
        kq = *reinterpret_cast<const uint16_t*>(sub + panel * 8 * kPanel + tau * (kPanel / 2) + 2 * lane);
        vw = *reinterpret_cast<const uint16_t*>(sub + v_word<D>(tau, c, i + 4 * panel));
        const int grp = panel * (kPanel / G) + lane / (G / 4);
        const __half2 k2 = *reinterpret_cast<const __half2*>(sub + 16 * D + 64 * grp + 4 * tau);
        const __half2 v2 = *reinterpret_cast<const __half2*>(sub + 16 * D + 64 * (D / G) + 64 * grp + 4 * tau);
        ks = __low2float(k2), kz = __high2float(k2), vs = __low2float(v2), vz = __high2float(v2);
    }
    // dim 4 lane + j of the panel is nibble n = lane / 2 % 4 of the word (i = lane / 8, c = 4 (lane % 2) + j)
    const int base = (threadIdx.x & 31) - lane;
    float x[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = __shfl_sync(0xFFFFFFFFu, vw, base + (lane & ~7) + 4 * (lane & 1) + j);
        x[j] = (static_cast<float>((kq >> (4 * j)) & 15u) - kz) * ks;
        y[j] = (static_cast<float>((w >> (4 * ((lane >> 1) & 3))) & 15u) - vz) * vs;
    }
    if (!in) return;
    const int64_t o = (tok * p.heads + head) * D + panel * kPanel + 4 * lane;
    store4(static_cast<T*>(p.k_out) + o, x);
    store4(static_cast<T*>(p.v_out) + o, y);
}

template <typename T, bool kAppend>
cudaError_t launch_cache(const sgemv_kv_layout& L, const CacheParams& p, cudaStream_t s) {
    const int lanes = L.dim < 128 ? L.dim / 4 : 32;
    const int64_t blocks = (p.units * lanes + kCacheThreads - 1) / kCacheThreads;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks));
#define SGEMV_KV_CASE(D, G)                                                                                   \
    if (L.dim == D && L.group == G) {                                                                         \
        if constexpr (kAppend) return launch_pdl(append_kernel<T, D, G>, grid, dim3(kCacheThreads), 0, s, p); \
        else return launch_pdl(read_kernel<T, D, G>, grid, dim3(kCacheThreads), 0, s, p);                     \
    }
    SGEMV_KV_CASE(64, 64)
    SGEMV_KV_CASE(128, 64)
    SGEMV_KV_CASE(128, 128)
    SGEMV_KV_CASE(256, 64)
    SGEMV_KV_CASE(256, 128)
#undef SGEMV_KV_CASE
    return cudaErrorInvalidValue;
}

CacheParams params_of(const sgemv_kv_layout& L, const void* cache, const int64_t* slots, int n, int32_t* status) {
    CacheParams p = {};
    p.cache = const_cast<uint8_t*>(static_cast<const uint8_t*>(cache));
    p.slots = slots;
    p.status = status;
    p.sub_bytes = L.sub_bytes;
    p.head_bytes = L.head_bytes;
    p.page_bytes = L.page_bytes;
    p.n_slots = static_cast<int64_t>(L.n_pages) * L.page;
    p.heads = L.heads;
    p.page = L.page;
    p.n_tokens = n;
    p.units = static_cast<int64_t>(n) * L.heads * (L.dim > 128 ? L.dim / 128 : 1);
    return p;
}

}  // namespace

int check_kv_layout(const sgemv_kv_layout* layout) {
    if (layout == nullptr) return SGEMV_ERR_ARG;
    sgemv_kv_layout ref;
    const int rc = sgemv_kv_layout_query(layout->heads, layout->dim, layout->group, layout->page, layout->n_pages, &ref);
    if (rc != SGEMV_OK) return SGEMV_ERR_FORMAT;
    return ref.sub_bytes == layout->sub_bytes && ref.head_bytes == layout->head_bytes &&
                   ref.page_bytes == layout->page_bytes && ref.total_bytes == layout->total_bytes
               ? SGEMV_OK
               : SGEMV_ERR_FORMAT;
}

}  // namespace sgemv

using namespace sgemv;

extern "C" {

int sgemv_kv_layout_query(int heads, int dim, int group, int page, int n_pages, sgemv_kv_layout* out) {
    if (out == nullptr) return SGEMV_ERR_ARG;
    if (heads < 1 || heads > 1024 || n_pages < 1) return SGEMV_ERR_SHAPE;
    if (dim != 64 && dim != 128 && dim != 256) return SGEMV_ERR_SHAPE;
    if ((group != 64 && group != 128) || group > dim) return SGEMV_ERR_SHAPE;
    if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return SGEMV_ERR_SHAPE;
    sgemv_kv_layout L = {};
    L.heads = heads;
    L.dim = dim;
    L.group = group;
    L.page = page;
    L.n_pages = n_pages;
    L.sub_bytes = 16ull * dim + 128ull * (dim / group);
    L.head_bytes = L.sub_bytes * (page / kSub);
    L.page_bytes = L.head_bytes * heads;
    L.total_bytes = L.page_bytes * n_pages;
    *out = L;
    return SGEMV_OK;
}

int sgemv_kv_append(const sgemv_kv_layout* layout, void* cache_dev, int dtype, const void* k_dev,
                    int64_t k_token_stride, int64_t k_head_stride, const void* v_dev, int64_t v_token_stride,
                    int64_t v_head_stride, const int64_t* slots_dev, int n_tokens, int32_t* status_dev, void* stream) {
    const int rc = check_kv_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if ((dtype != SGEMV_F16 && dtype != SGEMV_BF16) || n_tokens < 0) return SGEMV_ERR_ARG;
    if (n_tokens == 0) return SGEMV_OK;
    if (cache_dev == nullptr || k_dev == nullptr || v_dev == nullptr || slots_dev == nullptr) return SGEMV_ERR_ARG;
    if (!is_aligned(cache_dev, 16) || !is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(slots_dev, 8) ||
        !is_aligned(status_dev, 4) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8)
        return SGEMV_ERR_ALIGN;
    CacheParams p = params_of(*layout, cache_dev, slots_dev, n_tokens, status_dev);
    p.k = k_dev;
    p.v = v_dev;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SGEMV_F16 ? launch_cache<__half, true>(*layout, p, s)
                                             : launch_cache<__nv_bfloat16, true>(*layout, p, s);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}

int sgemv_kv_read(const sgemv_kv_layout* layout, const void* cache_dev, const int64_t* slots_dev, int n_tokens,
                  int dtype, void* k_dev, void* v_dev, int32_t* status_dev, void* stream) {
    const int rc = check_kv_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if (dtype < SGEMV_F16 || dtype > SGEMV_F32 || n_tokens < 0) return SGEMV_ERR_ARG;
    if (n_tokens == 0) return SGEMV_OK;
    if (cache_dev == nullptr || k_dev == nullptr || v_dev == nullptr || slots_dev == nullptr) return SGEMV_ERR_ARG;
    if (!is_aligned(cache_dev, 16) || !is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(slots_dev, 8) ||
        !is_aligned(status_dev, 4))
        return SGEMV_ERR_ALIGN;
    CacheParams p = params_of(*layout, cache_dev, slots_dev, n_tokens, status_dev);
    p.k_out = k_dev;
    p.v_out = v_dev;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SGEMV_F16    ? launch_cache<__half, false>(*layout, p, s)
                          : dtype == SGEMV_BF16 ? launch_cache<__nv_bfloat16, false>(*layout, p, s)
                                                : launch_cache<float, false>(*layout, p, s);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}

}  // extern "C"
