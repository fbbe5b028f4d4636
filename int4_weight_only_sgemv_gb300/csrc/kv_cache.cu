// The paged 4-bit KV cache: its layout, writing K and V rows into it, and reading them back.
//
// Both kernels move bytes, each input and output once. Work unit: one panel of min(dim, 128) dims of one (token, head), by
// width / 8 lanes with 8 dims each: 16-byte loads and stores on the wide side, 4 bytes of K nibbles, and V's nibbles through a
// 4 x 4 byte transpose over 4 lanes (two shuffles), since a 16-bit word of V holds one nibble from each of them. With 4 dims a
// lane and a division an element, append and read of 20011 tokens (8 heads of 128, bf16, 210 MB in all) took 110 us; so they
// take 54.5, 57% of the measured HBM rate. Instructions bound them: 26 an element in append, 14 in read. Of append's, the quotient,
// exact to the last bit, is four and rounding and clamping two; the others are a unit's place (a division, the slot, the address),
// the group's minimum and maximum with their shuffles, and V's transpose and 2-byte stores, over the 8 elements of a lane.
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
    uint32_t units;
    int heads, log2_page, n_tokens;
};

template <typename T>
struct Two;
template <>
struct Two<__half> { using type = __half2; };
template <>
struct Two<__nv_bfloat16> { using type = __nv_bfloat162; };

// Quantises the 8 values of this lane with the group of kLanes neighbouring lanes: nibbles (first dim lowest), scale and zero
// point, in binary32 without fused multiply-adds but for the quotients. A quotient v / s is formed from the reciprocal r of s as
// t = v r, t + r (v - t s), the remainder exact in one fused multiply-add (Markstein's correction). The rounded integer is that
// of the correctly rounded quotient: v and s have 11 bits at most, so a quotient that is not half way between two integers
// is at least 2^-13 of its size away from there, and one that is half way comes out exactly.
template <typename T, int kLanes>
__device__ __forceinline__ uint32_t quantise(const uint4& raw, __half& s16, float& z, bool& bad) {
    using T2 = typename Two<T>::type;
    const T2* h = reinterpret_cast<const T2*>(&raw);
    // the largest value and the largest negated value, exactly, NaN if one is
    T2 hi = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    T2 lo = __hmax2_nan(__hmax2_nan(__hneg2(h[0]), __hneg2(h[1])), __hmax2_nan(__hneg2(h[2]), __hneg2(h[3])));
    T2 m = __hmax2_nan(T2(hi.x, lo.x), T2(hi.y, lo.y));
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, *reinterpret_cast<const uint32_t*>(&m), d);
        m = __hmax2_nan(m, *reinterpret_cast<const T2*>(&o));
    }
    const float mx = to_f32(m.x), mn = -to_f32(m.y);
    bad = !(mx < INFINITY) || !(mn > -INFINITY);
    const float top = fmaxf(mx, 0.0f), bottom = fminf(mn, 0.0f);
    s16 = __float2half_rn(__fdiv_rn(__fsub_rn(top, bottom), 15.0f));
    bad = bad || __hisinf(s16);
    if (bad || __half2float(s16) == 0.0f) s16 = __float2half_rn(1.0f);
    z = 0.0f;
    if (bad) return 0;
    const float s = __half2float(s16), r = __frcp_rn(s);
    // the quotient rounded to an integer, as the low bits of kMagic plus it (ties to even, as the addition rounds)
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
    const auto rounded = [&](float v) {
        const float t = __fmul_rn(v, r);
        return __fadd_rn(fmaf(r, fmaf(-t, s, v), t), kMagic);
    };
    z = fminf(fmaxf(rounded(-bottom) - kMagic, 0.0f), 15.0f) + 0.0f;  // + 0: never -0
    const int zero = __float_as_int(z + kMagic) - 2 * __float_as_int(kMagic);
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float v = to_f32(reinterpret_cast<const T*>(&raw)[j]);
        q += static_cast<uint32_t>(__viaddmin_s32_relu(__float_as_int(rounded(v)), zero, 15)) * (1u << (4 * j));
    }
    return q;
}

// Lane n of 4 neighbouring ones holds the bytes b[n][0..3]; afterwards b[0..3][n].
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t w, int lane) {
    uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
    w = (lane & 1) ? __byte_perm(w, o, 0x3715) : __byte_perm(w, o, 0x6240);
    o = __shfl_xor_sync(0xFFFFFFFFu, w, 2);
    return (lane & 2) ? __byte_perm(w, o, 0x3276) : __byte_perm(w, o, 0x5410);
}
// The low nibbles of 4 bytes as a 16-bit word, and back.
__device__ __forceinline__ uint32_t pack_nibbles(uint32_t x) {
    x &= 0x0F0F0F0Fu;
    x = (x | (x >> 4)) & 0x00FF00FFu;
    return (x | (x >> 8)) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t x) {
    x = (x | (x << 8)) & 0x00FF00FFu;
    return (x | (x << 4)) & 0x0F0F0F0Fu;
}

// Byte offset in a subtile of the 16-bit word of V with dims c + 8n + 32i (n = 0..3) of token tau.
template <int D>
__device__ __forceinline__ uint32_t v_word(int tau, int c, int i) {
    const int w = ((tau >> 1) & 1) * (D / 32) + i;
    return 8 * D + (w >> 2) * 512 + (4 * c + (tau >> 2)) * 16 + (w & 3) * 4 + (tau & 1) * 2;
}

// Where a unit's lane works.
template <int D>
struct Place {
    static constexpr int kPanel = D < 128 ? D : 128, kPanels = D / kPanel, kLanes = kPanel / 8;
    uint32_t tok;
    int lane, panel, head, tau;
    int64_t slot;   // -1: nothing there
    bool in;        // a unit of the call (a warp's last ones may not be: they still take part in the shuffles)
    uint8_t* sub;
    __device__ __forceinline__ explicit Place(const CacheParams& p) {
        const uint32_t unit = blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
        lane = threadIdx.x % kLanes;
        in = unit < p.units;
        panel = unit % kPanels;
        tok = unit / kPanels / static_cast<uint32_t>(p.heads);
        head = static_cast<int>(unit / kPanels - tok * static_cast<uint32_t>(p.heads));
        slot = in ? p.slots[tok] : -1;
        if (slot >= p.n_slots) {
            report(p.status, SGEMV_ERR_ARG);
            slot = -1;
        }
        if (slot < 0) slot = -1;
        const int at = static_cast<int>(slot) & ((1 << p.log2_page) - 1);
        tau = at % kSub;
        sub = p.cache + static_cast<uint64_t>(slot >> p.log2_page) * p.page_bytes + head * p.head_bytes + (at / kSub) * p.sub_bytes;
    }
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(kCacheThreads) append_kernel(const CacheParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const Place<D> at(p);
    constexpr int kPanel = Place<D>::kPanel;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (at.slot >= 0) {
        const int d = at.panel * kPanel + 8 * at.lane;
        x = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + at.tok * p.k_token + at.head * p.k_head + d);
        y = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + at.tok * p.v_token + at.head * p.v_head + d);
    }
    __half ks, vs;
    float kz, vz;
    bool kbad, vbad;
    const uint32_t kq = quantise<T, G / 8>(x, ks, kz, kbad);
    // lane l holds dims 8l .. of block l / 4, n = l % 4: byte c / 2 of its nibbles is dims c, c + 1
    const uint32_t vb = transpose_bytes(quantise<T, G / 8>(y, vs, vz, vbad), at.lane);
    if (at.slot < 0) return;
    if (kbad || vbad) report(p.status, SGEMV_ERR_NONFINITE);
    *reinterpret_cast<uint32_t*>(at.sub + at.panel * 8 * kPanel + at.tau * (kPanel / 2) + 4 * at.lane) = kq;
    const int c = 2 * (at.lane & 3), i = (at.lane >> 2) + 4 * at.panel;
    *reinterpret_cast<uint16_t*>(at.sub + v_word<D>(at.tau, c, i)) = static_cast<uint16_t>(pack_nibbles(vb));
    *reinterpret_cast<uint16_t*>(at.sub + v_word<D>(at.tau, c + 1, i)) = static_cast<uint16_t>(pack_nibbles(vb >> 4));
    if (at.lane % (G / 8) == 0) {
        const int grp = at.panel * (kPanel / G) + at.lane / (G / 8);
        const __half2 k2 = __halves2half2(ks, __float2half_rn(kz)), v2 = __halves2half2(vs, __float2half_rn(vz));
        *reinterpret_cast<__half2*>(at.sub + 16 * D + 64 * grp + 4 * at.tau) = k2;
        *reinterpret_cast<__half2*>(at.sub + 16 * D + 64 * (D / G) + 64 * grp + 4 * at.tau) = v2;
    }
}

// The 8 values of nibbles q, each rounded once. q - z comes out of the fp16 numbers 1024 + q and 1024 + 16 q exactly, dims j and
// j + 4 at a time.
template <typename T>
__device__ __forceinline__ void store8(T* p, uint32_t q, __half2 sz) {
    const __half2 z = __high2half2(sz), s = __low2half2(sz);
    const __half2 z0 = __hsub2(__floats2half2_rn(-1024.0f, -1024.0f), z), z1 = __hsub2(__floats2half2_rn(-64.0f, -64.0f), z);
    const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
    __half2 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = (((j & 2) ? q >> 8 : q) & ((j & 1) ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
        const __half2 n = *reinterpret_cast<const __half2*>(&w);
        h[j] = (j & 1) ? __hfma2(n, sixteenth, z1) : __hadd2(n, z0);
    }
    if constexpr (std::is_same<T, __half>::value) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 f = __hmul2(h[j], s);
            w[j] = *reinterpret_cast<const uint32_t*>(&f);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                                                  __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
    } else {
        const float sf = __low2float(sz);
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = __half22float2(h[j]);
            f[j] = t.x * sf, f[j + 4] = t.y * sf;
        }
        if constexpr (sizeof(T) == 2) {
            T o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = from_f32<T>(f[j]);
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const CacheParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const Place<D> at(p);
    constexpr int kPanel = Place<D>::kPanel;
    uint32_t kq = 0, vb = 0;
    __half2 kf = __floats2half2_rn(0.0f, 0.0f), vf = kf;  // scale, zero point
    if (at.slot >= 0) {
        kq = *reinterpret_cast<const uint32_t*>(at.sub + at.panel * 8 * kPanel + at.tau * (kPanel / 2) + 4 * at.lane);
        const int c = 2 * (at.lane & 3), i = (at.lane >> 2) + 4 * at.panel;
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(at.sub + v_word<D>(at.tau, c, i));
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(at.sub + v_word<D>(at.tau, c + 1, i));
        const int grp = at.panel * (kPanel / G) + at.lane / (G / 8);
        kf = *reinterpret_cast<const __half2*>(at.sub + 16 * D + 64 * grp + 4 * at.tau);
        vf = *reinterpret_cast<const __half2*>(at.sub + 16 * D + 64 * (D / G) + 64 * grp + 4 * at.tau);
        vb = spread_nibbles(lo) | (spread_nibbles(hi) << 4);
    }
    const uint32_t vq = transpose_bytes(vb, at.lane);
    if (!at.in) return;
    const int64_t o = (static_cast<int64_t>(at.tok) * p.heads + at.head) * D + at.panel * kPanel + 8 * at.lane;
    store8(static_cast<T*>(p.k_out) + o, kq, kf);
    store8(static_cast<T*>(p.v_out) + o, vq, vf);
}

template <typename T, bool kAppend>
cudaError_t launch_cache(const sgemv_kv_layout& L, const CacheParams& p, cudaStream_t s) {
    const unsigned units = kCacheThreads / (L.dim < 128 ? L.dim / 8 : 16);  // of a CTA
    const dim3 grid((p.units + units - 1) / units);
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

// Units of a call fit 31 bits (a unit's K and V take 256 bytes at least: no GPU holds so many).
bool too_many(const sgemv_kv_layout& L, int n) { return static_cast<int64_t>(n) * L.heads * (L.dim > 128 ? 2 : 1) > INT_MAX; }

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
    while ((1 << p.log2_page) < L.page) ++p.log2_page;
    p.n_tokens = n;
    p.units = static_cast<uint32_t>(n) * L.heads * (L.dim > 128 ? L.dim / 128 : 1);
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
    if (too_many(*layout, n_tokens)) return SGEMV_ERR_SHAPE;
    if (cache_dev == nullptr || k_dev == nullptr || v_dev == nullptr || slots_dev == nullptr) return SGEMV_ERR_ARG;
    if (!is_aligned(cache_dev, 16) || !is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(slots_dev, 8) ||
        !is_aligned(status_dev, 4) || !strides_aligned(n_tokens, k_token_stride, layout->heads, k_head_stride) ||
        !strides_aligned(n_tokens, v_token_stride, layout->heads, v_head_stride))
        return SGEMV_ERR_ALIGN;
    const Bytes written[] = {{cache_dev, layout->total_bytes}, {status_dev, 4}};
    const Bytes read[] = {span_bytes(k_dev, n_tokens, k_token_stride, layout->heads, k_head_stride, layout->dim),
                          span_bytes(v_dev, n_tokens, v_token_stride, layout->heads, v_head_stride, layout->dim),
                          {slots_dev, 8ull * n_tokens}};
    if (!apart(written, read)) return SGEMV_ERR_ARG;
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
    if (too_many(*layout, n_tokens)) return SGEMV_ERR_SHAPE;
    if (cache_dev == nullptr || k_dev == nullptr || v_dev == nullptr || slots_dev == nullptr) return SGEMV_ERR_ARG;
    if (!is_aligned(cache_dev, 16) || !is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(slots_dev, 8) ||
        !is_aligned(status_dev, 4))
        return SGEMV_ERR_ALIGN;
    const uint64_t out_bytes = (dtype == SGEMV_F32 ? 4ull : 2ull) * n_tokens * layout->heads * layout->dim;
    const Bytes written[] = {{k_dev, out_bytes}, {v_dev, out_bytes}, {status_dev, 4}};
    const Bytes read[] = {{cache_dev, layout->total_bytes}, {slots_dev, 8ull * n_tokens}};
    if (!apart(written, read)) return SGEMV_ERR_ARG;
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
