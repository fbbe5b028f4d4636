// Matrices in block-scaled 4-bit floating point: layout, quantisation, reading back.
//
// A lane has 32 consecutive values of a row at a time: their codes are 16 contiguous bytes of the matrix, and a scale needs no other lane.
// The 8 rows of a CTA are the pairs (2p, 2p + 1) of each 32 of a tile's 128, so that the two halves of a 32-byte sector of codes, and the
// eight words of a sector of scales, are written by one CTA at about the same time.
//
// The quotients. x has 11 significant bits, a scale 4, a midpoint between two codes 3: a quotient x / scale is a midpoint or at least 2^-11
// of one away, so that a binary32 quotient which is exact where it has few bits rounds as the true one does. It is formed by a
// reciprocal and one correction (the remainder is exact), without a division for each element. The same holds for m / 6 and e4m3.
#include "fp4_common.cuh"

namespace sgemv {

namespace {

constexpr int kWarpsQ = 8;

struct QuantParams {
    Fp4Matrix m;
    const void* x;   // or the output of read
    int64_t stride;
    int32_t* status;
    int wpr;         // warps a row
    int vec;         // rows in 16-byte pieces
};

// The row of a CTA's slot.
__device__ __forceinline__ int row_of_slot(const Fp4Matrix& m, int64_t slot) {
    if (m.tile < 128) return static_cast<int>(slot);
    const int s = static_cast<int>(slot & 127);
    return static_cast<int>(slot - s) + 32 * ((s >> 1) & 3) + 2 * (s >> 3) + (s & 1);
}

// 32 values of a row from column 32 c, zeros past its end.
template <typename T>
__device__ __forceinline__ void load32(const T* row, int c, int k, bool vec, uint32_t (&w)[16]) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (32 * c + 8 * i < k) v = *reinterpret_cast<const uint4*>(row + 32 * c + 8 * i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at = 32 * c + 2 * i;
            const uint32_t lo = at < k ? h[at] : 0, hi = at + 1 < k ? h[at + 1] : 0;
            w[i] = lo | (hi << 16);
        }
    }
}
// The largest magnitude of 8 words' elements, as 16 bits (infinities and NaN above all numbers).
__device__ __forceinline__ uint32_t most16(const uint32_t* w) {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
}
template <typename T>
__device__ __forceinline__ float as_f32(uint32_t bits) {
    return two_f32<T>(bits).x;
}
template <typename T>
constexpr uint32_t kInfBits = 0x7C00u;
template <>
constexpr uint32_t kInfBits<__nv_bfloat16> = 0x7F80u;

template <typename T, int kBlock>
__global__ void __launch_bounds__(32 * kWarpsQ) quantize_kernel(const QuantParams p) {
    __shared__ uint32_t s_most[kWarpsQ];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = warp / p.wpr, part = warp % p.wpr;
    if (threadIdx.x < kWarpsQ) s_most[threadIdx.x] = 0;
    pdl_launch_dependents();
    const int row = row_of_slot(p.m, static_cast<int64_t>(blockIdx.x) * (kWarpsQ / p.wpr) + slot);
    const bool live = row < p.m.rows;
    const T* const x = static_cast<const T*>(p.x) + (live ? row : 0) * p.stride;
    const int chunks = live ? p.m.kp / 32 : 0, step = 32 * p.wpr;
    const bool vec = p.vec != 0;
    __syncthreads();
    pdl_wait();
    float unit = 1.0f, down = 1.0f;
    bool bad = false;
    if constexpr (kBlock == 16) {
        // the row's largest magnitude, and from it the row's power of two
        uint32_t most = 0;
        for (int c = 32 * part + lane; c < chunks; c += step) {
            uint32_t w[16];
            load32(x, c, p.m.k, vec, w);
            most = max(most, max(most16(w), most16(w + 8)));
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (p.wpr > 1) {
            if (lane == 0) atomicMax(&s_most[slot], most);
            __syncthreads();
            most = s_most[slot];
        }
        bad = most >= kInfBits<T>;
        const uint32_t b = __float_as_uint(as_f32<T>(most));  // 2688 = 1.3125 * 2^11
        const int e = bad || b == 0 ? 0 : max(-100, static_cast<int>(b >> 23) - 138 + ((b & 0x7FFFFFu) > 0x280000u));
        unit = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }
    uint32_t seen = 0;
    for (int base = 32 * part; base < chunks; base += step) {
        const int c = base + lane;
        uint32_t w[16];
        uint32_t scale = 0;
        uint4 codes;
        if (c < chunks) {
            load32(x, c, p.m.k, vec, w);
            const uint32_t m0 = most16(w), m1 = most16(w + 8);
            float s[2], inv[2];
            if constexpr (kBlock == 32) {
                const uint32_t m = max(m0, m1);
                seen = max(seen, m);
                scale = max(0, static_cast<int>(__float_as_uint(as_f32<T>(m)) >> 23) - 2);
                inv[0] = inv[1] = __uint_as_float((254u - scale) << 23);
                s[0] = s[1] = 0.0f;
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float m = as_f32<T>(h ? m1 : m0) * down;
                    const uint32_t b = to_e4m3(__fdiv_rn(m, 6.0f));
                    scale |= b << (8 * h);
                    s[h] = from_e4m3(b) * unit;
                    inv[h] = s[h] > 0.0f ? __frcp_rn(s[h]) : 0.0f;
                }
            }
            uint32_t* const out = &codes.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t[8];
                const uint64_t r = pair(inv[i / 2], inv[i / 2]), d = pair(-s[i / 2], -s[i / 2]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = two_f32<T>(w[4 * i + j]);
                    const uint64_t v = pair(f.x, f.y);
                    uint64_t q = mul2(v, r);
                    if constexpr (kBlock == 16) q = fma2(fma2(q, d, v), r, q);
                    const float2 g = parts_of(q);
                    t[2 * j] = g.x, t[2 * j + 1] = g.y;
                }
                out[i] = to_e2m1x8(t);
            }
            *reinterpret_cast<uint4*>(codes_at(p.m, row, c)) = codes;
        }
        if constexpr (kBlock == 16) {
            scale |= __shfl_down_sync(0xFFFFFFFFu, scale, 1) << 16;
            if ((lane & 1) == 0 && c < chunks) *reinterpret_cast<uint32_t*>(scales_at(p.m, row, c / 2)) = scale;
        } else {
            scale |= __shfl_down_sync(0xFFFFFFFFu, scale, 1) << 8;
            scale |= __shfl_down_sync(0xFFFFFFFFu, scale, 2) << 16;
            if ((lane & 3) == 0 && c < chunks) *reinterpret_cast<uint32_t*>(scales_at(p.m, row, c / 4)) = scale;
        }
    }
    if constexpr (kBlock == 32) {
        seen = __reduce_max_sync(0xFFFFFFFFu, seen);
        if (p.wpr > 1) {
            if (lane == 0) atomicMax(&s_most[slot], seen);
            __syncthreads();
            seen = s_most[slot];
        }
        bad = seen >= kInfBits<T>;
    }
    if (live && part == 0 && lane == 0) {
        p.m.row_scale[row] = bad ? __int_as_float(0x7FC00000) : unit;
        if (bad) report(p.status, SGEMV_ERR_NONFINITE);
    }
}

template <typename T, int kBlock>
__global__ void __launch_bounds__(32 * kWarpsQ) read_kernel(const QuantParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot = warp / p.wpr, part = warp % p.wpr;
    pdl_launch_dependents();
    const int row = row_of_slot(p.m, static_cast<int64_t>(blockIdx.x) * (kWarpsQ / p.wpr) + slot);
    pdl_wait();
    if (row >= p.m.rows) return;
    T* const out = const_cast<T*>(static_cast<const T*>(p.x)) + row * p.stride;
    const float unit = p.m.row_scale[row];
    for (int c = 32 * part + lane; 32 * c < p.m.k; c += 32 * p.wpr) {
        const uint4 codes = *reinterpret_cast<const uint4*>(codes_at(p.m, row, c));
        const uint8_t* const sc = scales_at(p.m, row, c * 32 / kBlock / 4) + c * 32 / kBlock % 4;
        float s[2];
        if constexpr (kBlock == 16) s[0] = from_e4m3(sc[0]) * unit, s[1] = from_e4m3(sc[1]) * unit;
        else s[0] = s[1] = from_e8m0(sc[0]) * unit;
        const uint32_t in[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            from_e2m1x8(in[i], h);
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = two_f32<__half>(h[j]);
                f[2 * j] = v.x * s[i / 2], f[2 * j + 1] = v.y * s[i / 2];
            }
            const int col = 32 * c + 8 * i;
            if (p.vec && col < p.m.k) {
                if constexpr (sizeof(T) == 4) {
                    *reinterpret_cast<float4*>(out + col) = make_float4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<float4*>(out + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                    *reinterpret_cast<uint4*>(out + col) = make_uint4(pack_two<T>(f[0], f[1]), pack_two<T>(f[2], f[3]),
                                                                      pack_two<T>(f[4], f[5]), pack_two<T>(f[6], f[7]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < p.m.k) out[col + j] = from_f32<T>(f[j]);
            }
        }
    }
}

// Warps a row: one, where there are rows enough for 8 warps an SM; else more, as far as each has 1024 columns.
int warps_a_row(int rows, int k, int sms) {
    int w = 1;
    while (w < kWarpsQ && static_cast<int64_t>(rows) * w < 8ll * sms && k > 1024 * w) w *= 2;
    return w;
}

int launch_rows(const sgemv_fp4_layout& l, QuantParams& p, void (*kern)(const QuantParams), void* stream) {
    DeviceInfo di;
    const int rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    p.wpr = warps_a_row(l.rows, l.k, di.sm_count);
    const int64_t slots = (static_cast<int64_t>(l.rows) + l.tile - 1) / l.tile * l.tile;
    const int64_t used = l.tile < 128 ? l.rows : slots;
    const int64_t per = kWarpsQ / p.wpr;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>((used + per - 1) / per)), dim3(32 * kWarpsQ), 0,
                                     static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}

}  // namespace

int check_fp4_layout(const sgemv_fp4_layout* layout) {
    if (layout == nullptr) return SGEMV_ERR_ARG;
    sgemv_fp4_layout ref;
    if (sgemv_fp4_layout_query(layout->rows, layout->k, layout->block, &ref) != SGEMV_OK) return SGEMV_ERR_FORMAT;
    return ref.tile == layout->tile && ref.kp == layout->kp && ref.scale_off == layout->scale_off && ref.row_off == layout->row_off &&
                   ref.total_bytes == layout->total_bytes
               ? SGEMV_OK
               : SGEMV_ERR_FORMAT;
}

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_fp4_layout_query(int rows, int k, int block, sgemv_fp4_layout* out) {
    if (out == nullptr) return SGEMV_ERR_ARG;
    if (rows < 1 || rows > (1 << 24) || k < 1 || k > (1 << 20) || (block != 16 && block != 32)) return SGEMV_ERR_SHAPE;
    sgemv_fp4_layout l = {};
    l.rows = rows, l.k = k, l.block = block;
    l.tile = 8;
    while (l.tile < rows && l.tile < 128) l.tile *= 2;
    l.kp = (k + 63) / 64 * 64;
    const uint64_t tiles = (static_cast<uint64_t>(rows) + l.tile - 1) / l.tile, big = (static_cast<uint64_t>(rows) + 127) / 128;
    l.scale_off = tiles * l.tile * (l.kp / 2);
    l.row_off = l.scale_off + big * ((l.kp + 4 * block - 1) / (4 * block)) * 512;
    l.total_bytes = l.row_off + big * 512;
    *out = l;
    return SGEMV_OK;
}

extern "C" int sgemv_fp4_quantize(const sgemv_fp4_layout* layout, const void* x_dev, int dtype, int64_t stride, void* packed_dev,
                                  int32_t* status_dev, void* stream) {
    const int rc = check_fp4_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if ((dtype != SGEMV_F16 && dtype != SGEMV_BF16) || x_dev == nullptr || packed_dev == nullptr) return SGEMV_ERR_ARG;
    if (layout->rows > 1 && (stride < layout->k || stride > (1ll << 40))) return SGEMV_ERR_ARG;
    if (!is_aligned(packed_dev, 16) || !is_aligned(x_dev, 2) || !is_aligned(status_dev, 4)) return SGEMV_ERR_ALIGN;
    const int64_t st = layout->rows > 1 ? stride : layout->k;
    const Bytes x(x_dev, 2 * ((layout->rows - 1) * st + layout->k));
    const Bytes written[] = {{packed_dev, layout->total_bytes}, {status_dev, 4}};
    if (!apart(written, {x})) return SGEMV_ERR_ARG;
    QuantParams p;
    p.m = Fp4Matrix(*layout, packed_dev);
    p.x = x_dev, p.stride = st, p.status = status_dev;
    p.vec = is_aligned(x_dev, 16) && layout->k % 8 == 0 && (layout->rows < 2 || st % 8 == 0);
    const bool half = dtype == SGEMV_F16;
    return launch_rows(*layout, p,
                       layout->block == 16 ? (half ? quantize_kernel<__half, 16> : quantize_kernel<__nv_bfloat16, 16>)
                                           : (half ? quantize_kernel<__half, 32> : quantize_kernel<__nv_bfloat16, 32>),
                       stream);
}

extern "C" int sgemv_fp4_read(const sgemv_fp4_layout* layout, const void* packed_dev, void* out_dev, int dtype, int64_t stride,
                              void* stream) {
    const int rc = check_fp4_layout(layout);
    if (rc != SGEMV_OK) return rc;
    if (dtype < SGEMV_F16 || dtype > SGEMV_F32 || out_dev == nullptr || packed_dev == nullptr) return SGEMV_ERR_ARG;
    if (layout->rows > 1 && (stride < layout->k || stride > (1ll << 40))) return SGEMV_ERR_ARG;
    const unsigned size = dtype == SGEMV_F32 ? 4 : 2;
    if (!is_aligned(packed_dev, 16) || !is_aligned(out_dev, size)) return SGEMV_ERR_ALIGN;
    const int64_t st = layout->rows > 1 ? stride : layout->k;
    if (rows_meet({out_dev, size * static_cast<uint64_t>(layout->k)}, layout->rows, size * st, {packed_dev, layout->total_bytes}))
        return SGEMV_ERR_ARG;
    QuantParams p;
    p.m = Fp4Matrix(*layout, packed_dev);
    p.x = out_dev, p.stride = st, p.status = nullptr;
    p.vec = is_aligned(out_dev, 16) && layout->k % 8 == 0 && (layout->rows < 2 || st % 8 == 0);
    const bool b16 = layout->block == 16;
    return launch_rows(*layout, p,
                       dtype == SGEMV_F16    ? (b16 ? read_kernel<__half, 16> : read_kernel<__half, 32>)
                       : dtype == SGEMV_BF16 ? (b16 ? read_kernel<__nv_bfloat16, 16> : read_kernel<__nv_bfloat16, 32>)
                                             : (b16 ? read_kernel<float, 16> : read_kernel<float, 32>),
                       stream);
}
