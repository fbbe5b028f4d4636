// Shared by the kernels of 4-bit matrices: their layout, and conversions.
#pragma once

#include "kv_common.cuh"
#include "sgemv_prompt.h"

namespace sgemv {

// Host: the caller's layout is the one sgemv_fp4_layout_query computes.
int check_fp4_layout(const sgemv_fp4_layout* layout);

// A 4-bit matrix on the device.
struct Fp4Matrix {
    uint8_t* codes;
    uint8_t* scales;
    float* row_scale;
    int rows, k, tile, kp;
    int groups;  // of 4 scales a row
    Fp4Matrix() = default;
    Fp4Matrix(const sgemv_fp4_layout& l, const void* packed)
        : codes(static_cast<uint8_t*>(const_cast<void*>(packed))), scales(codes + l.scale_off),
          row_scale(reinterpret_cast<float*>(codes + l.row_off)), rows(l.rows), k(l.k), tile(l.tile), kp(l.kp),
          groups((l.kp + 4 * l.block - 1) / (4 * l.block)) {}
};

// Where the 16 bytes of 32 codes are, and the 4 scales of a group.
__device__ __forceinline__ uint8_t* codes_at(const Fp4Matrix& m, int row, int chunk) {
    const int64_t t = row / m.tile;
    return m.codes + ((t * (m.kp / 32) + chunk) * m.tile + row % m.tile) * 16;
}
__device__ __forceinline__ uint8_t* scales_at(const Fp4Matrix& m, int row, int group) {
    const int64_t t = row / 128;
    return m.scales + (t * m.groups + group) * 512 + (row % 32) * 16 + (row % 128) / 32 * 4;
}

// Two elements of 16 bits as binary32.
template <typename T>
__device__ __forceinline__ float2 two_f32(uint32_t w);
template <>
__device__ __forceinline__ float2 two_f32<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
template <>
__device__ __forceinline__ float2 two_f32<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_two(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_two<__half>(float lo, float hi) { return pack_half2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack_two<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// e4m3, to the nearest (ties to even, past 448: 448), and back, exactly.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
    return r & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(b)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}
// 2^(b - 127)
__device__ __forceinline__ float from_e8m0(uint32_t b) { return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23); }

// Eight e2m1 codes, the first in the lowest bits: to the nearest, ties to the even code, at most 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
// Eight codes as four fp16 pairs.
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

}  // namespace sgemv
