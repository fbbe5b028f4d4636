// Shared by the cache's kernels: element types, the byte layout of a subtile, small device helpers.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <climits>

#include "common.cuh"
#include "sgemv_kv.h"

namespace sgemv {

constexpr int kSub = 16;  // tokens of a subtile

// Host: the caller's layout is the one sgemv_kv_layout_query computes.
int check_kv_layout(const sgemv_kv_layout* layout);

inline bool is_aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Host: bytes that a call reads or writes.
struct Bytes {
    uintptr_t at;
    uint64_t size;  // 0: nothing
    Bytes(const void* p, uint64_t n) : at(reinterpret_cast<uintptr_t>(p)), size(p != nullptr ? n : 0) {}
};
inline bool meet(const Bytes& a, const Bytes& b) { return a.size != 0 && b.size != 0 && a.at < b.at + b.size && b.at < a.at + a.size; }
// Whether one of `rows` rows of row.size bytes, `stride` bytes apart (row.size at least), has some of b's.
inline bool rows_meet(const Bytes& row, uint64_t rows, uint64_t stride, const Bytes& b) {
    if (row.size == 0 || rows == 0 || !meet({reinterpret_cast<const void*>(row.at), (rows - 1) * stride + row.size}, b)) return false;
    const uint64_t i = b.at < row.at + row.size ? 0 : (b.at - row.at - row.size) / stride + 1;  // the first row that ends after b starts
    return i < rows && row.at + i * stride < b.at + b.size;
}
// Everything from the first to the last row of [tokens][heads][dim] elements of 2 bytes.
inline Bytes span_bytes(const void* p, int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t dim) {
    const int64_t t = (tokens - 1) * token_stride, h = (heads - 1) * head_stride;
    const int64_t lo = (t < 0 ? t : 0) + (h < 0 ? h : 0), hi = (t > 0 ? t : 0) + (h > 0 ? h : 0) + dim;
    Bytes b(p, 2 * (hi - lo));
    b.at += 2 * lo;
    return b;
}
// What a call writes meets neither what else it writes nor what it reads.
template <int W, int R>
bool apart(const Bytes (&written)[W], const Bytes (&read)[R]) {
    for (int i = 0; i < W; ++i) {
        for (int j = i + 1; j < W; ++j)
            if (meet(written[i], written[j])) return false;
        for (int j = 0; j < R; ++j)
            if (meet(written[i], read[j])) return false;
    }
    return true;
}

// Strides of [tokens][heads][dim] that keep rows 16-byte aligned; that of an axis of length 1 is never used.
inline bool strides_aligned(int tokens, int64_t token_stride, int heads, int64_t head_stride) {
    return (tokens < 2 || token_stride % 8 == 0) && (heads < 2 || head_stride % 8 == 0);
}

// Host: launch with programmatic dependent launch (the kernels call pdl_wait before their first read).
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, dim3 block, uint32_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

constexpr int kChunkRows = 256;  // rows of a CTA of the chunk kernel

// Host: requests with more rows (new tokens x query heads of a KV head) than this go to the chunk kernel; INT_MAX where none does.
// Its tensor memory holds dims up to 128. It takes the same time for 1 row as for the 256 of a CTA, the decode kernel a time in
// proportion: 16 requests of up to 4096 keys, 8 KV heads of 128, 77 rows on average: decode 64 us, chunk 91; 154: 109, 93; heads of
// 64, 154: 65, 78; 308: 112, 80. So the average decides, and half of a batch does not go either way (154 rows, divided at 128: 124
// us). Where there are fewer segments than SMs, so that the chunk kernel splits them over the keys and joins large partials, it
// wins later: one request of 4096 keys with 614 rows: 60, 70; with 1228: 103, 81.
inline int chunk_threshold(int dim, int heads, int ratio, int n_req, int n_tokens, int max_q, int sms) {
    const int64_t all_rows = static_cast<int64_t>(n_tokens) * ratio;
    const bool few = (all_rows / kChunkRows + n_req) * heads < sms;
    const bool dense = all_rows > static_cast<int64_t>(n_req) * (dim == 64 ? 224 : 112);
    const int rows = few ? 1024 : dense ? 64 : 512;
    return dim <= 128 && static_cast<int64_t>(max_q) * ratio > rows ? rows : INT_MAX;
}

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

// Two binary32 operations an instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 parts_of(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace sgemv
