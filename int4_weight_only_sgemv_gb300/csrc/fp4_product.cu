// The product of two 4-bit matrices: the entry point (argument checks, choice of the kernel).
#include <algorithm>
#include <climits>

#include "fp4_few.cuh"
#include "fp4_many.cuh"
#include "tensor_map.cuh"

namespace sgemv {

namespace {

// Whether a call goes to the kernel of many tiles: with more than 64 tokens, but where few tiles meet a long sum, which the other splits. us a call,
// many and few: 65 x 4096 x 4096 7.4, 10.6; 129 x 1024 x 4096 7.0, 8.2; 129 x 1024 x 6144 9.0, 9.3; 129 x 1024 x 8192 10.7, 10.3; 512 x 512 x 8192 11.0,
// 10.5; 100 x 200 x 16384 17.8, 9.8; 256 x 300 x 16384 18.7, 10.6.
bool many_tiles(const sgemv_fp4_layout& w, const sgemv_fp4_layout& x) {
    const int64_t tiles = static_cast<int64_t>((x.rows + 255) / 256) * ((w.rows + 255) / 256);
    return x.rows > 64 && w.rows > 64 && (tiles >= 8 || w.kp <= 6144);
}

// Whether its tiles are 256 weight rows wide, or 128, of which there are twice as many. us a call, 256 and 128: 512 x 4096 x 4096 (32 tiles of 256) 10.0, 8.5;
// 333 x 4096 x 11008 (32) 17.6, 14.6; 100 x 11008 x 4096 (43) 10.6, 13.3; 1024 x 4096 x 4096 (64) 10.7, 13.5.
bool wide_tiles(const sgemv_fp4_layout& w, const sgemv_fp4_layout& x, int sms) {
    const int64_t tiles = static_cast<int64_t>((x.rows + 255) / 256) * ((w.rows + 255) / 256);
    return tiles > sms / 4;
}

template <typename T, int kBlock, int kStageK>
cudaError_t launch_few_stage(const ProductParams& p, int64_t tiles, int smem, cudaStream_t s) {
    auto kern = fp4_few_kernel<T, kBlock, kStageK>;
    static std::atomic<int> attr_set[64];  // per device: dynamic shared memory already enabled
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (attr_set[dev].load() == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMost);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = static_cast<unsigned>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}
template <typename T, int kBlock>
cudaError_t launch_few(const ProductParams& p, int64_t tiles, int smem, cudaStream_t s) {
    return few_stage_k(p.x.tile) == 512 ? launch_few_stage<T, kBlock, 512>(p, tiles, smem, s) : launch_few_stage<T, kBlock, 256>(p, tiles, smem, s);
}

// `rows` rows of a tile's codes (128 or 64) and the scales of `tiles` tiles at a time.
bool map_fp4(Fp4Maps* maps, const Fp4Matrix& m, unsigned chunks_a_box, unsigned groups_a_box, unsigned rows, unsigned scale_tiles) {
    const cuuint64_t tiles = static_cast<cuuint64_t>((m.rows + 127) / 128), chunks = static_cast<cuuint64_t>(m.kp / 32), groups = static_cast<cuuint64_t>(m.groups);
    return encode_map(&maps->codes, CU_TENSOR_MAP_DATA_TYPE_UINT64, m.codes, {256, chunks, tiles}, {2048, chunks * 2048}, {2 * rows, chunks_a_box, 1},
                      CU_TENSOR_MAP_SWIZZLE_NONE) &&
           encode_map(&maps->scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, m.scales, {64, groups, tiles}, {512, groups * 512}, {64, groups_a_box, scale_tiles},
                      CU_TENSOR_MAP_SWIZZLE_NONE);
}
template <typename T, int kBlock, int kN>
cudaError_t launch_many_wide(ProductParams p, int sms, cudaStream_t s) {
    using S = ManyShape<kBlock, kN>;
    auto kern = fp4_many_kernel<T, kBlock, kN>;
    static std::atomic<int> attr_set[64];  // per device: dynamic shared memory already enabled
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (attr_set[dev].load() == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(1);
    }
    Fp4Maps x_maps, w_maps;
    if (!map_fp4(&x_maps, p.x, S::kChunks, S::kGroups, 128, 1) || !map_fp4(&w_maps, p.w, S::kChunks, S::kGroups, kN / 2, kN / 128)) return cudaErrorInvalidValue;
    p.tiles_x = (p.x.rows + 255) / 256, p.tiles_w = (p.w.rows + kN - 1) / kN;
    p.k_stages = (p.w.kp + S::kStageK - 1) / S::kStageK;
    const int pairs = std::min(p.tiles_x * p.tiles_w, sms / 2);
    return launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(S::kThreads), S::kSmem, s, x_maps, w_maps, p);
}
template <typename T, int kBlock>
cudaError_t launch_many(const ProductParams& p, bool wide, int sms, cudaStream_t s) {
    return wide ? launch_many_wide<T, kBlock, 256>(p, sms, s) : launch_many_wide<T, kBlock, 128>(p, sms, s);
}

}  // namespace

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_fp4_product(const sgemv_fp4_layout* w_layout, const void* w_dev, const sgemv_fp4_layout* x_layout,
                                 const void* x_dev, void* y_dev, int dtype, int64_t stride, int32_t* status_dev, void* stream) {
    int rc = check_fp4_layout(w_layout);
    if (rc == SGEMV_OK) rc = check_fp4_layout(x_layout);
    if (rc != SGEMV_OK) return rc;
    const sgemv_fp4_layout &w = *w_layout, &x = *x_layout;
    if (w.k != x.k || w.block != x.block) return SGEMV_ERR_FORMAT;
    if (dtype != SGEMV_F16 && dtype != SGEMV_BF16) return SGEMV_ERR_ARG;
    if (w.rows == 0 || x.rows == 0) return SGEMV_OK;
    if (w_dev == nullptr || x_dev == nullptr || y_dev == nullptr) return SGEMV_ERR_ARG;
    if (x.rows > 1 && (stride < w.rows || stride > (1ll << 40))) return SGEMV_ERR_ARG;
    if (!is_aligned(w_dev, 16) || !is_aligned(x_dev, 16) || !is_aligned(y_dev, 2) || !is_aligned(status_dev, 4)) return SGEMV_ERR_ALIGN;
    const int64_t st = x.rows > 1 ? stride : w.rows;
    const Bytes row(y_dev, 2ull * w.rows), status(status_dev, 4);
    for (const Bytes& b : {Bytes(w_dev, w.total_bytes), Bytes(x_dev, x.total_bytes), status})
        if (rows_meet(row, x.rows, 2 * st, b)) return SGEMV_ERR_ARG;
    if (meet(status, {w_dev, w.total_bytes}) || meet(status, {x_dev, x.total_bytes})) return SGEMV_ERR_ARG;
    DeviceInfo di;
    rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    ProductParams p;
    p.w = Fp4Matrix(w, w_dev), p.x = Fp4Matrix(x, x_dev);
    p.y = y_dev, p.stride = st, p.status = status_dev;
    p.k_stages = (w.kp + few_stage_k(x.tile) - 1) / few_stage_k(x.tile);
    p.x_tiles = (x.rows + 127) / 128;
    const int64_t tiles = static_cast<int64_t>((w.rows + 127) / 128) * p.x_tiles;
    if (tiles * 8 > INT_MAX) return SGEMV_ERR_SHAPE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool half = dtype == SGEMV_F16;
    if (many_tiles(w, x)) {
        const int sms = di.sm_count;
        const bool wide = wide_tiles(w, x, sms);
        const cudaError_t e = w.block == 16 ? (half ? launch_many<__half, 16>(p, wide, sms, s) : launch_many<__nv_bfloat16, 16>(p, wide, sms, s))
                                            : (half ? launch_many<__half, 32>(p, wide, sms, s) : launch_many<__nv_bfloat16, 32>(p, wide, sms, s));
        return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
    }
    const FewPlan plan = few_plan(w.block, x.tile, tiles, p.k_stages, di.sm_count);
    p.split = plan.split, p.ring = plan.ring;
    const cudaError_t e = w.block == 16 ? (half ? launch_few<__half, 16>(p, tiles, plan.smem, s) : launch_few<__nv_bfloat16, 16>(p, tiles, plan.smem, s))
                                        : (half ? launch_few<__half, 32>(p, tiles, plan.smem, s) : launch_few<__nv_bfloat16, 32>(p, tiles, plan.smem, s));
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
