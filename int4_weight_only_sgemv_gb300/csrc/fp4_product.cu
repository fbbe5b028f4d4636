// The product of two 4-bit matrices: the entry point (argument checks, choice of the kernel).
#include <algorithm>
#include <climits>

#include "fp4_few.cuh"

namespace sgemv {

namespace {

template <typename T, int kBlock>
cudaError_t launch_few(const ProductParams& p, int64_t tiles, cudaStream_t s) {
    auto kern = fp4_few_kernel<T, kBlock>;
    static std::atomic<int> attr_set[64];  // per device: dynamic shared memory already enabled
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (attr_set[dev].load() == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = kFewSmem;
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
    if ((dtype != SGEMV_F16 && dtype != SGEMV_BF16) || w_dev == nullptr || x_dev == nullptr || y_dev == nullptr) return SGEMV_ERR_ARG;
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
    p.k_stages = (w.kp + kStageK - 1) / kStageK;
    p.x_tiles = (x.rows + 127) / 128;
    const int64_t tiles = static_cast<int64_t>((w.rows + 127) / 128) * p.x_tiles;
    // CTAs a tile: as many as fill two places an SM, each with a stage at least
    p.split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, 2 * di.sm_count / tiles, p.k_stages})));
    p.ring = std::min(kFewMaxRing, kFewSmem / few_stage_bytes(w.block, x.tile));
    if (tiles * p.split > INT_MAX) return SGEMV_ERR_SHAPE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool half = dtype == SGEMV_F16;
    const cudaError_t e = w.block == 16 ? (half ? launch_few<__half, 16>(p, tiles, s) : launch_few<__nv_bfloat16, 16>(p, tiles, s))
                                        : (half ? launch_few<__half, 32>(p, tiles, s) : launch_few<__nv_bfloat16, 32>(p, tiles, s));
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}
