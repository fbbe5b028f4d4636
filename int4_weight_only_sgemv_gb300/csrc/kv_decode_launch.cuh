// Launcher of decode_kernel<T, ...>, shared by the translation units of the two query types.
#pragma once

#include <algorithm>

#include "kv_decode.cuh"

namespace sgemv {

template <typename T, int D, int G, int NT>
cudaError_t launch_decode_shape(const AttnParams& p, int sms, cudaStream_t s) {
    using S = AttnShape<D, G, NT>;
    static_assert(4096 + 4 * (kMaxCtas * (S::kWarps + 2)) * S::kPartial <= SGEMV_KV_WORKSPACE, "workspace");
    auto kern = decode_kernel<T, D, G, NT>;
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
    const int grid = sms < kMaxCtas ? sms : kMaxCtas;
    return launch_pdl(kern, dim3(grid), dim3(S::kThreads), S::kSmem, s, p);
}

template <typename T, int D, int G>
cudaError_t launch_decode_rows(const AttnParams& p, int sms, cudaStream_t s) {
    const int64_t rows = std::min(static_cast<int64_t>(p.q.max_q) * p.ratio, static_cast<int64_t>(p.max_rows));
    if (rows <= 8) return launch_decode_shape<T, D, G, 1>(p, sms, s);
    if constexpr (D == 256) return launch_decode_shape<T, D, G, 1>(p, sms, s);
    else return launch_decode_shape<T, D, G, 2>(p, sms, s);  // more rows are more row tiles
}

template <typename T>
cudaError_t launch_decode(int dim, int group, const AttnParams& p, int sms, cudaStream_t s) {
    if (dim == 64) return launch_decode_rows<T, 64, 64>(p, sms, s);
    if (dim == 128 && group == 64) return launch_decode_rows<T, 128, 64>(p, sms, s);
    if (dim == 128) return launch_decode_rows<T, 128, 128>(p, sms, s);
    if (group == 64) return launch_decode_rows<T, 256, 64>(p, sms, s);
    return launch_decode_rows<T, 256, 128>(p, sms, s);
}

}  // namespace sgemv
