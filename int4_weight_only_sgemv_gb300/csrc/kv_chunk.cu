// Prompt-chunk attention kernels.
#include <algorithm>
#include <climits>

#include "kv_chunk.cuh"

namespace sgemv {

namespace {

template <typename T, int D, int G>
cudaError_t launch_chunk_shape(const AttnParams& p, cudaStream_t s) {
    using S = ChunkShape<D, G>;
    static_assert(4096 + 4ull * kMaxCtas * S::kPartial <= SGEMV_KV_WORKSPACE, "workspace");
    auto kern = chunk_kernel<T, D, G>;
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
    // at most so many segments: every request's last row tile may be short
    const int64_t most = (static_cast<int64_t>(p.q.n_tokens) * p.ratio / S::kRows + p.q.n_req) * p.heads;
    const int64_t grid = std::max<int64_t>(kMaxCtas, most);
    if (grid > INT_MAX) return cudaErrorInvalidValue;
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), S::kSmem, s, p);
}

template <typename T>
cudaError_t launch_chunk_type(int dim, int group, const AttnParams& p, cudaStream_t s) {
    if (dim == 64) return launch_chunk_shape<T, 64, 64>(p, s);
    if (group == 64) return launch_chunk_shape<T, 128, 64>(p, s);
    return launch_chunk_shape<T, 128, 128>(p, s);
}

}  // namespace

cudaError_t launch_chunk(int dtype, int dim, int group, const AttnParams& p, cudaStream_t s) {
    return dtype == SGEMV_F16 ? launch_chunk_type<__half>(dim, group, p, s)
                              : launch_chunk_type<__nv_bfloat16>(dim, group, p, s);
}

}  // namespace sgemv
