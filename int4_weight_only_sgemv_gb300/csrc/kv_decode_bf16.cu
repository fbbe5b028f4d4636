// Decode attention kernels of bf16 queries.
#include "kv_decode_launch.cuh"

namespace sgemv {
cudaError_t launch_decode_bf16(int dim, int group, const AttnParams& p, int sms, cudaStream_t s) {
    return launch_decode<__nv_bfloat16>(dim, group, p, sms, s);
}
}  // namespace sgemv
