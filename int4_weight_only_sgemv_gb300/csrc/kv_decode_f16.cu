// Decode attention kernels of fp16 queries.
#include "kv_decode_launch.cuh"

namespace sgemv {
cudaError_t launch_decode_f16(int dim, int group, const AttnParams& p, int sms, cudaStream_t s) {
    return launch_decode<__half>(dim, group, p, sms, s);
}
}  // namespace sgemv
