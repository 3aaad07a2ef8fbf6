// The chunked gated delta rule for bf16.
#include "kda_delta_launch.cuh"

namespace kda {
cudaError_t launch_chunked_bf16(const DeltaParams &p, const DeltaMaps &prep, const DeltaMaps &scan, int device, int sms,
                               cudaStream_t s) {
    return launch_chunked<__nv_bfloat16>(p, prep, scan, device, sms, s);
}
}  // namespace kda
