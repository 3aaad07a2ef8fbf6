// The chunked gated delta rule for f16.
#include "kda_delta_launch.cuh"

namespace kda {
cudaError_t launch_chunked_f16(const DeltaParams &p, const DeltaMaps &prep, const DeltaMaps &scan, int device, int sms,
                               cudaStream_t s) {
    return launch_chunked<__half>(p, prep, scan, device, sms, s);
}
}  // namespace kda
