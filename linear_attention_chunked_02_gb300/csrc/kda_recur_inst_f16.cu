// kda_recur_inst_f16.cu -- the recurrence and its gradients for F16 inputs.
#include "kda_recur_launch.cuh"

namespace kda {
cudaError_t launch_scan_f16(RecurParams &p, const RecurLaunch &l, cudaStream_t s) { return launch_scan<__half>(p, l, s); }
cudaError_t launch_scan_backward_f16(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return launch_backward<__half>(p, l, s);
}
}  // namespace kda
