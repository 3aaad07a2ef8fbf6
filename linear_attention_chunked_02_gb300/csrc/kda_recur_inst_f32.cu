// kda_recur_inst_f32.cu -- the recurrence and its gradients for F32 inputs.
#include "kda_recur_launch.cuh"

namespace kda {
cudaError_t launch_scan_f32(RecurParams &p, const RecurLaunch &l, cudaStream_t s) { return launch_scan<float>(p, l, s); }
cudaError_t launch_scan_backward_f32(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return launch_backward<float>(p, l, s);
}
}  // namespace kda
