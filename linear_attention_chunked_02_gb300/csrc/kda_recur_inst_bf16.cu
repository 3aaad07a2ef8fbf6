// kda_recur_inst_bf16.cu -- the recurrence and its gradients for BF16 inputs.
#include "kda_recur_launch.cuh"

namespace kda {
cudaError_t launch_scan_bf16(RecurParams &p, const RecurLaunch &l, cudaStream_t s) { return launch_scan<__nv_bfloat16>(p, l, s); }
cudaError_t launch_scan_backward_bf16(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return launch_backward<__nv_bfloat16>(p, l, s);
}
}  // namespace kda
