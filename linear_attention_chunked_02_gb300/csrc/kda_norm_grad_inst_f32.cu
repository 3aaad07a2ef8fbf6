// kda_norm_grad_inst_f32.cu -- the gated norm's gradients for F32 rows.
#include "kda_norm_grad_launch.cuh"

namespace kda {
cudaError_t launch_norm_grad_f32(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s) {
    return launch_norm_grad<float>(p, l, s);
}
}  // namespace kda
