// kda_norm_grad_inst_f16.cu -- the gated norm's gradients for F16 rows.
#include "kda_norm_grad_launch.cuh"

namespace kda {
cudaError_t launch_norm_grad_f16(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s) {
    return launch_norm_grad<__half>(p, l, s);
}
}  // namespace kda
