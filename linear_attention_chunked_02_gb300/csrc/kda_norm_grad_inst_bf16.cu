// kda_norm_grad_inst_bf16.cu -- the gated norm's gradients for BF16 rows.
#include "kda_norm_grad_launch.cuh"

namespace kda {
cudaError_t launch_norm_grad_bf16(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s) {
    return launch_norm_grad<__nv_bfloat16>(p, l, s);
}
}  // namespace kda
