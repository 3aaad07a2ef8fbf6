// kda_norm_grad_launch.cuh -- the gated norm's gradients for one type.
#pragma once

#include "kda_launch.cuh"
#include "kda_norm_grad.cuh"

namespace kda {

template <typename T, typename X, typename Z, int VEC>
cudaError_t launch_norm_grad_vec(const NormGradParams &p, unsigned grid, cudaStream_t s) {
    const int nvec = p.dim / VEC;
    if (nvec <= NORM_GRAD_NARROW) {
        int lanes = 1;
        while (lanes < 32 && lanes < nvec) lanes *= 2;
        return nvec > 32
                   ? launch_pdl(true, kda_norm_grad_narrow_kernel<T, X, Z, VEC, 2>, grid, NORM_GRAD_THREADS, 0, s, p, lanes)
                   : launch_pdl(true, kda_norm_grad_narrow_kernel<T, X, Z, VEC, 1>, grid, NORM_GRAD_THREADS, 0, s, p, lanes);
    }
    const size_t smem = size_t(p.dim) * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kda_norm_grad_wide_kernel<T, X, Z, VEC>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    const unsigned threads = unsigned(nvec < 1024 ? (nvec + 31) / 32 * 32 : 1024);
    return launch_pdl(true, kda_norm_grad_wide_kernel<T, X, Z, VEC>, grid, threads, smem, s, p);
}

template <typename T, typename X, typename Z>
cudaError_t launch_norm_grad_xz(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s) {
    return l.wide ? launch_norm_grad_vec<T, X, Z, 16 / int(sizeof(T))>(p, l.grid, s)
                  : launch_norm_grad_vec<T, X, Z, 1>(p, l.grid, s);
}

template <typename T>
cudaError_t launch_norm_grad(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s) {
    if (l.x8) return l.z8 ? launch_norm_grad_xz<T, int8_t, int8_t>(p, l, s) : launch_norm_grad_xz<T, int8_t, T>(p, l, s);
    return l.z8 ? launch_norm_grad_xz<T, T, int8_t>(p, l, s) : launch_norm_grad_xz<T, T, T>(p, l, s);
}

}  // namespace kda
