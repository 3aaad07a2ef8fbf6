// kda_norm_grad_launch.cuh -- the gated norm's gradients for one type.
#pragma once

#include "kda_launch.cuh"
#include "kda_norm_grad.cuh"

namespace kda {

// Rows of whole warps, or of a part of one, NV vectors to a thread.
template <typename T, typename X, typename Z, int VEC, int NV, int THREADS, int REGS>
cudaError_t launch_norm_grad_rows(const NormGradParams &p, unsigned grid, cudaStream_t s) {
    using Shape = NormShape<T, X, Z, VEC, NV, THREADS, REGS>;
    constexpr auto kernel = kda_norm_grad_kernel<T, X, Z, VEC, NV, THREADS, REGS>;
    const int each = (p.dim / VEC + NV - 1) / NV;           // threads that have a vector
    int lanes = (each + 31) / 32 * 32;
    if (each <= 32)
        for (lanes = 1; lanes < each;) lanes *= 2;
    if constexpr (Shape::BYTES > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::BYTES);
        if (e != cudaSuccess) return e;
    }
    const unsigned threads = unsigned(lanes <= 32 ? THREADS : THREADS / lanes * lanes);
    return launch_pdl(true, kernel, grid, threads, Shape::BYTES, s, p, lanes);
}

// The threads to a row follow from its vectors: as few as hold it, so that a block has several rows at once and they wait for
// one another's sums as little as can be.
//   one vector of 16 bytes to a thread, up to 256 threads: three rows on their way in registers; with 16-bit
//     tensors and rows of two warps and more, a ring (16384 x 2048 BF16: 63 us, registers 69; 8192 x 64 rows of 128: 121, 111);
//   then 16 elements to a thread and a ring (8192 x 4096 BF16: 62 us, 512 threads and registers 80); from codes, whose
//     exponents and values find no room in 128 registers then, up to 512 threads with registers (80 us, 85);
//   unaligned rows: eight single elements to a thread, one row on its way (8192 x 2305 FP32: 89 us, BF16 78).
template <typename T, typename X, typename Z, int VEC>
cudaError_t launch_norm_grad_vec(const NormGradParams &p, unsigned grid, cudaStream_t s) {
    const int nvec = p.dim / VEC;
    constexpr int FEW = 8, MORE = 16 / VEC;
    constexpr bool CODES = sizeof(X) == 1 || sizeof(Z) == 1;
    if constexpr (VEC > 1) {
        if constexpr (VEC == 8 && !CODES)
            if (nvec > 32 && nvec <= 256) return launch_norm_grad_rows<T, X, Z, VEC, 1, 256, 0>(p, grid, s);
        if (nvec <= 256) return launch_norm_grad_rows<T, X, Z, VEC, 1, 256, 3>(p, grid, s);
        if constexpr (CODES)
            if (nvec <= 512) return launch_norm_grad_rows<T, X, Z, VEC, 1, 512, 3>(p, grid, s);
        if constexpr (!CODES || VEC < 8)
            if (nvec <= 256 * MORE) return launch_norm_grad_rows<T, X, Z, VEC, MORE, 256, 0>(p, grid, s);
        if (nvec <= 512 * MORE) return launch_norm_grad_rows<T, X, Z, VEC, MORE, 512, 0>(p, grid, s);
    } else {
        if (nvec <= 256 * FEW) return launch_norm_grad_rows<T, X, Z, VEC, FEW, 256, 1>(p, grid, s);
        if (nvec <= 512 * FEW) return launch_norm_grad_rows<T, X, Z, VEC, FEW, 512, 1>(p, grid, s);
    }
    const size_t smem = size_t(p.dim) * 4;
    if (smem > 40 * 1024) {                                 // beside what the kernel has of its own, 48 KB without asking
        const cudaError_t e = cudaFuncSetAttribute(kda_norm_grad_wide_kernel<T, X, Z, VEC>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(true, kda_norm_grad_wide_kernel<T, X, Z, VEC>, grid, NORM_GRAD_WIDE, smem, s, p);
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
