// kda_norm_grad.cu -- C ABI of the gated norm's gradients: checks, launch shape, and the
// sum of the blocks' weight gradients.
#include <cuda_runtime.h>

#include "kda_internal.h"
#include "kda_launch.cuh"
#include "kda_norm_grad.cuh"
#include "kda_recurrent.h"
#include "kda_spans.h"

namespace {

using namespace kda;

// dweight[c] = sum of partial[b][c] over the blocks: 32 columns to a block, its warps taking every eighth partial sum.
__global__ void __launch_bounds__(256) kda_norm_grad_sum_kernel(const float *partial, float *dweight, int blocks, int dim) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = int(blockIdx.x) * 32 + lane;
    pdl_launch_dependents();
    pdl_wait();
    float sum = 0.f;
    if (col < dim)
        for (int b = warp; b < blocks; b += 8) sum += partial[int64_t(b) * dim + col];
    part[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || col >= dim) return;
    for (int w = 1; w < 8; ++w) sum += part[w][lane];
    dweight[col] = sum;
}

// Blocks of the first kernel: two to an SM, or one to a row where there are fewer.  The workspace's size
// follows from them, so that they do not depend on alignment.
unsigned norm_grad_blocks(int64_t rows, int32_t dim) {
    const int64_t most = 152 * 2, each = dim <= 32 ? 8 : 1, need = (rows + each - 1) / each;
    return unsigned(need < most ? need : most);
}

}  // namespace

extern "C" {

size_t kda_gated_norm_backward_workspace_size(int64_t rows, int32_t dim) {
    if (rows < 1 || dim < 1 || dim > KDA_NORM_MAX_DIM) return 0;
    return (size_t(norm_grad_blocks(rows, dim)) * size_t(dim) * 4 + 15) / 16 * 16;
}

kda_status_t kda_gated_norm_backward(const void *dy, const void *x, const uint8_t *x_exponents, const void *gate,
                                     const uint8_t *gate_exponents, const void *weight, void *dx, void *dgate,
                                     float *dweight, int64_t rows, int32_t dim, float eps, int32_t act, int32_t dtype,
                                     void *workspace, size_t workspace_bytes, void *stream) {
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || dim < 1 || !(eps >= 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARGUMENT;
    if (dim > KDA_NORM_MAX_DIM || rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (dweight == nullptr || !aligned_to(dweight, 4)) return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned grid = 0;
    float *partial = nullptr;
    if (rows > 0) {
        const bool x8 = x_exponents != nullptr, z8 = gate_exponents != nullptr;
        const size_t es = size_t(elt_size(dtype)), n = size_t(rows) * size_t(dim), wn = size_t(dim) * es;
        const size_t ex = size_t(rows) * size_t((dim + CKPT_BLOCK - 1) / CKPT_BLOCK);
        if (dy == nullptr || x == nullptr || gate == nullptr || weight == nullptr || dx == nullptr || dgate == nullptr)
            return KDA_ERR_INVALID_ARGUMENT;
        if (!aligned_to(dy, es) || !aligned_to(weight, es) || !aligned_to(dx, es) || !aligned_to(dgate, es) ||
            !aligned_to(x, x8 ? 1 : es) || !aligned_to(gate, z8 ? 1 : es))
            return KDA_ERR_INVALID_ARGUMENT;
        const size_t need = kda_gated_norm_backward_workspace_size(rows, dim);
        if (workspace == nullptr || workspace_bytes < need) return KDA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return KDA_ERR_INVALID_ARGUMENT;
        const Span in[] = {{dy, n * es}, {x, n * (x8 ? 1 : es)}, {gate, n * (z8 ? 1 : es)}, {weight, wn},
                           {x_exponents, ex}, {gate_exponents, ex}};
        const Span out[] = {{dx, n * es}, {dgate, n * es}, {dweight, size_t(dim) * 4}, {workspace, need}};
        if (any_meet(out, in)) return KDA_ERR_INVALID_ARGUMENT;
        grid = norm_grad_blocks(rows, dim);
        partial = static_cast<float *>(workspace);
        const NormGradParams p{dy, x, gate, weight, x_exponents, gate_exponents, dx, dgate, partial, rows, dim,
                               act == KDA_ACT_SILU, eps, 1.f / float(dim)};
        // vectors of 16 bytes of the type (and as many codes) where every row of every tensor starts on one
        const size_t vec = 16 / es;
        const bool wide = size_t(dim) % vec == 0 && aligned16(dy) && aligned16(weight) && aligned16(dx) &&
                          aligned16(dgate) && aligned_to(x, x8 ? vec : 16) && aligned_to(gate, z8 ? vec : 16);
        const NormGradLaunch l{x8, z8, wide, grid};
        const cudaError_t e = dtype == KDA_F32    ? launch_norm_grad_f32(p, l, s)
                              : dtype == KDA_BF16 ? launch_norm_grad_bf16(p, l, s)
                                                  : launch_norm_grad_f16(p, l, s);
        if (e != cudaSuccess) return KDA_ERR_CUDA;
    }
    const cudaError_t e = launch_pdl(true, kda_norm_grad_sum_kernel, unsigned((dim + 31) / 32), 256, 0, s,
                                     static_cast<const float *>(partial), dweight, int(grid), int(dim));
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
