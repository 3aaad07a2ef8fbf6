// kda_norm.cu -- the norms of a gated-delta-rule layer: kda_add_norm (residual
// sum, then the norm before the block) and kda_gated_norm (the norm after it,
// times its gate).
//
//   add:    r = residual + alpha x;  y = r rsqrt(mean(r^2) + eps) weight
//   gated:  y = x rsqrt(mean(x^2) + eps) weight act(gate)
//
// Both read every input once and write every output once: a row is loaded into
// registers, its squares are summed in FP32 over the row's threads, and the row
// is finished from the registers (so y or residual_out may be an input's buffer).
// The bound is HBM; nothing else is close.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_launch.cuh"
#include "kda_layer.h"

namespace kda {
namespace {

struct NormParams {
    const void *x;         // [rows, dim]
    const void *other;     // add: residual or nullptr; gated: gate
    const void *weight;    // [dim]
    void *y;               // [rows, dim]
    void *out;             // add: residual_out or nullptr
    int64_t rows;
    int32_t dim;
    float alpha, eps;
};

enum { NORM_ADD = 0, NORM_GATED_SIGMOID = 1, NORM_GATED_SILU = 2 };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// VEC consecutive elements as they lie in memory: 16 bytes, or one element.
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Raw {
    T v[VEC];
};

// One row for each group of TPR threads (a power of two up to 32: several rows to a
// warp; else TPR is the block: one row to a block), NV vectors of VEC elements
// to a thread, vector i of thread t at element (i TPR + t) VEC.
template <typename T, int KIND, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 256) kda_norm_kernel(const NormParams p, const int lanes) {
    const int tpr = BLOCK ? int(blockDim.x) : lanes;
    const int t = BLOCK ? int(threadIdx.x) : int(threadIdx.x) & (lanes - 1);
    const int64_t row = BLOCK ? int64_t(blockIdx.x)
                              : int64_t(blockIdx.x) * (blockDim.x / lanes) + int(threadIdx.x) / lanes;
    using R = Raw<T, VEC>;
    pdl_launch_dependents();
    pdl_wait();
    const bool live = row < p.rows;
    const int nvec = p.dim / VEC;              // VEC > 1 only where it divides dim
    const int64_t base = row * p.dim;
    R xr[NV], zr[NV];
    const bool second = KIND != NORM_ADD || p.other != nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * tpr + t;
        if (live && j < nvec) {
            xr[i] = *reinterpret_cast<const R *>(static_cast<const T *>(p.x) + base + int64_t(j) * VEC);
            if (second) zr[i] = *reinterpret_cast<const R *>(static_cast<const T *>(p.other) + base + int64_t(j) * VEC);
        }
    }
    float r[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = live && i * tpr + t < nvec;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float a = in ? to_f32(xr[i].v[e]) : 0.f;
            if (KIND == NORM_ADD) {
                a *= p.alpha;
                if (second && in) a += to_f32(zr[i].v[e]);
            }
            r[i][e] = a;
            ss = fmaf(a, a, ss);
        }
    }
    if (BLOCK) {
        __shared__ float part[32];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = (threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    } else {
        for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (!live) return;
    const float inv = rsqrtf(ss / float(p.dim) + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * tpr + t;
        if (j >= nvec) break;
        const R w = *reinterpret_cast<const R *>(static_cast<const T *>(p.weight) + int64_t(j) * VEC);
        R y, s;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float a = r[i][e] * inv * to_f32(w.v[e]);
            if (KIND != NORM_ADD) {
                const float z = to_f32(zr[i].v[e]);
                const float g = 1.f / (1.f + __expf(-z));
                a *= KIND == NORM_GATED_SILU ? z * g : g;
            }
            put1(&y.v[e], a);
            if (KIND == NORM_ADD) put1(&s.v[e], r[i][e]);
        }
        if (KIND == NORM_ADD && p.out != nullptr)
            *reinterpret_cast<R *>(static_cast<T *>(p.out) + base + int64_t(j) * VEC) = s;
        *reinterpret_cast<R *>(static_cast<T *>(p.y) + base + int64_t(j) * VEC) = y;
    }
}

constexpr int NORM_THREADS = 256;              // block of the several-rows form

template <typename T, int KIND, int VEC>
cudaError_t launch_norm(const NormParams &p, cudaStream_t s) {
    const int nvec = p.dim / VEC;
    // rows of up to 64 vectors: up to two vectors to each of up to 32 lanes
    if (nvec <= 64) {
        int lanes = 1;
        while (lanes < 32 && lanes < nvec) lanes *= 2;
        const int64_t per = NORM_THREADS / lanes;
        const int64_t grid = (p.rows + per - 1) / per;
        if (nvec <= 32)
            return launch_pdl(true, kda_norm_kernel<T, KIND, VEC, 1, false>, unsigned(grid), NORM_THREADS, 0, s, p, lanes);
        return launch_pdl(true, kda_norm_kernel<T, KIND, VEC, 2, false>, unsigned(grid), NORM_THREADS, 0, s, p, lanes);
    }
    // wider rows: one to a block, as few vectors to a thread as 1024 threads allow
    // (two from 256 vectors on: fewer, busier warps to sum over)
    int nv = 1;
    while ((nv < 2 && nvec > 256) || nvec > nv * 1024) nv *= 2;
    const unsigned threads = unsigned((nvec + nv - 1) / nv + 31) / 32 * 32;
    const unsigned grid = unsigned(p.rows);
    switch (nv) {
        case 1: return launch_pdl(true, kda_norm_kernel<T, KIND, VEC, 1, true>, grid, threads, 0, s, p, 0);
        case 2: return launch_pdl(true, kda_norm_kernel<T, KIND, VEC, 2, true>, grid, threads, 0, s, p, 0);
        case 4: return launch_pdl(true, kda_norm_kernel<T, KIND, VEC, 4, true>, grid, threads, 0, s, p, 0);
        case 8: if (VEC == 1) return launch_pdl(true, kda_norm_kernel<T, KIND, 1, 8, true>, grid, threads, 0, s, p, 0);
        default: return launch_pdl(true, kda_norm_kernel<T, KIND, 1, 16, true>, grid, threads, 0, s, p, 0);
    }
}

template <typename T>
cudaError_t launch_kind(int kind, const NormParams &p, cudaStream_t s) {
    // 16-byte vectors where every row of every tensor starts on one
    constexpr int VEC = 16 / int(sizeof(T));
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.other) |
                         reinterpret_cast<uintptr_t>(p.weight) | reinterpret_cast<uintptr_t>(p.y) |
                         reinterpret_cast<uintptr_t>(p.out);
    const bool wide = (at & 15u) == 0 && p.dim % VEC == 0;
    switch (kind) {
        case NORM_ADD: return wide ? launch_norm<T, NORM_ADD, VEC>(p, s) : launch_norm<T, NORM_ADD, 1>(p, s);
        case NORM_GATED_SIGMOID:
            return wide ? launch_norm<T, NORM_GATED_SIGMOID, VEC>(p, s) : launch_norm<T, NORM_GATED_SIGMOID, 1>(p, s);
        default: return wide ? launch_norm<T, NORM_GATED_SILU, VEC>(p, s) : launch_norm<T, NORM_GATED_SILU, 1>(p, s);
    }
}

kda_status_t run_norm(int kind, int32_t dtype, const NormParams &p, cudaStream_t s) {
    cudaError_t e;
    switch (dtype) {
        case KDA_F32: e = launch_kind<float>(kind, p, s); break;
        case KDA_BF16: e = launch_kind<__nv_bfloat16>(kind, p, s); break;
        default: e = launch_kind<__half>(kind, p, s); break;
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Checks shared by the two entries; sizes are those of every [rows, dim] tensor.
kda_status_t check_norm(int64_t rows, int32_t dim, float eps, int32_t dtype) {
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || dim < 1 || !(eps >= 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    if (dim > KDA_NORM_MAX_DIM || rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_add_norm(const void *x, const void *residual, const void *weight, void *y, void *residual_out,
                          int64_t rows, int32_t dim, float alpha, float eps, int32_t dtype, void *stream) {
    const kda_status_t st = check_norm(rows, dim, eps, dtype);
    if (st != KDA_OK || rows == 0) return st;
    const size_t es = size_t(elt_size(dtype)), n = size_t(rows) * size_t(dim) * es, wn = size_t(dim) * es;
    if (x == nullptr || weight == nullptr || y == nullptr) return KDA_ERR_INVALID_ARGUMENT;
    for (const void *q : {x, residual, weight, static_cast<const void *>(y), static_cast<const void *>(residual_out)})
        if (reinterpret_cast<uintptr_t>(q) % es != 0) return KDA_ERR_INVALID_ARGUMENT;
    if ((y != x && overlaps(y, n, x, n)) || overlaps(y, n, weight, wn) ||
        (residual != nullptr && overlaps(y, n, residual, n)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (residual_out != nullptr &&
        (overlaps(residual_out, n, x, n) || overlaps(residual_out, n, y, n) || overlaps(residual_out, n, weight, wn) ||
         (residual != nullptr && residual_out != residual && overlaps(residual_out, n, residual, n))))
        return KDA_ERR_INVALID_ARGUMENT;
    const NormParams p{x, residual, weight, y, residual_out, rows, dim, alpha, eps};
    return run_norm(NORM_ADD, dtype, p, static_cast<cudaStream_t>(stream));
}

kda_status_t kda_gated_norm(const void *x, const void *gate, const void *weight, void *y, int64_t rows, int32_t dim,
                            float eps, int32_t act, int32_t dtype, void *stream) {
    const kda_status_t st = check_norm(rows, dim, eps, dtype);
    if (st != KDA_OK) return st;
    if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARGUMENT;
    if (rows == 0) return KDA_OK;
    const size_t es = size_t(elt_size(dtype)), n = size_t(rows) * size_t(dim) * es, wn = size_t(dim) * es;
    if (x == nullptr || gate == nullptr || weight == nullptr || y == nullptr) return KDA_ERR_INVALID_ARGUMENT;
    for (const void *q : {x, gate, weight, static_cast<const void *>(y)})
        if (reinterpret_cast<uintptr_t>(q) % es != 0) return KDA_ERR_INVALID_ARGUMENT;
    if ((y != x && overlaps(y, n, x, n)) || (y != gate && overlaps(y, n, gate, n)) || overlaps(y, n, weight, wn))
        return KDA_ERR_INVALID_ARGUMENT;
    const NormParams p{x, gate, weight, y, nullptr, rows, dim, 1.f, eps};
    return run_norm(act == KDA_ACT_SILU ? NORM_GATED_SILU : NORM_GATED_SIGMOID, dtype, p,
                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
