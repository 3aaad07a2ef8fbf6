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
// The bound is HBM: add_norm of 8192 BF16 rows of 4096 takes 40.7 us, 0.97 of a copy's rate,
// gated_norm of 8192 x 64 rows of 128 62.3 us, 0.95.
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
    float alpha, eps, inv_dim;
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

// VEC values rounded to the type, two at a time where there are two.
template <typename T, int VEC>
__device__ __forceinline__ void pack(Raw<T, VEC> &to, const float (&a)[VEC]) {
    if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
        uint32_t *u = reinterpret_cast<uint32_t *>(&to);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) u[e / 2] = pack2(a[e], a[e + 1], (T *)nullptr);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) put1(&to.v[e], a[e]);
    }
}

// A row's elements on its group of threads: NV vectors of VEC elements to a thread, vector i
// of thread t at element (i tpr + t) VEC.
template <typename T, int KIND, int VEC, int NV>
struct NormRow {
    using R = Raw<T, VEC>;
    R x[NV], z[NV];
    float r[NV][VEC];

    __device__ __forceinline__ void load(const NormParams &p, int64_t row, int t, int tpr, int nvec) {
        const bool second = KIND != NORM_ADD || p.other != nullptr;
        const int64_t base = row * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * tpr + t;
            if (row < p.rows && j < nvec) {
                x[i] = *reinterpret_cast<const R *>(static_cast<const T *>(p.x) + base + int64_t(j) * VEC);
                if (second) z[i] = *reinterpret_cast<const R *>(static_cast<const T *>(p.other) + base + int64_t(j) * VEC);
            }
        }
    }
    // the row to be normed, in FP32; this thread's sum of its squares
    __device__ __forceinline__ float squares(const NormParams &p, int64_t row, int t, int tpr, int nvec) {
        const bool second = KIND != NORM_ADD || p.other != nullptr;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = row < p.rows && i * tpr + t < nvec;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float a = in ? to_f32(x[i].v[e]) : 0.f;
                if (KIND == NORM_ADD) {
                    a *= p.alpha;
                    if (second && in) a += to_f32(z[i].v[e]);
                }
                r[i][e] = a;
                ss = fmaf(a, a, ss);
            }
        }
        return ss;
    }
    __device__ __forceinline__ void store(const NormParams &p, const R (&w)[NV], float inv, int64_t row, int t, int tpr,
                                          int nvec) {
        const int64_t base = row * p.dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * tpr + t;
            if (row >= p.rows || j >= nvec) continue;
            R y, s;
            float a[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                a[e] = r[i][e] * inv * to_f32(w[i].v[e]);
                if (KIND != NORM_ADD) {
                    // 16-bit types take the fast quotient and exponential, whose error grows with a gate below
                    // zero: 6e-6 at -86, far below their rounding, and 0 further down, where the divisor
                    // passes 2^126.  In FP32 that would be 64 units in the last place
                    const float g = to_f32(z[i].v[e]);
                    const float sg = sizeof(T) == 4 ? 1.f / (1.f + expf(-g)) : __fdividef(1.f, 1.f + __expf(-g));
                    a[e] *= KIND == NORM_GATED_SILU ? g * sg : sg;
                }
            }
            pack(y, a);
            if (KIND == NORM_ADD) pack(s, r[i]);
            if (KIND == NORM_ADD && p.out != nullptr)
                *reinterpret_cast<R *>(static_cast<T *>(p.out) + base + int64_t(j) * VEC) = s;
            *reinterpret_cast<R *>(static_cast<T *>(p.y) + base + int64_t(j) * VEC) = y;
        }
    }
};

template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_weight(const NormParams &p, Raw<T, VEC> (&w)[NV], int t, int tpr, int nvec) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * tpr + t;
        if (j < nvec) w[i] = *reinterpret_cast<const Raw<T, VEC> *>(static_cast<const T *>(p.weight) + int64_t(j) * VEC);
    }
}

// Narrow rows: `lanes` threads (a power of two up to 32) to a row, ROWS rows to a thread: one row of
// 128 bf16 values alone keeps 32 bytes of a thread in flight.  Gated norm of 8192 x 64 rows of 128
// (bound: 59 us of copies) with one, two, three and four rows to a thread: 73, 65, 63 and 64 us in
// blocks of 128 threads, 72, 78, 67 and 72 us in blocks of 256; in FP32, half as many rows: 68, 58, 58
// and 58 us in blocks of 128.
constexpr int NORM_THREADS = 128, ROWS = 3;
template <typename T, int KIND, int VEC, int NV>
__global__ void __launch_bounds__(NORM_THREADS) kda_norm_narrow_kernel(const NormParams p, const int lanes) {
    const int t = int(threadIdx.x) & (lanes - 1), groups = NORM_THREADS / lanes;
    const int64_t row0 = int64_t(blockIdx.x) * groups * ROWS + int(threadIdx.x) / lanes;
    const int nvec = p.dim / VEC;              // VEC > 1 only where it divides dim
    pdl_launch_dependents();
    pdl_wait();
    NormRow<T, KIND, VEC, NV> row[ROWS];
    Raw<T, VEC> w[NV];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) row[i].load(p, row0 + i * groups, t, lanes, nvec);
    load_weight<T, VEC, NV>(p, w, t, lanes, nvec);
    float ss[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) ss[i] = row[i].squares(p, row0 + i * groups, t, lanes, nvec);
    for (int o = lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        row[i].store(p, w, rsqrtf(ss[i] * p.inv_dim + p.eps), row0 + i * groups, t, lanes, nvec);
}

// Wide rows: one to a block.
template <typename T, int KIND, int VEC, int NV>
__global__ void __launch_bounds__(1024) kda_norm_wide_kernel(const NormParams p) {
    __shared__ float part[32];
    const int t = threadIdx.x, tpr = blockDim.x, nvec = p.dim / VEC;
    pdl_launch_dependents();
    pdl_wait();
    NormRow<T, KIND, VEC, NV> row;
    Raw<T, VEC> w[NV];
    row.load(p, blockIdx.x, t, tpr, nvec);
    load_weight<T, VEC, NV>(p, w, t, tpr, nvec);
    float ss = row.squares(p, blockIdx.x, t, tpr, nvec);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((t & 31) == 0) part[t >> 5] = ss;
    __syncthreads();
    ss = (t & 31) < (tpr >> 5) ? part[t & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    row.store(p, w, rsqrtf(ss * p.inv_dim + p.eps), blockIdx.x, t, tpr, nvec);
}

template <typename T, int KIND, int VEC, int NV>
cudaError_t launch_narrow(const NormParams &p, int lanes, cudaStream_t s) {
    const int64_t per = int64_t(NORM_THREADS / lanes) * ROWS;
    return launch_pdl(true, kda_norm_narrow_kernel<T, KIND, VEC, NV>, unsigned((p.rows + per - 1) / per), NORM_THREADS,
                      0, s, p, lanes);
}

template <typename T, int KIND, int VEC>
cudaError_t launch_norm(const NormParams &p, cudaStream_t s) {
    const int nvec = p.dim / VEC;
    // rows of up to 64 vectors: up to two vectors to each of up to 32 lanes
    if (nvec <= 64) {
        int lanes = 1;
        while (lanes < 32 && lanes < nvec) lanes *= 2;
        return nvec > 32 ? launch_narrow<T, KIND, VEC, 2>(p, lanes, s) : launch_narrow<T, KIND, VEC, 1>(p, lanes, s);
    }
    // wider rows: one to a block, two vectors to a thread or as many more as 1024 threads need.  add_norm
    // of 8192 BF16 rows of 2048 / 4096 / 8192 with one vector to a thread: 19.7, 41.5 and 92.4 us, with
    // two 19.1, 40.6 and 85.3 us, with four (rows of 4096 and 8192) 53.2 and 107.7 us
    int nv = 2;
    while (nvec > nv * 1024) nv *= 2;
    const unsigned threads = unsigned((nvec + nv - 1) / nv + 31) / 32 * 32;
    const unsigned grid = unsigned(p.rows);
    if (nv == 2) return launch_pdl(true, kda_norm_wide_kernel<T, KIND, VEC, 2>, grid, threads, 0, s, p);
    if (nv == 4) return launch_pdl(true, kda_norm_wide_kernel<T, KIND, VEC, 4>, grid, threads, 0, s, p);
    // only rows read one element at a time are this wide
    if constexpr (VEC == 1) {
        if (nv == 8) return launch_pdl(true, kda_norm_wide_kernel<T, KIND, 1, 8>, grid, threads, 0, s, p);
        return launch_pdl(true, kda_norm_wide_kernel<T, KIND, 1, 16>, grid, threads, 0, s, p);
    }
    return cudaErrorInvalidValue;
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
    const NormParams p{x, residual, weight, y, residual_out, rows, dim, alpha, eps, 1.f / float(dim)};
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
    const NormParams p{x, gate, weight, y, nullptr, rows, dim, 1.f, eps, 1.f / float(dim)};
    return run_norm(act == KDA_ACT_SILU ? NORM_GATED_SILU : NORM_GATED_SIGMOID, dtype, p,
                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
