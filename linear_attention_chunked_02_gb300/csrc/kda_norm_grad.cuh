// kda_norm_grad.cuh -- the gradients of the gated norm.
//
// With n = x r, r = 1 / sqrt(mean(x^2) + eps), s = act(gate) and u = dy w s,
//
//     dx = r (u - n mean(u n));   dgate = dy n w act'(gate);   dw = sum over rows of dy n s
//
// One pass: a row's x, gate and dy are loaded into registers, the sums of x^2 and of u x are
// taken over its threads, and the row is finished from the registers.  dw is summed in
// registers over the rows that a thread meets, then over a block, and the blocks' sums by a second kernel, all in
// an order that the shape alone sets.
#pragma once

#include <cuda_runtime.h>

#include "kda_kernels.cuh"
#include "kda_recur.cuh"
#include "kda_vec.cuh"

namespace kda {

struct NormGradParams {
    const void *dy, *x, *gate, *weight;
    const uint8_t *xe, *ze;     // exponents of codes in place of x, gate
    void *dx, *dgate;
    float *partial;             // [blocks, dim]
    int64_t rows;
    int32_t dim, silu;
    float eps, inv_dim;
};

constexpr int NORM_GRAD_THREADS = 256;
constexpr int NORM_GRAD_NARROW = 64;   // vectors of a row up to which its threads are a part of a warp

// One vector of a row.
template <typename S, int VEC>
struct Piece {
    raw_t<S, VEC> raw;
    unsigned e;

    __device__ __forceinline__ void fetch(const void *base, const uint8_t *exps, int64_t row, int dim, int col) {
        raw = load_once<S, VEC>(static_cast<const S *>(base) + row * dim + col);
        if constexpr (sizeof(S) == 1) e = exps[row * ((dim + CKPT_BLOCK - 1) / CKPT_BLOCK) + col / CKPT_BLOCK];
    }
    __device__ __forceinline__ void value(float (&v)[VEC]) const {
        widen<S, VEC>(raw, v);
        if constexpr (sizeof(S) == 1) {
            const float s = ckpt_scale(e);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] *= s;
        }
    }
};

// act(z) and its slope.
__device__ __forceinline__ void act_pair(int silu, float z, float &s, float &slope) {
    float a[1] = {z}, rest[1];
    sigmoid_pair<true, 1>(a, rest);
    s = silu ? z * a[0] : a[0];
    slope = silu ? a[0] * fmaf(z, rest[0], 1.f) : a[0] * rest[0];
}

// Narrow rows: `lanes` threads to a row (a power of two up to 32), NV vectors to a thread.
template <typename T, typename X, typename Z, int VEC, int NV>
__global__ void __launch_bounds__(NORM_GRAD_THREADS) kda_norm_grad_narrow_kernel(const NormGradParams p, const int lanes) {
    __shared__ float part[NORM_GRAD_THREADS * VEC];
    const int t = int(threadIdx.x) & (lanes - 1), groups = NORM_GRAD_THREADS / lanes, group = int(threadIdx.x) / lanes;
    const int nvec = p.dim / VEC;
    pdl_launch_dependents();
    pdl_wait();
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * lanes + t;
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[i][v] = dw[i][v] = 0.f;
        if (j < nvec) widen<T, VEC>(*reinterpret_cast<const raw_t<T, VEC> *>(static_cast<const T *>(p.weight) + j * VEC), w[i]);
    }
    // the same number of turns for all threads of a warp, whose shuffles go over all of them
    const int64_t step = int64_t(gridDim.x) * groups;
    for (int64_t base = int64_t(blockIdx.x) * groups; base < p.rows; base += step) {
        const int64_t row = base + group;
        const bool live = row < p.rows;
        Piece<X, VEC> xs[NV];
        Piece<Z, VEC> zs[NV];
        Piece<T, VEC> ds[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * lanes + t;
            if (!live || j >= nvec) continue;
            xs[i].fetch(p.x, p.xe, row, p.dim, j * VEC);
            zs[i].fetch(p.gate, p.ze, row, p.dim, j * VEC);
            ds[i].fetch(p.dy, nullptr, row, p.dim, j * VEC);
        }
        float x[NV][VEC], u[NV][VEC], ss = 0.f, ux = 0.f;   // u: dy w s
        float q[NV][VEC], k[NV][VEC];                        // dy s, dy w slope
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool have = live && i * lanes + t < nvec;
            float z[VEC], d[VEC];
            if (have) {
                xs[i].value(x[i]);
                zs[i].value(z);
                ds[i].value(d);
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (!have) x[i][v] = z[v] = d[v] = 0.f;
                float s, slope;
                act_pair(p.silu, z[v], s, slope);
                q[i][v] = d[v] * s;
                k[i][v] = d[v] * w[i][v] * slope;
                u[i][v] = q[i][v] * w[i][v];
                ss = fmaf(x[i][v], x[i][v], ss);
                ux = fmaf(u[i][v], x[i][v], ux);
            }
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            ux += __shfl_xor_sync(0xffffffffu, ux, o);
        }
        const float r = rsqrtf(ss * p.inv_dim + p.eps), m = ux * p.inv_dim * r * r;   // mean(u n) n = m x
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * lanes + t;
            if (!live || j >= nvec) continue;
            float ox[VEC], oz[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float n = x[i][v] * r;
                ox[v] = r * fmaf(-m, x[i][v], u[i][v]);
                oz[v] = k[i][v] * n;
                dw[i][v] = fmaf(q[i][v], n, dw[i][v]);
            }
            store_raw<T, VEC>(static_cast<T *>(p.dx) + row * p.dim + j * VEC, narrow<T, VEC>(ox));
            store_raw<T, VEC>(static_cast<T *>(p.dgate) + row * p.dim + j * VEC, narrow<T, VEC>(oz));
        }
    }
    // the groups' sums, one set of vectors after another
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; ++v) part[threadIdx.x * VEC + v] = dw[i][v];
        __syncthreads();
        for (int c = threadIdx.x; c < lanes * VEC; c += NORM_GRAD_THREADS) {
            float sum = 0.f;
            for (int gq = 0; gq < groups; ++gq) sum += part[gq * lanes * VEC + c];
            const int col = i * lanes * VEC + c;
            if (col < p.dim) p.partial[int64_t(blockIdx.x) * p.dim + col] = sum;
        }
    }
}

// Wide rows: one to a block, read once for the sums and once more (from the caches) for the results; dw in
// shared memory, each thread adding to its own columns.
template <typename T, typename X, typename Z, int VEC>
__global__ void __launch_bounds__(1024) kda_norm_grad_wide_kernel(const NormGradParams p) {
    extern __shared__ float dw[];
    __shared__ float part[2][2][32];
    const int nvec = p.dim / VEC, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    for (int j = threadIdx.x; j < nvec; j += blockDim.x) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) dw[j * VEC + v] = 0.f;
    }
    int buf = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, buf ^= 1) {
        float ss = 0.f, ux = 0.f;
        for (int j = threadIdx.x; j < nvec; j += blockDim.x) {
            Piece<X, VEC> xs;
            Piece<Z, VEC> zs;
            Piece<T, VEC> ds;
            xs.fetch(p.x, p.xe, row, p.dim, j * VEC);
            zs.fetch(p.gate, p.ze, row, p.dim, j * VEC);
            ds.fetch(p.dy, nullptr, row, p.dim, j * VEC);
            float x[VEC], z[VEC], d[VEC], w[VEC];
            xs.value(x);
            zs.value(z);
            ds.value(d);
            widen<T, VEC>(*reinterpret_cast<const raw_t<T, VEC> *>(static_cast<const T *>(p.weight) + j * VEC), w);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float s, slope;
                act_pair(p.silu, z[v], s, slope);
                ss = fmaf(x[v], x[v], ss);
                ux = fmaf(d[v] * s * w[v], x[v], ux);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            ux += __shfl_xor_sync(0xffffffffu, ux, o);
        }
        if (lane == 0) part[buf][0][warp] = ss, part[buf][1][warp] = ux;
        __syncthreads();                                    // two sets: the next row's sums go to the other
        ss = lane < warps ? part[buf][0][lane] : 0.f;
        ux = lane < warps ? part[buf][1][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            ux += __shfl_xor_sync(0xffffffffu, ux, o);
        }
        const float r = rsqrtf(ss * p.inv_dim + p.eps), m = ux * p.inv_dim * r * r;
        for (int j = threadIdx.x; j < nvec; j += blockDim.x) {
            Piece<X, VEC> xs;
            Piece<Z, VEC> zs;
            Piece<T, VEC> ds;
            xs.fetch(p.x, p.xe, row, p.dim, j * VEC);
            zs.fetch(p.gate, p.ze, row, p.dim, j * VEC);
            ds.fetch(p.dy, nullptr, row, p.dim, j * VEC);
            float x[VEC], z[VEC], d[VEC], w[VEC], ox[VEC], oz[VEC];
            xs.value(x);
            zs.value(z);
            ds.value(d);
            widen<T, VEC>(*reinterpret_cast<const raw_t<T, VEC> *>(static_cast<const T *>(p.weight) + j * VEC), w);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float s, slope;
                act_pair(p.silu, z[v], s, slope);
                const float n = x[v] * r, q = d[v] * s;
                ox[v] = r * fmaf(-m, x[v], q * w[v]);
                oz[v] = d[v] * w[v] * slope * n;
                dw[j * VEC + v] = fmaf(q, n, dw[j * VEC + v]);
            }
            store_raw<T, VEC>(static_cast<T *>(p.dx) + row * p.dim + j * VEC, narrow<T, VEC>(ox));
            store_raw<T, VEC>(static_cast<T *>(p.dgate) + row * p.dim + j * VEC, narrow<T, VEC>(oz));
        }
    }
    for (int j = threadIdx.x; j < nvec; j += blockDim.x) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) p.partial[int64_t(blockIdx.x) * p.dim + j * VEC + v] = dw[j * VEC + v];
    }
}

struct NormGradLaunch {
    bool x8, z8, wide;          // wide: vectors of 16 bytes of T, else single elements
    unsigned grid;
};

cudaError_t launch_norm_grad_f32(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s);
cudaError_t launch_norm_grad_bf16(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s);
cudaError_t launch_norm_grad_f16(const NormGradParams &p, const NormGradLaunch &l, cudaStream_t s);

}  // namespace kda
