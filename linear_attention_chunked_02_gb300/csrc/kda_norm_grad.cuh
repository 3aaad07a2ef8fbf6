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
        if constexpr (sizeof(S) == 1) code_values<VEC>(raw, ckpt_scale(e), v);
        else widen<S, VEC>(raw, v);
    }
};

// act(z) and its slope; the sigmoid's faster form for 16-bit gates and codes, as in the recurrence.
template <bool FULL, int VEC>
__device__ __forceinline__ void act_pair(int silu, const float (&z)[VEC], float (&s)[VEC], float (&slope)[VEC]) {
    float rest[VEC], one[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = z[v], one[v] = 1.f;
    sigmoid_pair<FULL, VEC>(s, rest);
    if (silu) {
        fma_to<VEC>(slope, z, rest, one);
        mul_to<VEC>(slope, slope, s);
        mul_to<VEC>(s, s, z);
    } else {
        mul_to<VEC>(slope, s, rest);
    }
}

// Narrow rows: `lanes` threads to a row (a power of two up to 32), NV vectors to a thread, three rows on their way to a
// thread while a fourth is worked on.  8192 x 64 rows of 128, BF16, with one, two and three rows ahead: 132, 117 and 110 us
// from tensors (floor 99), 123, 111 and 107 from codes (floor 80), which issue bounds.
template <typename T, typename X, typename Z, int VEC, int NV>
__global__ void __launch_bounds__(NORM_GRAD_THREADS, NV == 1 ? 2 : 1) kda_norm_grad_narrow_kernel(const NormGradParams p, const int lanes) {
    constexpr int AHEAD = NV == 1 ? 3 : 1;
    constexpr bool FULL = sizeof(Z) == 4;
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
    struct Row {
        Piece<X, VEC> x[NV];
        Piece<Z, VEC> z[NV];
        Piece<T, VEC> d[NV];
    } next[AHEAD];
    auto fetch = [&](Row &r, int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * lanes + t;
            if (row >= p.rows || j >= nvec) continue;
            r.x[i].fetch(p.x, p.xe, row, p.dim, j * VEC);
            r.z[i].fetch(p.gate, p.ze, row, p.dim, j * VEC);
            r.d[i].fetch(p.dy, nullptr, row, p.dim, j * VEC);
        }
    };
    // the same number of turns for all threads of a block: shuffles go over whole warps
    const int64_t step = int64_t(gridDim.x) * groups, first = int64_t(blockIdx.x) * groups;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) fetch(next[k], first + k * step + group);
    for (int64_t base = first; base < p.rows; base += AHEAD * step) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = base + k * step + group;
            const bool live = row < p.rows;
            float x[NV][VEC], u[NV][VEC], q[NV][VEC], g[NV][VEC], ss = 0.f, ux = 0.f;   // dy w s, dy s, dy w slope
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool have = live && i * lanes + t < nvec;
                float z[VEC], d[VEC], s[VEC], sum[VEC];
                if (have) {
                    next[k].x[i].value(x[i]);
                    next[k].z[i].value(z);
                    next[k].d[i].value(d);
                } else {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) x[i][v] = z[v] = d[v] = 0.f;
                }
                act_pair<FULL, VEC>(p.silu, z, s, g[i]);
                mul_to<VEC>(q[i], d, s);
                mul_to<VEC>(u[i], q[i], w[i]);
                mul_to<VEC>(d, d, w[i]);
                mul_to<VEC>(g[i], d, g[i]);
                mul_to<VEC>(sum, x[i], x[i]);
#pragma unroll
                for (int v = 0; v < VEC; ++v) ss += sum[v];
                mul_to<VEC>(sum, u[i], x[i]);
#pragma unroll
                for (int v = 0; v < VEC; ++v) ux += sum[v];
            }
            fetch(next[k], row + AHEAD * step);
            for (int o = lanes >> 1; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                ux += __shfl_xor_sync(0xffffffffu, ux, o);
            }
            const float r = rsqrtf(ss * p.inv_dim + p.eps), m = ux * p.inv_dim * r * r;   // mean(u n) n = m x
            float rr[VEC], mm[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) rr[v] = r, mm[v] = -m;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = i * lanes + t;
                if (!live || j >= nvec) continue;
                float n[VEC];
                mul_to<VEC>(n, x[i], rr);
                fma_to<VEC>(dw[i], q[i], n, dw[i]);
                mul_to<VEC>(g[i], g[i], n);
                fma_to<VEC>(u[i], mm, x[i], u[i]);
                mul_to<VEC>(u[i], u[i], rr);
                store_raw<T, VEC>(static_cast<T *>(p.dx) + row * p.dim + j * VEC, narrow<T, VEC>(u[i]));
                store_raw<T, VEC>(static_cast<T *>(p.dgate) + row * p.dim + j * VEC, narrow<T, VEC>(g[i]));
            }
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
            float s[VEC], slope[VEC];
            act_pair<sizeof(Z) == 4, VEC>(p.silu, z, s, slope);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                ss = fmaf(x[v], x[v], ss);
                ux = fmaf(d[v] * s[v] * w[v], x[v], ux);
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
            float s[VEC], slope[VEC];
            act_pair<sizeof(Z) == 4, VEC>(p.silu, z, s, slope);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float n = x[v] * r, q = d[v] * s[v];
                ox[v] = r * fmaf(-m, x[v], q * w[v]);
                oz[v] = d[v] * w[v] * slope[v] * n;
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
