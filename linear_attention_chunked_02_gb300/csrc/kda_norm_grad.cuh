// kda_norm_grad.cuh -- the gradients of the gated norm.
//
// With n = x r, r = 1 / sqrt(mean(x^2) + eps), s = act(gate) and u = dy w s,
//
//     dx = r (u - n mean(u n));   dgate = dy n w act'(gate);   dw = sum over rows of dy n s
//
// One pass: a row's x, gate and dy are loaded once, the next rows' on the way meanwhile, the sums of x^2 and of u x are
// taken over its threads, and the row is finished from the registers.  dw is summed in
// registers over the rows that a thread meets, then over a block, and the blocks' sums by a second kernel, all in
// an order that the shape, the types and the alignment set.
//
// Bound by HBM for tensors (8192 x 64 rows of 128, BF16: 111 us, floor 99; 65536 x 512 FP32 110 and 99), for codes by
// issue (107 us, floor 79; 64 % of the slots and 59 % of the DRAM's peak), for unaligned 16-bit rows by single-element loads.
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

// act(z) and its slope; the sigmoid's faster form for 16-bit gates and codes, as in the recurrence, but 0 below 2^-126, at gates
// under -126 ln 2: SiLU's factor z, as low as -3e38 for a mask, would bring 2^-126 back to the size of 1.
template <bool FULL, int VEC>
__device__ __forceinline__ void act_pair(int silu, const float (&z)[VEC], float (&s)[VEC], float (&slope)[VEC]) {
    float rest[VEC], one[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = z[v], one[v] = 1.f;
    sigmoid_pair<FULL, VEC, true>(s, rest);
    if (silu) {
        fma_to<VEC>(slope, z, rest, one);
        mul_to<VEC>(slope, slope, s);
        mul_to<VEC>(s, s, z);
    } else {
        mul_to<VEC>(slope, s, rest);
    }
}

template <int BYTES>
__device__ __forceinline__ void copy_piece(uint32_t at, const void *source) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(source) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(source), "n"(BYTES) : "memory");
}

// One row operand of a thread: NV vectors a row, of type S, AHEAD rows on their way, to the thread's places in shared memory
// with RING (a thread reads what it copied itself), else to registers.
template <typename S, int VEC, int NV, int THREADS, int AHEAD, bool RING>
struct NormSource {
    static constexpr bool CODES = sizeof(S) == 1;
    static constexpr int PIECE = VEC * int(sizeof(S)), ROW = THREADS * NV * PIECE, BYTES = RING ? AHEAD * ROW : 0;
    unsigned char *ring;
    const S *from;              // the thread's first vector of the next row to fetch
    const uint8_t *exps;        // codes: the row's exponents
    int64_t down, exps_down;    // elements from one row of the thread to its next
    raw_t<S, VEC> raw[RING ? 1 : AHEAD][NV];
    unsigned e[CODES ? AHEAD : 1][NV];

    // the thread's rows begin at `row` and are `rows` apart; what it has no vector for reads as zeros
    __device__ __forceinline__ void open(unsigned char *at, const void *base, const uint8_t *exponents, int64_t row, int64_t rows,
                                         int dim, int first, int lanes) {
        ring = at + threadIdx.x * PIECE;
        from = static_cast<const S *>(base) + row * dim + first * VEC;
        down = rows * dim;
        if constexpr (CODES) {
            const int blocks = (dim + CKPT_BLOCK - 1) / CKPT_BLOCK;
            exps = exponents + row * blocks;
            exps_down = rows * blocks;
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (!RING) raw[k][i] = {};
                else if ((first + i * lanes) * VEC >= dim) *reinterpret_cast<raw_t<S, VEC> *>(ring + k * ROW + i * (THREADS * PIECE)) = {};
                if constexpr (CODES) e[k][i] = 0;
            }
        }
    }
    __device__ __forceinline__ void fetch(int k, bool live, int dim, int first, int lanes) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (first + i * lanes) * VEC;
            if (!live || col >= dim) continue;
            if constexpr (RING) copy_piece<PIECE>(smem_u32(ring) + k * ROW + i * (THREADS * PIECE), from + i * lanes * VEC);
            else raw[k][i] = load_once<S, VEC>(from + i * lanes * VEC);
            if constexpr (CODES) e[k][i] = exps[col / CKPT_BLOCK];
        }
        from += down;
        if constexpr (CODES) exps += exps_down;
    }
    __device__ __forceinline__ void value(int k, int i, float (&v)[VEC]) const {
        raw_t<S, VEC> r;
        if constexpr (RING) r = *reinterpret_cast<const raw_t<S, VEC> *>(ring + k * ROW + i * (THREADS * PIECE));
        else r = raw[k][i];
        if constexpr (CODES) code_values<VEC>(r, ckpt_scale(e[k][i]), v);
        else widen<S, VEC>(r, v);
    }
};

template <typename T, typename X, typename Z, int VEC, int NV, int THREADS, int REGS>
struct NormShape {
    static constexpr bool RING = REGS == 0;
    static constexpr int ROW = THREADS * NV * VEC * int(sizeof(T) + sizeof(X) + sizeof(Z)), ROOM = THREADS * 400;
    static constexpr int MOST = sizeof(X) == 1 || sizeof(Z) == 1 ? 2 : 4;   // exponents on their way are in registers
    static constexpr int AHEAD = !RING ? REGS : ROOM / ROW > MOST ? MOST : ROOM / ROW > 2 ? ROOM / ROW : 2;
    using Xs = NormSource<X, VEC, NV, THREADS, AHEAD, RING>;
    using Zs = NormSource<Z, VEC, NV, THREADS, AHEAD, RING>;
    using Ds = NormSource<T, VEC, NV, THREADS, AHEAD, RING>;
    static constexpr int SUMS = THREADS * VEC * 4, BYTES = RING && AHEAD * ROW > SUMS ? AHEAD * ROW : SUMS;
};

// `lanes` threads to a row, a power of two up to 32 or whole warps, and NV vectors to a thread.  REGS: rows on their way in
// registers, or 0 for a ring in shared memory.
template <typename T, typename X, typename Z, int VEC, int NV, int THREADS, int REGS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) kda_norm_grad_kernel(const NormGradParams p, const int lanes) {
    using Shape = NormShape<T, X, Z, VEC, NV, THREADS, REGS>;
    constexpr int AHEAD = Shape::AHEAD;
    constexpr bool FULL = sizeof(Z) == 4, RING = Shape::RING;
    extern __shared__ __align__(16) unsigned char shared[];
    __shared__ float2 part[2][THREADS / 32];
    const int tid = int(threadIdx.x), groups = int(blockDim.x) / lanes, group = tid / lanes, t = tid - group * lanes;
    const int lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    // the same number of turns for all threads of a block: shuffles go over whole warps
    const int64_t step = int64_t(gridDim.x) * groups, first = int64_t(blockIdx.x) * groups;
    typename Shape::Xs xs;
    typename Shape::Zs zs;
    typename Shape::Ds ds;
    xs.open(shared, p.x, p.xe, first + group, step, p.dim, t, lanes);
    zs.open(shared + xs.BYTES, p.gate, p.ze, first + group, step, p.dim, t, lanes);
    ds.open(shared + xs.BYTES + zs.BYTES, p.dy, nullptr, first + group, step, p.dim, t, lanes);
    auto fetch = [&](int64_t row, int k) {
        const bool live = row < p.rows;
        xs.fetch(k, live, p.dim, t, lanes);
        zs.fetch(k, live, p.dim, t, lanes);
        ds.fetch(k, live, p.dim, t, lanes);
        if constexpr (RING) asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) fetch(first + k * step + group, k);
    raw_t<T, VEC> w[NV];
    float dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * lanes + t) * VEC;
        w[i] = col < p.dim ? *reinterpret_cast<const raw_t<T, VEC> *>(static_cast<const T *>(p.weight) + col) : raw_t<T, VEC>{};
#pragma unroll
        for (int v = 0; v < VEC; ++v) dw[i][v] = 0.f;
    }
    int buf = 0;
    T *dx = static_cast<T *>(p.dx) + (first + group) * p.dim + t * VEC, *dgate = static_cast<T *>(p.dgate) + (first + group) * p.dim + t * VEC;
    const int64_t down = step * p.dim;
    auto work = [&](const int64_t row, const int k) {
        // rows and columns that are not there read as zeros: their sums are none
        float x[NV][VEC], q[NV][VEC], g[NV][VEC], ss = 0.f, ux = 0.f;   // q: dy s, g: dy w slope
        if constexpr (RING) asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float z[VEC], d[VEC], s[VEC], wv[VEC], sum[VEC];
            xs.value(k, i, x[i]);
            zs.value(k, i, z);
            ds.value(k, i, d);
            widen<T, VEC>(w[i], wv);
            act_pair<FULL, VEC>(p.silu, z, s, g[i]);
            mul_to<VEC>(q[i], d, s);
            mul_to<VEC>(d, d, wv);
            mul_to<VEC>(g[i], d, g[i]);
            mul_to<VEC>(sum, x[i], x[i]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) ss += sum[v];
            mul_to<VEC>(sum, q[i], wv);
            mul_to<VEC>(sum, sum, x[i]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) ux += sum[v];
        }
        fetch(row + AHEAD * step, k);                       // this row's values are in registers
        for (int o = (lanes < 32 ? lanes : 32) >> 1; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            ux += __shfl_xor_sync(0xffffffffu, ux, o);
        }
        if (lanes > 32) {
            // two sets: the next row's sums go to the other
            if (lane == 0) part[buf][warp] = make_float2(ss, ux);
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
            const int warps = lanes >> 5;
            const float2 *of = &part[buf][group * warps];
            ss = ux = 0.f;
            buf ^= 1;
            for (int i = 0; i < warps; ++i) ss += of[i].x, ux += of[i].y;
        }
        if (row >= p.rows) return;
        const float r = rsqrtf(ss * p.inv_dim + p.eps), m = ux * p.inv_dim * r * r;   // mean(u n) n = m x
        float rr[VEC], mm[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) rr[v] = r, mm[v] = -m;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * lanes + t) * VEC;
            if (col >= p.dim) continue;
            float n[VEC], u[VEC];
            mul_to<VEC>(n, x[i], rr);
            fma_to<VEC>(dw[i], q[i], n, dw[i]);
            mul_to<VEC>(g[i], g[i], n);
            widen<T, VEC>(w[i], u);
            mul_to<VEC>(u, u, q[i]);
            fma_to<VEC>(u, mm, x[i], u);
            mul_to<VEC>(u, u, rr);
            store_raw<T, VEC>(dx + i * lanes * VEC, narrow<T, VEC>(u));
            store_raw<T, VEC>(dgate + i * lanes * VEC, narrow<T, VEC>(g[i]));
        }
    };
    for (int64_t base = first; base < p.rows; base += AHEAD * step) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (k > 0 && base + k * step >= p.rows) break;
            work(base + k * step + group, k);
            dx += down;
            dgate += down;
        }
    }
    if constexpr (RING) asm volatile("cp.async.wait_all;" ::: "memory");
    // the groups' sums, one set of vectors after another
    float *const sums = reinterpret_cast<float *>(shared);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < VEC; ++v) sums[tid * VEC + v] = dw[i][v];
        __syncthreads();
        for (int c = tid; c < lanes * VEC; c += int(blockDim.x)) {
            float sum = 0.f;
            for (int k = 0; k < groups; ++k) sum += sums[k * lanes * VEC + c];
            const int col = i * lanes * VEC + c;
            if (col < p.dim) p.partial[int64_t(blockIdx.x) * p.dim + col] = sum;
        }
    }
}

// Rows that find no room in 512 threads' registers (over 8192 elements, unaligned over 4096): one to a block, read once for
// the sums and once more (from the caches) for the results; dw in shared memory, each thread adding to its own columns.
// 8192 x 16384 BF16: 384 us (floor 198).
constexpr int NORM_GRAD_WIDE = 1024;
template <typename T, typename X, typename Z, int VEC>
__global__ void __launch_bounds__(NORM_GRAD_WIDE) kda_norm_grad_wide_kernel(const NormGradParams p) {
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
