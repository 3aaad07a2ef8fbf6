// kda_recur.cu -- C ABI of the gated linear recurrence (argument checks, launch shapes), the
// decoding step, and 8-bit checkpoints of activations.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda_internal.h"
#include "kda_launch.cuh"
#include "kda_recur_launch.h"
#include "kda_recurrent.h"
#include "kda_spans.h"

namespace kda {

// Packed sequences whose lengths every block looks through.  65536 rows of 2048 channels, BF16, in 4096, 20000 and 65536
// sequences: 236, 291 and 392 us walked, 511, 550 and 684 chained.  Blocks that do not walk come one after the other
// and look each: gradients in 20000 sequences 510 us by parts alone and 579 by clusters, in 65536 864 and 687.
constexpr int MOST_LOOKED_AT = 1 << 16, MOST_LOOKED_AT_OFTEN = 1 << 15;

// Whether and how single warps walk the sequences: where there are enough of them for all SMs.  16 x 512 rows of 8192
// channels in BF16 take 61 us by 1024 warps of 128 channels each, 97 chained; 8 sequences' 512 warps 83, 1024 of half the
// channels 70.  Packed sequences are walked where none is longer than three parts of the stream, which the device sees.
// A lane takes `wide` channels, or half as many where that makes too few warps or `fit` says that the outputs' and
// states' addresses do not fit vectors of more (16 x 512 x 8192: 80 us; 65536 rows of 2048 in 4096 sequences 420, by four
// channels 235).
static bool walk_grid(RecurParams &p, int wide, int fit) {
    constexpr int64_t WARPS = 152 * 6;
    if (wide == 0 || p.rows == 0 || (p.cu != nullptr && p.nseq > MOST_LOOKED_AT)) return false;
    for (int vec = wide; vec >= wide / 2; vec -= wide / 2) {
        if (vec > fit) continue;
        const int64_t slabs = (p.D + 32 * vec - 1) / (32 * vec);
        if (slabs * p.nseq < WARPS) continue;
        int64_t parts = 2 * WARPS / slabs > 1 ? 2 * WARPS / slabs : 1;
        if (parts > p.nseq) parts = p.nseq;
        if (p.cu == nullptr) {
            const int64_t each = (p.nseq + parts - 1) / parts;
            parts = (p.nseq + each - 1) / each;
            p.walk_part = int32_t(each * p.T);
        } else {
            p.walk_part = int32_t((p.T + parts - 1) / parts);
            parts = (p.T + p.walk_part - 1) / p.walk_part;
            p.walk_most = p.walk_part < INT32_MAX / 3 ? 3 * p.walk_part : INT32_MAX;
        }
        p.walk_parts = int32_t(parts);
        p.walk_wide = vec == wide;
        return true;
    }
    return false;
}

// The grid: as many blocks as run at once, by clusters that share the rows and, for what they leave, by parts of the stream.  A
// cluster's size is the one that takes the fewest rounds of tiles, a round counting a sixth more where blocks
// exchange and a block half a round for its beginning.  Clusters come first for packed sequences, whose lengths only the
// device knows: however they differ, the blocks of a cluster share the rows.  Where the device sees that they are
// alike, or none longer than half a block's part, the blocks take parts of their own all the same, which saves the
// exchange (gradients of 16 x 512 rows of 8192 channels, BF16: 120 us, 158 by clusters of two).
RecurGrid recur_grid(RecurParams &p, const RecurRoom &room, int columns, int tile, int walk_wide, int walk_fit) {
    const int64_t slabs = (p.D + columns - 1) / columns, T = p.T, seqs = p.cu == nullptr ? p.nseq : 1;
    p.slabs = int32_t(slabs);
    if (walk_grid(p, walk_wide, walk_fit) && p.cu == nullptr) return {1, unsigned(room.blocks[1])};   // all warps of the blocks walk
    int64_t parts = 1, each = 1;
    int size = 1;
    double best = 0;
    for (int k = 1; k <= RECUR_CLUSTER; ++k) {
        if (room.blocks[k] == 0) continue;
        const int64_t fit = room.blocks[k] / (slabs * k) > 1 ? room.blocks[k] / (slabs * k) : 1;
        for (int64_t most = fit; most <= 8 * fit; most += fit) {             // also parts that run one after the other
            const int64_t m = most < seqs ? most : seqs > 0 ? seqs : 1;
            const int64_t per = seqs > 0 ? (seqs + m - 1) / m : 1, n = seqs > 0 ? (seqs + per - 1) / per : 1;
            const int64_t waves = (slabs * k * n + room.blocks[k] - 1) / room.blocks[k];
            const double rounds = double((per * T + tile * k - 1) / (tile * k));
            const double cost = double(waves) * (rounds * (k > 1 ? 7. / 6. : 1.) + 0.5);
            if (best == 0 || cost < best) best = cost, size = k, parts = n, each = per;
            if (m < most) break;
        }
    }
    if (p.cu == nullptr) {
        p.part = int32_t(each * T);
        p.parts = int32_t(parts);
        return {unsigned(size), unsigned(slabs * parts)};
    }
    const int64_t fit = room.blocks[size] / (slabs * size);
    // parts that run one after the other even out the end, as long as they hold two sequences each; walking warps are
    // all of the blocks' that run at once
    parts = p.walk_parts > 0 && fit > 0 ? fit : 4 * fit;
    while (parts > fit && 2 * parts * size > p.nseq) --parts;
    if (parts > p.nseq) parts = p.nseq;
    if (parts < 1) parts = 1;
    p.part = int32_t((T + parts - 1) / parts > 1 ? (T + parts - 1) / parts : 1);
    parts = T > 0 ? (T + p.part - 1) / p.part : 1;
    if (size > 1 && p.nseq > 1 && p.nseq <= MOST_LOOKED_AT_OFTEN) {
        const int64_t alone = parts * size;
        p.solo_part = int32_t((T + alone - 1) / alone > 1 ? (T + alone - 1) / alone : 1);
        const int64_t alike = p.nseq % alone == 0 || p.nseq >= 4 * alone ? T / p.nseq + T / p.nseq / 8 : 0;
        p.solo_most = int32_t(alike > p.solo_part / 2 ? alike : p.solo_part / 2);
    }
    p.parts = int32_t(parts);
    return {unsigned(size), unsigned(slabs * parts)};
}

}  // namespace kda

namespace {

using namespace kda;

// ------------------------------------------------------------- decoding step
// h <- a h + c x for one token of every request: a thread takes two vectors of VEC channels of one request, all loaded before
// the first is worked on.  Bound by the state's traffic.  In a graph, BF16, 256 and 1024 requests of 8192 channels: 6.2 and
// 19.5 us (floors 4.3 and 17.3) with vectors of four, 6.5 and 20.4 by one vector to a thread, 9.1 and 34.0 by one of two
// channels; 256 of 2305 in FP32 4.1 us, 5.3 by one channel to a thread.  One request takes the launch's 1.2 us.
struct StepParams {
    const void *x, *g;
    int64_t ldx, ldg;
    void *y;
    float *state;
    const int32_t *slots;
    int32_t num_slots, D, form, blocks;                     // blocks to a request
};
constexpr int STEP_THREADS = 128, STEP_TIMES = 2;

template <typename T, typename G, int VEC>
__global__ void __launch_bounds__(STEP_THREADS) kda_gated_step_kernel(const StepParams p) {
    const int n = int(blockIdx.x / unsigned(p.blocks));
    const int col = (int(blockIdx.x % unsigned(p.blocks)) * STEP_TIMES * STEP_THREADS + int(threadIdx.x)) * VEC;
    pdl_launch_dependents();
    pdl_wait();
    int entry = n;
    if (p.slots != nullptr) {
        entry = p.slots[n];
        if (entry >= p.num_slots) entry = -1;
    }
    const T *const x = static_cast<const T *>(p.x) + n * p.ldx;
    const G *const g = static_cast<const G *>(p.g) + n * p.ldg;
    raw_t<T, VEC> xr[STEP_TIMES];
    raw_t<G, VEC> gr[STEP_TIMES];
    raw_t<float, VEC> hr[STEP_TIMES] = {};
#pragma unroll
    for (int i = 0; i < STEP_TIMES; ++i) {
        const int c = col + i * STEP_THREADS * VEC;
        if (c >= p.D) break;
        xr[i] = load_once<T, VEC>(x + c);
        gr[i] = load_once<G, VEC>(g + c);
        if (entry >= 0) hr[i] = *reinterpret_cast<const raw_t<float, VEC> *>(p.state + int64_t(entry) * p.D + c);
    }
#pragma unroll
    for (int i = 0; i < STEP_TIMES; ++i) {
        const int c = col + i * STEP_THREADS * VEC;
        if (c >= p.D) break;
        float a[VEC], rest[VEC], b[VEC], h[VEC];
        widen<float, VEC>(hr[i], h);
        widen<T, VEC>(xr[i], b);
        widen<G, VEC>(gr[i], a);
        decays<sizeof(G) == 4, VEC>(p.form, a, rest);
        if (p.form & RECUR_COMPLEMENT) mul_to<VEC>(b, b, rest);
        fma_to<VEC>(h, a, h, b);
        if (entry >= 0) store_raw<float, VEC>(p.state + int64_t(entry) * p.D + c, narrow<float, VEC>(h));
        store_raw<T, VEC>(static_cast<T *>(p.y) + int64_t(n) * p.D + c, narrow<T, VEC>(h));
    }
}

template <typename T, typename G, int VEC>
cudaError_t launch_step_vec(StepParams p, int32_t N, cudaStream_t s) {
    constexpr int COLUMNS = STEP_THREADS * STEP_TIMES * VEC;
    p.blocks = (p.D + COLUMNS - 1) / COLUMNS;
    return launch_pdl(true, kda_gated_step_kernel<T, G, VEC>, unsigned(N) * unsigned(p.blocks), STEP_THREADS, 0, s, p);
}
template <typename T, typename G>
cudaError_t launch_step(const StepParams &p, int32_t N, int vec, cudaStream_t s) {
    return vec == 4   ? launch_step_vec<T, G, 4>(p, N, s)
           : vec == 2 ? launch_step_vec<T, G, 2>(p, N, s)
                      : launch_step_vec<T, G, 1>(p, N, s);
}

// ------------------------------------------------------------- checkpoints
struct CkptParams {
    const void *x;              // save: [rows, dim] at pitch ldx
    void *out;                  // load: [rows, dim]
    int64_t ldx, units;         // units: blocks of 32 elements
    int8_t *codes;
    uint8_t *exponents;
    int32_t dim, blocks;        // blocks of a row
};
constexpr int CKPT_THREADS = 256;

// The exponent byte of a block whose largest magnitude has these bits: 127 2^e = 1.984375 2^(e + 6).
__device__ __forceinline__ unsigned ckpt_exponent(unsigned top) {
    const int e = int(top >> 23);
    if (e == 255) return CKPT_BAD;
    return unsigned(max(0, e - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0)));
}

// The code of x in a block of exponent byte e, whose inverse scale is given: x / 2^e + 1.5 2^23 has it in the low byte, rounded to
// nearest even by the addition.  (A block that is not finite has an inverse of 0 and codes that mean nothing.)
__device__ __forceinline__ unsigned ckpt_code(float x, float inverse) {
    return __float_as_uint(fmaf(x, inverse, 12582912.f));
}
// 64 2^e is past the type's largest finite value where e is the largest exponent that the type can have: values that would
// round to it are cut to 63 2^e before.
template <typename T>
__device__ __forceinline__ bool ckpt_top(unsigned e) {
    return e == (sizeof(T) == 2 && !std::is_same_v<T, __nv_bfloat16> ? 10 : 122) + 127;
}
__device__ __forceinline__ float ckpt_cut(float x, unsigned e) {
    const float most = 63.f * ckpt_scale(e);
    return fminf(fmaxf(x, -most), most);
}

// The bits of the largest magnitude of a vector, 16-bit types two at a time; and those of a value of the type as FP32.
template <typename T, int N>
__device__ __forceinline__ unsigned top_of(raw_t<T, N> raw) {
    constexpr int WORDS = N * int(sizeof(T)) / 4;
    unsigned w[WORDS];
    memcpy(w, &raw, sizeof(raw));
    unsigned top = w[0] & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < WORDS; ++i) {
        if constexpr (sizeof(T) == 4) top = max(top, w[i] & 0x7fffffffu);
        else top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    }
    return top;
}
template <typename T>
__device__ __forceinline__ unsigned top_join(unsigned a, unsigned b) {
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return __vmaxu2(a, b);
}
template <typename T>
__device__ __forceinline__ unsigned top_bits(unsigned top) {
    if constexpr (sizeof(T) == 4) {
        return top;
    } else {
        const unsigned short m = static_cast<unsigned short>(max(top & 0xffffu, top >> 16));
        T v;
        memcpy(&v, &m, 2);
        return __float_as_uint(widen_one(v)) & 0x7fffffffu;
    }
}

// Rows of whole blocks, in vectors of 16 bytes of the type (and as many codes): 4 or 8 threads to a block of 32, four vectors to
// a thread at once.  Bound by HBM and, for saving, by issue beside it: 8192 x 8192 BF16 are saved in 34 us (floor 30; 47 with
// conversions to integers in place of ckpt_code) and read back in 31.
template <typename T>
struct CkptVec {
    static constexpr int N = 16 / int(sizeof(T)), LANES = CKPT_BLOCK / N, BATCH = 4;
};

// FLAT: the rows follow one another without a gap.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(CKPT_THREADS) kda_checkpoint_save_kernel(const CkptParams p) {
    using V = CkptVec<T>;
    const int64_t vectors = p.units * V::LANES, step = int64_t(gridDim.x) * CKPT_THREADS;
    const unsigned per_row = unsigned(p.blocks) * V::LANES;
    pdl_launch_dependents();
    pdl_wait();
    raw_t<T, V::N> next[V::BATCH];
    auto fetch = [&](int64_t base) {
#pragma unroll
        for (int i = 0; i < V::BATCH; ++i) {
            const int64_t v = base + i * step + threadIdx.x;
            if (v >= vectors) continue;
            const int64_t at = FLAT ? v * V::N : v / per_row * p.ldx + v % per_row * V::N;
            next[i] = load_once<T, V::N>(static_cast<const T *>(p.x) + at);
        }
    };
    fetch(int64_t(blockIdx.x) * CKPT_THREADS);
    // whole warps leave the loop together: vectors is a multiple of the lanes to a block, not of a warp
    for (int64_t base = int64_t(blockIdx.x) * CKPT_THREADS; base < vectors; base += V::BATCH * step) {
        raw_t<T, V::N> raw[V::BATCH];
#pragma unroll
        for (int i = 0; i < V::BATCH; ++i) raw[i] = next[i];
        fetch(base + V::BATCH * step);
#pragma unroll
        for (int i = 0; i < V::BATCH; ++i) {
            const int64_t v = base + i * step + threadIdx.x;
            if (base + i * step >= vectors) break;
            unsigned top = v < vectors ? top_of<T, V::N>(raw[i]) : 0u;
#pragma unroll
            for (int o = V::LANES / 2; o > 0; o >>= 1) top = top_join<T>(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (v >= vectors) continue;
            const unsigned e = ckpt_exponent(top_bits<T>(top));
            const float inverse = __uint_as_float(e == CKPT_BAD ? 0u : (254u - e) << 23);
            float x[V::N];
            widen<T, V::N>(raw[i], x);
            if (__builtin_expect(ckpt_top<T>(e), 0)) {
#pragma unroll
                for (int n = 0; n < V::N; ++n) x[n] = ckpt_cut(x[n], e);
            }
            unsigned w[V::N / 4];
#pragma unroll
            for (int n = 0; n < V::N; n += 4) {
                const unsigned lo = __byte_perm(ckpt_code(x[n], inverse), ckpt_code(x[n + 1], inverse), 0x0040);
                const unsigned hi = __byte_perm(ckpt_code(x[n + 2], inverse), ckpt_code(x[n + 3], inverse), 0x0040);
                w[n / 4] = __byte_perm(lo, hi, 0x5410);
            }
            raw_t<int8_t, V::N> out;
            memcpy(&out, w, sizeof(out));
            store_raw<int8_t, V::N>(p.codes + v * V::N, out);
            if (threadIdx.x % V::LANES == 0) p.exponents[v / V::LANES] = uint8_t(e);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(CKPT_THREADS) kda_checkpoint_load_kernel(const CkptParams p) {
    using V = CkptVec<T>;
    const int64_t vectors = p.units * V::LANES, step = int64_t(gridDim.x) * CKPT_THREADS;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t base = int64_t(blockIdx.x) * CKPT_THREADS + threadIdx.x; base < vectors; base += V::BATCH * step) {
        raw_t<int8_t, V::N> raw[V::BATCH];
        unsigned e[V::BATCH];
#pragma unroll
        for (int i = 0; i < V::BATCH; ++i) {
            const int64_t v = base + i * step;
            if (v >= vectors) continue;
            raw[i] = load_once<int8_t, V::N>(p.codes + v * V::N);
            e[i] = p.exponents[v / V::LANES];
        }
#pragma unroll
        for (int i = 0; i < V::BATCH; ++i) {
            const int64_t v = base + i * step;
            if (v >= vectors) break;
            float x[V::N];
            code_values<V::N>(raw[i], ckpt_scale(e[i]), x);
            store_raw<T, V::N>(static_cast<T *>(p.out) + v * V::N, narrow<T, V::N>(x));
        }
    }
}

// Any width and alignment: a warp takes eight blocks of 32 of a row, single elements, four neighbours to a lane, all loaded
// before the first is packed.  Bound by issue: 8192 x 2305 are saved in 20 us (BF16; floor 8) and 23 (FP32; 14), and read
// back in 25 and 23; by one element to a lane 57 and 63, 45 and 48.
constexpr int CKPT_ANY = 2;                                 // times four blocks of a warp

template <typename T>
__global__ void __launch_bounds__(CKPT_THREADS) kda_checkpoint_save_any_kernel(const CkptParams p) {
    const int lane = threadIdx.x & 31, spans = (p.blocks + 4 * CKPT_ANY - 1) / (4 * CKPT_ANY);
    const int64_t rows = p.units / p.blocks, items = rows * spans;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t item = int64_t(blockIdx.x) * (CKPT_THREADS / 32) + int(threadIdx.x >> 5); item < items;
         item += int64_t(gridDim.x) * (CKPT_THREADS / 32)) {
        const int64_t row = item / spans;
        const int first = int(item - row * spans) * (4 * CKPT_ANY * CKPT_BLOCK) + lane * 4;   // the lane's first column
        const T *const from = static_cast<const T *>(p.x) + row * p.ldx;
        int8_t *const to = p.codes + row * p.dim;
        float x[CKPT_ANY][4];
#pragma unroll
        for (int i = 0; i < CKPT_ANY; ++i) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int col = first + i * 4 * CKPT_BLOCK + n;
                x[i][n] = col < p.dim ? widen_one(from[col]) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < CKPT_ANY; ++i) {
            const int col = first + i * 4 * CKPT_BLOCK;
            unsigned top = 0;
#pragma unroll
            for (int n = 0; n < 4; ++n) top = max(top, __float_as_uint(x[i][n]) & 0x7fffffffu);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const unsigned e = ckpt_exponent(top);
            const float inverse = __uint_as_float(e == CKPT_BAD ? 0u : (254u - e) << 23);
            if (ckpt_top<T>(e)) {
#pragma unroll
                for (int n = 0; n < 4; ++n) x[i][n] = ckpt_cut(x[i][n], e);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (col + n < p.dim) to[col + n] = int8_t(ckpt_code(x[i][n], inverse) & 0xffu);
            if (lane % 8 == 0 && col < p.dim) p.exponents[row * p.blocks + col / CKPT_BLOCK] = uint8_t(e);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(CKPT_THREADS) kda_checkpoint_load_any_kernel(const CkptParams p) {
    const int lane = threadIdx.x & 31, spans = (p.blocks + 4 * CKPT_ANY - 1) / (4 * CKPT_ANY);
    const int64_t rows = p.units / p.blocks, items = rows * spans;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t item = int64_t(blockIdx.x) * (CKPT_THREADS / 32) + int(threadIdx.x >> 5); item < items;
         item += int64_t(gridDim.x) * (CKPT_THREADS / 32)) {
        const int64_t row = item / spans;
        const int first = int(item - row * spans) * (4 * CKPT_ANY * CKPT_BLOCK) + lane * 4;
        const int8_t *const from = p.codes + row * p.dim;
        T *const to = static_cast<T *>(p.out) + row * p.dim;
        float x[CKPT_ANY][4];
        unsigned e[CKPT_ANY];
#pragma unroll
        for (int i = 0; i < CKPT_ANY; ++i) {
            const int col = first + i * 4 * CKPT_BLOCK;
            e[i] = col < p.dim ? p.exponents[row * p.blocks + col / CKPT_BLOCK] : 0u;
#pragma unroll
            for (int n = 0; n < 4; ++n) x[i][n] = col + n < p.dim ? float(from[col + n]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < CKPT_ANY; ++i) {
            const int col = first + i * 4 * CKPT_BLOCK;
            const float scale = ckpt_scale(e[i]);
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (col + n < p.dim) narrow_one(to[col + n], x[i][n] * scale);
        }
    }
}

template <typename T>
cudaError_t launch_checkpoint(const CkptParams &p, cudaStream_t s) {
    using V = CkptVec<T>;
    const bool save = p.out == nullptr;
    const void *x = save ? p.x : p.out;
    const bool wide = p.dim % CKPT_BLOCK == 0 && p.ldx % V::N == 0 && aligned16(x) &&
                      reinterpret_cast<uintptr_t>(p.codes) % V::N == 0;
    const int64_t per = wide ? int64_t(CKPT_THREADS) * V::BATCH / V::LANES : CKPT_THREADS / 32 * 4 * CKPT_ANY;   // units to a block of threads
    // saving: four blocks to an SM, all at once, their next vectors on the way; reading back: a block to its vectors
    const int64_t need = (p.units + per - 1) / per, most = !wide ? 152 * 8 : save ? 152 * 4 : int64_t(1) << 30;
    const unsigned grid = unsigned(need < most ? need : most);
    if (wide && save)
        return p.ldx == p.dim ? launch_pdl(true, kda_checkpoint_save_kernel<T, true>, grid, CKPT_THREADS, 0, s, p)
                              : launch_pdl(true, kda_checkpoint_save_kernel<T, false>, grid, CKPT_THREADS, 0, s, p);
    if (wide) return launch_pdl(true, kda_checkpoint_load_kernel<T>, grid, CKPT_THREADS, 0, s, p);
    return save ? launch_pdl(true, kda_checkpoint_save_any_kernel<T>, grid, CKPT_THREADS, 0, s, p)
                : launch_pdl(true, kda_checkpoint_load_any_kernel<T>, grid, CKPT_THREADS, 0, s, p);
}

// ------------------------------------------------------------------- checks
// Types, forms and widths that all entries of the recurrence share.
kda_status_t check_form(int32_t D, int32_t dtype, int32_t g_dtype, int32_t decay, int32_t complement) {
    if (!dtype_ok(dtype) || (g_dtype != dtype && g_dtype != KDA_F32)) return KDA_ERR_UNSUPPORTED;
    if (decay != KDA_DECAY_LOG && decay != KDA_DECAY_SIGMOID) return KDA_ERR_INVALID_ARGUMENT;
    if (complement != 0 && complement != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (D < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (D > KDA_RECUR_MAX_DIM) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t check_stream(const int32_t *cu, int32_t num_seqs, int64_t B, int64_t T) {
    if (B < 0 || T < 0 || num_seqs < 0) return KDA_ERR_INVALID_ARGUMENT;
    if ((cu != nullptr) != (num_seqs > 0)) return KDA_ERR_INVALID_ARGUMENT;
    if (cu != nullptr && (B != 1 || !aligned_to(cu, 4))) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t limit = (int64_t(1) << 31) - (int64_t(1) << 16);
    if (B >= (int64_t(1) << 30) || num_seqs >= (1 << 30) || T >= limit || (T > 0 && B > (limit - 1) / T))
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

int form_bits(int32_t decay, int32_t complement) {
    return (decay == KDA_DECAY_SIGMOID ? RECUR_SIGMOID : 0) | (complement ? RECUR_COMPLEMENT : 0);
}

// A tensor of rows that the lanes read or write: its pitch and its elements' size.
struct RowTensor {
    const void *at;
    int64_t ld;
    size_t es;
};
// Whether all of them fit vectors of `bytes_of(es)` bytes.
template <size_t N, typename F>
bool vectors_fit(const RowTensor (&tensors)[N], int32_t D, F bytes_of) {
    for (const RowTensor &t : tensors)
        if (t.at != nullptr && (!aligned_to(t.at, bytes_of(t.es)) || size_t(t.ld) * t.es % bytes_of(t.es) != 0 ||
                                size_t(D) * t.es % bytes_of(t.es) != 0))
            return false;
    return true;
}

}  // namespace

extern "C" {

kda_status_t kda_gated_scan(const void *x, int64_t ldx, const void *g, int64_t ldg, void *y, const float *state_in,
                            float *state_out, const int32_t *slots, int32_t num_slots, float *chunk_states,
                            const int32_t *cu_seqlens, int32_t num_seqs, int64_t B, int64_t T, int32_t D, int32_t dtype,
                            int32_t g_dtype, int32_t decay, int32_t complement, void *stream) {
    kda_status_t st = check_form(D, dtype, g_dtype, decay, complement);
    if (st == KDA_OK) st = check_stream(cu_seqlens, num_seqs, B, T);
    if (st != KDA_OK) return st;
    if (slots != nullptr && num_slots < 0) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t seqs = cu_seqlens != nullptr ? num_seqs : B, rows = B * T;
    if (seqs == 0) return KDA_OK;
    const size_t es = size_t(elt_size(dtype)), gs = size_t(elt_size(g_dtype));
    if (rows > 0 && (x == nullptr || g == nullptr || y == nullptr || ldx < D || ldg < D)) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(x, es) || !aligned_to(g, gs) || !aligned_to(y, es) || !aligned_to(state_in, 4) ||
        !aligned_to(state_out, 4) || !aligned_to(chunk_states, 4) || !aligned_to(slots, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t entries = slots != nullptr ? num_slots : seqs;
    const Span xs = rows_span(x, rows, ldx, D, es), gsp = rows_span(g, rows, ldg, D, gs), ys = rows_span(y, rows, D, D, es);
    const Span chunk = rows_span(chunk_states, (rows + RECUR_CHUNK - 1) / RECUR_CHUNK, D, D, 4);
    const Span in_state = rows_span(state_in, entries, D, D, 4), out_state = rows_span(state_out, entries, D, D, 4);
    const Span in[] = {xs, gsp, {slots, size_t(seqs) * 4}, {cu_seqlens, size_t(seqs + 1) * 4},
                       state_in != state_out ? in_state : Span{nullptr, 0}};
    const Span out[] = {ys, chunk, out_state};
    if (any_meet(out, in) || meet(ys, in_state) || meet(chunk, in_state)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows == 0 && state_out == nullptr) return KDA_OK;
    RecurParams p{};
    p.x = x; p.g = g; p.ldx = ldx; p.ldg = ldg; p.cu = cu_seqlens; p.nseq = int32_t(seqs); p.T = int32_t(T);
    p.rows = int32_t(rows); p.D = D; p.form = form_bits(decay, complement);
    p.y = y; p.state_in = state_in; p.state_out = state_out; p.slots = slots; p.num_slots = num_slots;
    p.chunk = chunk_states;
    RecurLaunch l{};
    l.wide_g = g_dtype == KDA_F32;
    const RowTensor rowed[] = {{x, ldx, es}, {g, ldg, gs}, {y, D, es}, {state_in, D, 4}, {state_out, D, 4}, {chunk_states, D, 4}};
    const RowTensor inputs[] = {rowed[0], rowed[1]};
    l.staged = vectors_fit(rowed, D, [](size_t n) { return 2 * n; }) && vectors_fit(inputs, D, [](size_t) { return size_t(16); });
    l.walk_wide = l.staged ? 8 / int(es) : 0;
    l.walk_fit = vectors_fit(rowed, D, [](size_t n) { return 4 * n; }) ? 4 : 2;
    DeviceInfo info;
    if (cudaGetDevice(&l.device) != cudaSuccess || device_info(l.device, info) != cudaSuccess) return KDA_ERR_CUDA;
    p.err = info.err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KDA_F32    ? launch_scan_f32(p, l, s)
                          : dtype == KDA_BF16 ? launch_scan_bf16(p, l, s)
                                              : launch_scan_f16(p, l, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_gated_scan_backward(const void *dy, int64_t lddy, const void *x, const uint8_t *x_exponents,
                                     int64_t ldx, const void *g, const uint8_t *g_exponents, int64_t ldg,
                                     const float *chunk_states, const float *state_in, const float *dstate_out,
                                     void *dx, void *dg, float *dstate_in, const int32_t *cu_seqlens,
                                     int32_t num_seqs, int64_t B, int64_t T, int32_t D, int32_t dtype, int32_t g_dtype,
                                     int32_t decay, int32_t complement, void *stream) {
    kda_status_t st = check_form(D, dtype, g_dtype, decay, complement);
    if (st == KDA_OK) st = check_stream(cu_seqlens, num_seqs, B, T);
    if (st != KDA_OK) return st;
    const int64_t seqs = cu_seqlens != nullptr ? num_seqs : B, rows = B * T, blocks = (D + CKPT_BLOCK - 1) / CKPT_BLOCK;
    if (seqs == 0) return KDA_OK;
    const bool x8 = x_exponents != nullptr, g8 = g_exponents != nullptr;
    const size_t es = size_t(elt_size(dtype)), gs = size_t(elt_size(g_dtype)), xin = x8 ? 1 : es, gin = g8 ? 1 : gs;
    if (rows > 0 && (dy == nullptr || x == nullptr || g == nullptr || chunk_states == nullptr || dx == nullptr ||
                     dg == nullptr || lddy < D || ldx < D || ldg < D))
        return KDA_ERR_INVALID_ARGUMENT;
    if (rows > 0 && ((x8 && ldx != D) || (g8 && ldg != D))) return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(dy, es) || !aligned_to(x, xin) || !aligned_to(g, gin) || !aligned_to(dx, es) || !aligned_to(dg, gs) ||
        !aligned_to(chunk_states, 4) || !aligned_to(state_in, 4) || !aligned_to(dstate_out, 4) || !aligned_to(dstate_in, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const Span dys = rows_span(dy, rows, lddy, D, es), xs = rows_span(x, rows, ldx, D, xin);
    const Span gsp = rows_span(g, rows, ldg, D, gin), dxs = rows_span(dx, rows, D, D, es), dgs = rows_span(dg, rows, D, D, gs);
    const Span chunk = rows_span(chunk_states, (rows + RECUR_CHUNK - 1) / RECUR_CHUNK, D, D, 4);
    const Span first = rows_span(state_in, seqs, D, D, 4), last = rows_span(dstate_out, seqs, D, D, 4);
    const Span dfirst = rows_span(dstate_in, seqs, D, D, 4);
    const Span in[] = {dys, xs, gsp, chunk, first, last, rows_span(x_exponents, rows, blocks, blocks, 1),
                       rows_span(g_exponents, rows, blocks, blocks, 1), {cu_seqlens, size_t(seqs + 1) * 4}};
    const Span out[] = {dxs, dgs, dfirst};
    if (any_meet(out, in)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows == 0 && dstate_in == nullptr) return KDA_OK;
    RecurParams p{};
    p.x = x; p.g = g; p.xe = x_exponents; p.ge = g_exponents; p.ldx = ldx; p.ldg = ldg; p.cu = cu_seqlens;
    p.nseq = int32_t(seqs); p.T = int32_t(T); p.rows = int32_t(rows); p.D = D; p.form = form_bits(decay, complement);
    p.state_in = state_in; p.chunk = const_cast<float *>(chunk_states);
    p.dy = dy; p.lddy = lddy; p.dfinal = dstate_out; p.dx = dx; p.dg = dg; p.dinitial = dstate_in;
    RecurLaunch l{};
    l.wide_g = g_dtype == KDA_F32; l.x8 = x8; l.g8 = g8;
    const RowTensor rowed[] = {{dy, lddy, es}, {x, ldx, xin}, {g, ldg, gin}, {dx, D, es}, {dg, D, gs}, {chunk_states, D, 4},
                               {state_in, D, 4}, {dstate_out, D, 4}, {dstate_in, D, 4}};
    const RowTensor inputs[] = {rowed[0], rowed[1], rowed[2]};
    l.staged = vectors_fit(rowed, D, [](size_t n) { return 2 * n; }) && vectors_fit(inputs, D, [](size_t) { return size_t(16); });
    DeviceInfo info;
    if (cudaGetDevice(&l.device) != cudaSuccess || device_info(l.device, info) != cudaSuccess) return KDA_ERR_CUDA;
    p.err = info.err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KDA_F32    ? launch_scan_backward_f32(p, l, s)
                          : dtype == KDA_BF16 ? launch_scan_backward_bf16(p, l, s)
                                              : launch_scan_backward_f16(p, l, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_gated_step(const void *x, int64_t ldx, const void *g, int64_t ldg, void *y, float *state,
                            const int32_t *slots, int32_t num_slots, int32_t N, int32_t D, int32_t dtype,
                            int32_t g_dtype, int32_t decay, int32_t complement, void *stream) {
    const kda_status_t st = check_form(D, dtype, g_dtype, decay, complement);
    if (st != KDA_OK) return st;
    if (N < 0 || num_slots < 0 || (slots == nullptr && num_slots < N)) return KDA_ERR_INVALID_ARGUMENT;
    if (int64_t(N) * ((D + 255) / 256) >= (int64_t(1) << 30)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    const size_t es = size_t(elt_size(dtype)), gs = size_t(elt_size(g_dtype));
    if (x == nullptr || g == nullptr || y == nullptr || (state == nullptr && num_slots > 0) || ldx < D || ldg < D)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(x, es) || !aligned_to(g, gs) || !aligned_to(y, es) || !aligned_to(state, 4) || !aligned_to(slots, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const Span xs = rows_span(x, N, ldx, D, es), gsp = rows_span(g, N, ldg, D, gs), ys = rows_span(y, N, D, D, es);
    const Span pool = rows_span(state, num_slots, D, D, 4);
    const Span in[] = {xs, gsp, {slots, size_t(N) * 4}}, out[] = {ys, pool};
    if (any_meet(out, in)) return KDA_ERR_INVALID_ARGUMENT;
    const StepParams p{x, g, ldx, ldg, y, state, slots, num_slots, D, form_bits(decay, complement), 0};
    const RowTensor rowed[] = {{x, ldx, es}, {g, ldg, gs}, {y, D, es}, {state, D, 4}};
    const int vec = vectors_fit(rowed, D, [](size_t n) { return 4 * n; })   ? 4
                    : vectors_fit(rowed, D, [](size_t n) { return 2 * n; }) ? 2
                                                                            : 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == KDA_F32) e = launch_step<float, float>(p, N, vec, s);
    else if (dtype == KDA_BF16)
        e = g_dtype == KDA_F32 ? launch_step<__nv_bfloat16, float>(p, N, vec, s)
                               : launch_step<__nv_bfloat16, __nv_bfloat16>(p, N, vec, s);
    else e = g_dtype == KDA_F32 ? launch_step<__half, float>(p, N, vec, s) : launch_step<__half, __half>(p, N, vec, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Checks and launch of both directions; x at pitch ldx is read (save) or written (load, ldx = dim).
static kda_status_t run_checkpoint(bool save, void *x, int64_t ldx, int8_t *codes, uint8_t *exponents, int64_t rows,
                                   int32_t dim, int32_t dtype, void *stream) {
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if (rows < 0 || dim < 1) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t blocks = (dim + CKPT_BLOCK - 1) / CKPT_BLOCK;
    if (dim > KDA_RECUR_MAX_DIM || rows >= (int64_t(1) << 36) / blocks) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    const size_t es = size_t(elt_size(dtype));
    if (x == nullptr || codes == nullptr || exponents == nullptr || ldx < dim || !aligned_to(x, es))
        return KDA_ERR_INVALID_ARGUMENT;
    const Span xs = rows_span(x, rows, ldx, dim, es), cs{codes, size_t(rows) * size_t(dim)};
    const Span ex{exponents, size_t(rows) * size_t(blocks)};
    if (meet(xs, cs) || meet(xs, ex) || meet(cs, ex)) return KDA_ERR_INVALID_ARGUMENT;
    const CkptParams p{x, save ? nullptr : x, ldx, rows * blocks, codes, exponents, dim, int32_t(blocks)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KDA_F32    ? launch_checkpoint<float>(p, s)
                          : dtype == KDA_BF16 ? launch_checkpoint<__nv_bfloat16>(p, s)
                                              : launch_checkpoint<__half>(p, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_checkpoint_save(const void *x, int64_t ldx, int8_t *codes, uint8_t *exponents, int64_t rows,
                                 int32_t dim, int32_t dtype, void *stream) {
    return run_checkpoint(true, const_cast<void *>(x), ldx, codes, exponents, rows, dim, dtype, stream);
}

kda_status_t kda_checkpoint_load(const int8_t *codes, const uint8_t *exponents, void *x, int64_t rows, int32_t dim,
                                 int32_t dtype, void *stream) {
    return run_checkpoint(false, x, dim, const_cast<int8_t *>(codes), const_cast<uint8_t *>(exponents), rows, dim, dtype,
                          stream);
}

}  // extern "C"
