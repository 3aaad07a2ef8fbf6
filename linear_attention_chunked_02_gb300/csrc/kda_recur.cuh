// kda_recur.cuh -- the gated linear recurrence over whole sequences, and its gradients.
//
// Every channel keeps a state h; with its decay a and its input's factor c (1 or 1 - a),
//
//     h_t = a_t h_{t-1} + c_t x_t,   y_t = h_t.
//
// The sequences lie one after the other in a stream of rows.  A row maps the state before it to the
// state after it, h -> A h + H, and so does any run of rows; a sequence's first row maps everything
// to one state.  A block takes 32 lanes' channels of one part of the stream, tile by tile: each of
// its warps takes R consecutive rows of the tile into registers, works out their map, and all warps
// chain the maps of those before them (shared memory) to the state that their rows start from;
// then they walk their rows once more for the outputs.  So every input is read once.
//
// The gradients run backwards: with d_t the gradient of h_t and e_t = a_t d_t what it hands on,
//
//     d_t = dy_t + e_{t+1};   dx = c d;   da = d (h_{t-1} - [c = 1 - a] x);   dg = da a  or  da a (1 - a)
//
// and h_{t-1} comes again from the state that the forward pass left before every 64 rows: the
// tile's rows are chained forwards for h and backwards for e with one exchange.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>

#include "kda_kernels.cuh"
#include "kda_vec.cuh"

namespace kda {

constexpr int RECUR_CHUNK = 64;               // rows to a chunk state
constexpr int RECUR_SIGMOID = 1, RECUR_COMPLEMENT = 2;   // bits of RecurParams::form

struct RecurParams {
    const void *x, *g;          // [rows, D] at pitches ldx and ldg; int8 codes at pitch D
    const uint8_t *xe, *ge;     // exponents of codes [rows, ceil(D / 32)]
    int64_t ldx, ldg;
    const int32_t *cu;          // packed: cu_seqlens; dense: nullptr
    int32_t nseq;               // sequences (dense: batch rows)
    int32_t T;                  // dense: rows to a sequence; packed: all rows
    int32_t rows, D;
    int32_t form;
    int32_t part;               // rows of the stream whose sequences a block takes (dense: a multiple of T)
    // forward
    void *y;                    // [rows, D]
    const float *state_in;      // [entries, D] or nullptr; backward: [sequences, D]
    float *state_out;           // likewise
    const int32_t *slots;       // [sequences] or nullptr
    int32_t num_slots;
    float *chunk;               // [ceil(rows / 64), D]; forward: may be nullptr, is written; backward: is read
    // backward
    const void *dy;             // [rows, D] at pitch lddy
    int64_t lddy;
    const float *dfinal;        // [sequences, D] or nullptr
    void *dx, *dg;              // [rows, D]
    float *dinitial;            // [sequences, D] or nullptr
};

// Entries of cu[0 .. n) that are at most `row`, found by the whole warp.  Any contents give a count in [0, n].
__device__ __forceinline__ int count_until(const int32_t *cu, int n, int row, int lane) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo + 31) >> 5, at = lo + step * (lane + 1) - 1;
        const int k = __popc(__ballot_sync(0xffffffffu, at < hi && cu[at] <= row));
        const int next = lo + step * (k + 1) - 1;          // the first probe past `row`, if it is one
        lo = min(lo + step * k, hi);
        hi = max(lo, min(hi, next));
    }
    return lo;
}

// The rows [begin, end) of this block's sequences: those that start in its part of the stream.
__device__ __forceinline__ void part_rows(const RecurParams &p, int part, int parts, int lane, int &begin, int &end) {
    const int64_t from = int64_t(part) * p.part, to = from + p.part;
    if (p.cu == nullptr) {
        begin = int(from < p.rows ? from : p.rows);
        end = int(to < p.rows ? to : p.rows);
        return;
    }
    auto first_from = [&](int64_t row) {
        const int i = count_until(p.cu, p.nseq + 1, row > INT_MAX ? INT_MAX : int(row) - 1, lane);
        return i <= p.nseq ? p.cu[i] : p.cu[p.nseq];
    };
    begin = min(max(first_from(from), 0), p.rows);
    end = part + 1 < parts ? first_from(to) : p.cu[p.nseq];
    end = min(max(end, begin), p.rows);
}

// What a warp knows of its R rows: which are its block's, which begin a sequence, which end one.
struct Rows {
    int row0, first, bound;     // first: boundary number `lane` is entry first + lane of cu
    unsigned live, starts, lasts;
};

template <int R>
__device__ __forceinline__ Rows look_at(const RecurParams &p, int row0, int begin, int end, int lane) {
    Rows r{row0, 0, INT_MAX, 0, 0, 0};
    const int lo = max(begin - row0, 0), hi = min(end - row0, R);
    if (hi <= lo) return r;
    r.live = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    unsigned s;                                            // bits 0 .. R
    if (p.cu == nullptr) {
        s = __ballot_sync(0xffffffffu, lane <= R && unsigned(row0 + lane) % unsigned(p.T) == 0);
    } else {
        r.first = count_until(p.cu, p.nseq + 1, row0 - 1, lane);
        int at = r.first + lane;
        r.bound = at <= p.nseq ? p.cu[at] : INT_MAX;
        unsigned bits = 0;
        for (int v = r.bound;;) {
            const int d = v - row0;
            if (d >= 0 && d <= R) bits |= 1u << d;
            if (__shfl_sync(0xffffffffu, v, 31) > row0 + R) break;
            at += 32;                                      // only where sequences are empty
            v = at <= p.nseq ? p.cu[at] : INT_MAX;
        }
        s = __reduce_or_sync(0xffffffffu, bits);
    }
    r.starts = s & r.live;
    r.lasts = s >> 1;
    if (end - 1 - row0 < R) r.lasts |= 1u << (end - 1 - row0);
    r.lasts &= r.live;
    return r;
}

// The sequence that `row` belongs to, for one of the warp's live rows; all lanes call it.
__device__ __forceinline__ int sequence_of(const RecurParams &p, const Rows &r, int row, int lane) {
    if (p.cu == nullptr) return row / p.T;
    const int k = __popc(__ballot_sync(0xffffffffu, r.bound <= row));
    return (k < 32 ? r.first + k : count_until(p.cu, p.nseq + 1, row, lane)) - 1;
}

// State entry of sequence n, or -1 for none.
__device__ __forceinline__ int recur_entry(const RecurParams &p, int n) {
    if (n < 0 || n >= p.nseq) return -1;                   // malformed cu_seqlens
    if (p.slots == nullptr) return n;
    const int s = p.slots[n];
    return s >= 0 && s < p.num_slots ? s : -1;
}

template <int VEC>
__device__ __forceinline__ void load_state(float (&h)[VEC], const float *base, int entry, int D, int col) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = 0.f;
    if (base == nullptr || entry < 0 || col >= D) return;
    widen<float, VEC>(*reinterpret_cast<const raw_t<float, VEC> *>(base + int64_t(entry) * D + col), h);
}
template <int VEC>
__device__ __forceinline__ void store_state(const float (&h)[VEC], float *base, int64_t entry, int D, int col) {
    if (base == nullptr || entry < 0 || col >= D) return;
    store_raw<float, VEC>(base + entry * D + col, narrow<float, VEC>(h));
}

// a and 1 - a from the sigmoid's argument, both without cancellation: with z = exp(-|g|), 1 / (1 + z) is the larger.
// The quotient is the approximate reciprocal with one Newton step, since a decay's relative error
// counts as often as the state remembers tokens.
__device__ __forceinline__ void sigmoid_pair(float g, float &a, float &rest) {
    const float z = expf(-fabsf(g)), d = 1.f + z;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = fmaf(r, fmaf(-d, r, 1.f), r);
    const float s = z * r;
    a = g >= 0.f ? r : s;
    rest = g >= 0.f ? s : r;
    if (g != g) a = rest = g;
}

// The decays a of N values g and, where the form asks for it, 1 - a (else 1).  Log decays take the exponential of
// full accuracy, for the reason above.
template <int N>
__device__ __forceinline__ void decays(int form, float (&g)[N], float (&rest)[N]) {
    if (form & RECUR_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a;
            sigmoid_pair(g[i], a, rest[i]);
            g[i] = a;
        }
    } else if (form & RECUR_COMPLEMENT) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            rest[i] = -expm1f(g[i]);
            g[i] = expf(g[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            rest[i] = 1.f;
            g[i] = expf(g[i]);
        }
    }
}

// States of empty sequences: `from` to `to`, zeros without `from`.  The warps of all blocks of these channels
// share the sequences.
template <int VEC>
__device__ __forceinline__ void copy_empty(const RecurParams &p, const float *from, float *to, int worker, int workers,
                                           int lane, int col) {
    if (to == nullptr || (from == to)) return;
    if (p.cu == nullptr && p.rows > 0) return;             // dense: none or all are empty
    for (int64_t n0 = int64_t(worker) * 32; n0 < p.nseq; n0 += int64_t(workers) * 32) {
        const int n = int(n0) + lane;
        unsigned empty = __ballot_sync(0xffffffffu, n < p.nseq && (p.cu == nullptr || p.cu[n + 1] <= p.cu[n]));
        for (; empty != 0; empty &= empty - 1) {
            const int e = recur_entry(p, int(n0) + __ffs(empty) - 1);
            float h[VEC];
            load_state<VEC>(h, from, e, p.D, col);
            store_state<VEC>(h, to, e, p.D, col);
        }
    }
}

// ------------------------------------------------------------------ forward
// Maps of the warps of a block, two tiles' worth: A and H of each lane's channels.
template <int VEC, int W>
struct MapsOf {
    float a[2][W][32][VEC], h[2][W][32][VEC];
    int set[2][W];                                          // whether the map is one state, whatever came before
};

template <typename T, typename G, int VEC, int R, int W>
__global__ void __launch_bounds__(W * 32) kda_gated_scan_kernel(const RecurParams p) {
    constexpr int TILE = R * W;
    static_assert(RECUR_CHUNK % R == 0 && R <= 16, "chunk states lie at warps' first rows");
    __shared__ MapsOf<VEC, W> maps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (int(blockIdx.x) * 32 + lane) * VEC, part = blockIdx.y, parts = gridDim.y;
    const bool in = col < p.D;
    pdl_launch_dependents();
    pdl_wait();
    int begin, end;
    part_rows(p, part, parts, lane, begin, end);
    const int tile0 = begin / TILE, tiles = end > begin ? (end - 1) / TILE + 1 - tile0 : 0;
    raw_t<T, VEC> xr[R];
    raw_t<G, VEC> gr[R];
    auto fetch = [&](int tile) {
        const int row0 = (tile0 + tile) * TILE + warp * R;
        const T *x = static_cast<const T *>(p.x) + row0 * p.ldx + col;
        const G *g = static_cast<const G *>(p.g) + row0 * p.ldg + col;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool live = in && tile < tiles && row0 + j >= begin && row0 + j < end;
            xr[j] = live ? load_once<T, VEC>(x + j * p.ldx) : raw_t<T, VEC>{};
            gr[j] = live ? load_once<G, VEC>(g + j * p.ldg) : raw_t<G, VEC>{};
        }
    };
    float carry[VEC] = {};
    fetch(0);
    for (int tile = 0; tile < tiles; ++tile) {
        const int row0 = (tile0 + tile) * TILE + warp * R, buf = tile & 1;
        float a[R][VEC], b[R][VEC];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float c[VEC];
            widen<T, VEC>(xr[j], b[j]);
            widen<G, VEC>(gr[j], a[j]);
            decays<VEC>(p.form, a[j], c);
            if (p.form & RECUR_COMPLEMENT) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) b[j][v] *= c[v];
            }
        }
        fetch(tile + 1);
        const Rows rows = look_at<R>(p, row0, begin, end, lane);
        float start[VEC] = {};                              // the state before the first row, where that starts a sequence
        if (rows.starts != 0) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (!(rows.starts >> j & 1u)) continue;
                float h[VEC];
                load_state<VEC>(h, p.state_in, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    b[j][v] = fmaf(a[j][v], h[v], b[j][v]);
                    if (j == 0) start[v] = h[v];
                }
            }
        }
        float A[VEC], H[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool starts = rows.starts >> j & 1u;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                H[v] = starts ? b[j][v] : fmaf(a[j][v], H[v], b[j][v]);
                A[v] *= a[j][v];
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            maps.a[buf][warp][lane][v] = A[v];
            maps.h[buf][warp][lane][v] = H[v];
        }
        if (lane == 0) maps.set[buf][warp] = rows.starts != 0;
        // two sets of maps: a warp writes the next tile's while others still read this one's, and the
        // one after that behind the next barrier
        __syncthreads();
        float h[VEC];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == warp) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = carry[v];
            }
            const bool set = maps.set[buf][w] != 0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float hw = maps.h[buf][w][lane][v];
                carry[v] = set ? hw : fmaf(maps.a[buf][w][lane][v], carry[v], hw);
            }
        }
        if (rows.live == 0) continue;
        if (p.chunk != nullptr && row0 % RECUR_CHUNK == 0 && (rows.live & 1u))
            store_state<VEC>(rows.starts & 1u ? start : h, p.chunk, row0 / RECUR_CHUNK, p.D, col);
        T *y = static_cast<T *>(p.y) + int64_t(row0) * p.D + col;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool starts = rows.starts >> j & 1u;
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = starts ? b[j][v] : fmaf(a[j][v], h[v], b[j][v]);
            if (in && (rows.live >> j & 1u)) store_raw<T, VEC>(y + int64_t(j) * p.D, narrow<T, VEC>(h));
            if (rows.lasts >> j & 1u)
                store_state<VEC>(h, p.state_out, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
        }
    }
    copy_empty<VEC>(p, p.state_in, p.state_out, part * W + warp, parts * W, lane, col);
}

// ----------------------------------------------------------------- backward
template <int VEC, int W>
struct GradMapsOf {
    float a[2][W][32][VEC], h[2][W][32][VEC], e[2][W][32][VEC];
    int set[2][W], cut[2][W];   // forwards: rows.starts != 0; backwards: rows.lasts != 0
};

// One row operand: T, or codes whose exponents are spread over the lanes (32 / R blocks to a warp's row at most).
template <typename S, int VEC, int R>
struct Source {
    raw_t<S, VEC> raw[R];
    unsigned scales = 0;        // codes: the exponent of row lane / VEC, block lane % VEC of the warp's columns

    // rows row0 .. row0 + R of [rows, D] at pitch ld; only those with their bit in `live`
    __device__ __forceinline__ void fetch(const void *base, const uint8_t *exps, int64_t ld, int row0, unsigned live,
                                          int D, int col, int lane) {
        const S *s = static_cast<const S *>(base) + row0 * ld + col;
#pragma unroll
        for (int j = 0; j < R; ++j)
            raw[j] = col < D && (live >> j & 1u) ? load_once<S, VEC>(s + j * ld) : raw_t<S, VEC>{};
        if constexpr (sizeof(S) == 1) {
            // 32 VEC columns are VEC blocks of 32; the warp's first column is a multiple of 32
            const int j = lane / VEC, block = (col - lane * VEC) / CKPT_BLOCK + lane % VEC;
            const int blocks = (D + CKPT_BLOCK - 1) / CKPT_BLOCK;
            scales = j < R && block < blocks && (live >> j & 1u) ? exps[int64_t(row0 + j) * blocks + block] : 0u;
        }
    }
    __device__ __forceinline__ void value(int j, float (&v)[VEC], int lane) const {
        widen<S, VEC>(raw[j], v);
        if constexpr (sizeof(S) == 1) {
            const float s = ckpt_scale(__shfl_sync(0xffffffffu, scales, j * VEC + lane * VEC / CKPT_BLOCK));
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] *= s;
        }
    }
};

__device__ __forceinline__ unsigned live_bits(int row0, int begin, int end, int R) {
    const int lo = max(begin - row0, 0), hi = min(end - row0, R);
    return hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}

// T: dy, dx; X, S: x and g, or int8_t for codes; G: dg.
template <typename T, typename X, typename S, typename G, int VEC, int R, int W>
__global__ void __launch_bounds__(W * 32) kda_gated_scan_backward_kernel(const RecurParams p) {
    constexpr int TILE = R * W;
    static_assert(TILE == RECUR_CHUNK && R * VEC <= 32, "a tile is a chunk");
    __shared__ GradMapsOf<VEC, W> maps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (int(blockIdx.x) * 32 + lane) * VEC, part = blockIdx.y, parts = gridDim.y;
    const bool in = col < p.D;
    pdl_launch_dependents();
    pdl_wait();
    int begin, end;
    part_rows(p, part, parts, lane, begin, end);
    const int tile0 = begin / TILE, tiles = end > begin ? (end - 1) / TILE + 1 - tile0 : 0;
    Source<X, VEC, R> xs;
    Source<S, VEC, R> gs;
    Source<T, VEC, R> ds;
    float chunk[VEC];
    auto fetch = [&](int tile) {                            // counted from the last
        const int t = tile0 + tiles - 1 - tile, row0 = t * TILE + warp * R;
        const unsigned live = tile < tiles ? live_bits(row0, begin, end, R) : 0u;
        xs.fetch(p.x, p.xe, p.ldx, row0, live, p.D, col, lane);
        gs.fetch(p.g, p.ge, p.ldg, row0, live, p.D, col, lane);
        ds.fetch(p.dy, nullptr, p.lddy, row0, live, p.D, col, lane);
        load_state<VEC>(chunk, p.chunk, warp == 0 && (live & 1u) ? t : -1, p.D, col);
    };
    float carry[VEC] = {};
    fetch(0);
    for (int tile = 0; tile < tiles; ++tile) {
        const int t = tile0 + tiles - 1 - tile, row0 = t * TILE + warp * R, buf = tile & 1;
        // x: in the end h before the row, less x where c = 1 - a
        float a[R][VEC], rest[R][VEC], x[R][VEC], d[R][VEC], h[VEC];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            xs.value(j, x[j], lane);
            gs.value(j, a[j], lane);
            ds.value(j, d[j], lane);
            decays<VEC>(p.form, a[j], rest[j]);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = chunk[v];
        fetch(tile + 1);
        const Rows rows = look_at<R>(p, row0, begin, end, lane);
        const bool complement = p.form & RECUR_COMPLEMENT;
        float A[VEC], H[VEC], E[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, H[v] = warp == 0 ? h[v] : 0.f, E[v] = 0.f;
        // forwards; a first row's state is looked up here and once more below, where it is in the cache
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (rows.starts >> j & 1u)
                load_state<VEC>(H, p.state_in, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                H[v] = fmaf(a[j][v], H[v], complement ? rest[j][v] * x[j][v] : x[j][v]);
                A[v] *= a[j][v];
            }
        }
        // backwards
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            if (rows.lasts >> j & 1u)
                load_state<VEC>(E, p.dfinal, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
#pragma unroll
            for (int v = 0; v < VEC; ++v) E[v] = a[j][v] * (d[j][v] + E[v]);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            maps.a[buf][warp][lane][v] = A[v];
            maps.h[buf][warp][lane][v] = H[v];
            maps.e[buf][warp][lane][v] = E[v];
        }
        if (lane == 0) maps.set[buf][warp] = warp == 0 || rows.starts != 0, maps.cut[buf][warp] = rows.lasts != 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            if (w >= warp) break;
            const bool set = maps.set[buf][w] != 0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float hw = maps.h[buf][w][lane][v];
                h[v] = set ? hw : fmaf(maps.a[buf][w][lane][v], h[v], hw);
            }
        }
        float e[VEC];
#pragma unroll
        for (int w = W - 1; w >= 0; --w) {
            if (w == warp) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) e[v] = carry[v];
            }
            const bool cut = maps.cut[buf][w] != 0;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float ew = maps.e[buf][w][lane][v];
                carry[v] = cut ? ew : fmaf(maps.a[buf][w][lane][v], carry[v], ew);
            }
        }
        if (rows.live == 0) continue;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (rows.starts >> j & 1u)
                load_state<VEC>(h, p.state_in, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float was = h[v];
                h[v] = fmaf(a[j][v], h[v], complement ? rest[j][v] * x[j][v] : x[j][v]);
                x[j][v] = complement ? was - x[j][v] : was;
            }
        }
        T *dx = static_cast<T *>(p.dx) + int64_t(row0) * p.D + col;
        G *dg = static_cast<G *>(p.dg) + int64_t(row0) * p.D + col;
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            if (rows.lasts >> j & 1u)
                load_state<VEC>(e, p.dfinal, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
            float ox[VEC], og[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float dh = d[j][v] + e[v];
                e[v] = a[j][v] * dh;
                ox[v] = complement ? rest[j][v] * dh : dh;
                og[v] = e[v] * x[j][v];
                if (p.form & RECUR_SIGMOID) og[v] *= rest[j][v];
            }
            if (in && (rows.live >> j & 1u)) {
                store_raw<T, VEC>(dx + int64_t(j) * p.D, narrow<T, VEC>(ox));
                store_raw<G, VEC>(dg + int64_t(j) * p.D, narrow<G, VEC>(og));
            }
            if (p.dinitial != nullptr && (rows.starts >> j & 1u))
                store_state<VEC>(e, p.dinitial, recur_entry(p, sequence_of(p, rows, row0 + j, lane)), p.D, col);
        }
    }
    copy_empty<VEC>(p, p.dfinal, p.dinitial, part * W + warp, parts * W, lane, col);
}

}  // namespace kda
