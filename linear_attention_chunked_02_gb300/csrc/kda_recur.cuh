// kda_recur.cuh -- the gated linear recurrence over whole sequences, and its gradients.
//
// Every channel keeps a state h; with its decay a and its input's factor c (1 or 1 - a),
//
//     h_t = a_t h_{t-1} + c_t x_t,   y_t = h_t.
//
// The sequences lie one after the other in a stream of rows.  A row maps the state before it to the
// state after it, h -> A h + H, and so does any run of rows; a sequence's first row maps everything
// to one state.  A cluster of blocks takes 32 lanes' channels of one part of the stream, tile after tile
// in turn: each warp takes R consecutive rows of its block's tile into registers and works out their map; the maps
// of the block's warps, and of the cluster's blocks, which go from one's shared memory to the others', are chained (by
// a warp of its own, in the gradients by a thread to a channel) to the state that every warp's rows start from; then
// the warps walk their rows once more for the outputs.  So every input is read once, and one long
// sequence of few channels still keeps many SMs busy.  The order of all sums is set by the shape alone.
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

#include <type_traits>

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
    int32_t slabs, parts;       // clusters are numbered by columns, then by parts of the stream
    int32_t part;               // rows of the stream whose sequences a cluster takes (dense: a multiple of T)
    int32_t solo_part;          // packed: where no sequence is longer than solo_most, every block takes a part of this many
    int32_t solo_most;          // rows by itself, cluster or not (0: never)
    int32_t walk_parts;         // forward, sequences walked by single warps: their parts of the stream, or 0 for never,
    int32_t walk_part;          // the parts' rows,
    int32_t walk_most;          // the longest sequence for which that is done,
    int32_t walk_wide;          // and whether a warp takes 8 bytes of x to a lane or 4
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
    unsigned *err;              // device error word
};

// How many of the numbers 0 .. n - 1 `holds` is true for, if it is true up to some number and false from there on; found by
// the whole warp.  Whatever holds() says, the answer is in [0, n].
template <typename F>
__device__ __forceinline__ int count_while(int n, int lane, F holds) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (hi - lo + 31) >> 5, at = lo + step * (lane + 1) - 1;
        const int k = __popc(__ballot_sync(0xffffffffu, at < hi && holds(at)));
        const int next = lo + step * (k + 1) - 1;          // the first probe that is false, if there is one
        lo = min(lo + step * k, hi);
        hi = max(lo, min(hi, next));
    }
    return lo;
}
// Entries of cu[0 .. n) that are at most `row`.
__device__ __forceinline__ int count_until(const int32_t *cu, int n, int row, int lane) {
    return count_while(n, lane, [&](int i) { return cu[i] <= row; });
}

// The rows [begin, end) of a part's sequences: those whose middle is in its `length` rows of the stream (their
// first rows would put two of equal lengths into one part where the length is rounded up).
__device__ __forceinline__ void part_rows(const RecurParams &p, int part, int parts, int length, int lane, int &begin, int &end) {
    const int64_t from = int64_t(part) * length, to = from + length;
    if (p.cu == nullptr) {
        begin = int(from < p.rows ? from : p.rows);
        end = int(to < p.rows ? to : p.rows);
        return;
    }
    auto first_from = [&](int64_t row) {
        return p.cu[count_while(p.nseq, lane, [&](int n) { return int64_t(p.cu[n]) + p.cu[n + 1] < 2 * row; })];
    };
    begin = min(max(part > 0 ? first_from(from) : p.cu[0], 0), p.rows);
    end = part + 1 < parts ? first_from(to) : p.cu[p.nseq];
    end = min(max(end, begin), p.rows);
}

// Boundaries of sequences near a warp's rows: between `low` and `high`, both exclusive, there is none.
struct Near {
    int low = INT_MAX, high = INT_MIN;
};

// The longest of the packed sequences, by the whole block, whose threads all call this.
__device__ __forceinline__ int longest_of(const RecurParams &p) {
    __shared__ int most[32];
    int longest = 0;
#pragma unroll 4
    for (int n = threadIdx.x; n < p.nseq; n += blockDim.x) longest = max(longest, p.cu[n + 1] - p.cu[n]);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = longest;
    __syncthreads();
    for (int w = 0; w < int(blockDim.x >> 5); ++w) longest = max(longest, most[w]);
    return longest;
}

// A block's place: the part of the stream whose rows it shares with the other blocks of a cluster, or takes alone.
struct Place {
    int part, parts, length, rank, size;

    __device__ __forceinline__ Place(const RecurParams &p, int cluster_rank, int cluster_size, int longest)
        : part(int(blockIdx.x) / cluster_size / p.slabs), parts(p.parts), length(p.part), rank(cluster_rank), size(cluster_size) {
        if (longest <= p.solo_most && p.solo_part > 0) {
            part = part * size + rank;
            parts *= size;
            length = p.solo_part;
            rank = 0, size = 1;
        }
    }
};

// What a warp knows of its R rows: which are its part's, which begin a sequence, which end one.
struct Rows {
    unsigned live, starts, lasts;
    int entry;                  // lane j: the state entry of row j's sequence, where a row begins or ends one
};

template <int R>
__device__ __forceinline__ unsigned live_bits(int row0, int begin, int end) {
    if (row0 >= begin && row0 + R <= end) return (1u << R) - 1u;
    const int lo = max(begin - row0, 0), hi = min(end - row0, R);
    return hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}

// State entry of sequence n, or -1 for none.
__device__ __forceinline__ int recur_entry(const RecurParams &p, int n) {
    if (n < 0 || n >= p.nseq) return -1;                   // malformed cu_seqlens
    if (p.slots == nullptr) return n;
    const int s = p.slots[n];
    return s >= 0 && s < p.num_slots ? s : -1;
}

struct Looked {
    Rows rows;
    Near near;
};
template <int R>
__device__ __noinline__ Looked look_closely(const RecurParams &p, int row0, unsigned live, int end, int lane) {
    Near near;
    int n = 0;                                             // of row row0 + lane
    unsigned s;                                            // bits 0 .. R: rows at which a sequence begins
    if (p.cu == nullptr) {
        const unsigned t = unsigned(p.T), before = unsigned(row0) / t * t;
        n = int(unsigned(row0 + lane) / t);
        s = __ballot_sync(0xffffffffu, lane <= R && unsigned(n) * t == unsigned(row0 + lane));
        near.low = int(before) - (before == unsigned(row0) ? 1 : 0);
        near.high = int(before == unsigned(row0) ? before : before + t);
    } else {
        const int first = count_until(p.cu, p.nseq + 1, row0 - 1, lane);
        int at = first + lane;
        const int bound = at <= p.nseq ? p.cu[at] : INT_MAX;
        near.low = first > 0 ? p.cu[first - 1] : -1;
        near.high = __shfl_sync(0xffffffffu, bound, 0);
        unsigned bits = 0;
        for (int v = bound;;) {
            const int d = v - row0;
            if (d >= 0 && d <= R) bits |= 1u << d;
            if (__shfl_sync(0xffffffffu, v, 31) > row0 + R) break;
            at += 32;                                      // only where sequences are short or empty
            v = at <= p.nseq ? p.cu[at] : INT_MAX;
        }
        s = __reduce_or_sync(0xffffffffu, bits);
        if (s != 0 || end - row0 <= R) {
#pragma unroll 1
            for (int j = 0; j < R; ++j) {
                int k = __popc(__ballot_sync(0xffffffffu, bound <= row0 + j));
                if (k == 32) k = count_until(p.cu, p.nseq + 1, row0 + j, lane) - first;
                if (lane == j) n = first + k - 1;
            }
        }
    }
    Rows r{live, s & live, s >> 1, -1};
    if (end - 1 - row0 < R) r.lasts |= 1u << (end - 1 - row0);
    r.lasts &= live;
    if ((r.starts | r.lasts) >> (lane & 31) & 1u) r.entry = recur_entry(p, n);
    return {r, near};
}

// What there is to know of the rows row0 .. row0 + R, those with their bit in `live`; most tiles are
// inside a sequence that an earlier one has shown.
template <int R>
__device__ __forceinline__ Rows look_at(const RecurParams &p, Near &near, int row0, unsigned live, int end, int lane) {
    if (live == 0 || (near.low < row0 && row0 + R < near.high && row0 + R < end)) return Rows{live, 0, 0, -1};
    const Looked l = look_closely<R>(p, row0, live, end, lane);
    near = l.near;
    return l.rows;
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

// ---------------------------------------------------------------- arithmetic
// VEC channels at once; two of them by the paired instructions, which halves what is issued.
template <int VEC>
__device__ __forceinline__ void mul_to(float (&r)[VEC], const float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
            const float2 t = __fmul2_rn(make_float2(a[v], a[v + 1]), make_float2(b[v], b[v + 1]));
            r[v] = t.x, r[v + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[v] = a[v] * b[v];
    }
}
template <int VEC>
__device__ __forceinline__ void add_to(float (&r)[VEC], const float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
            const float2 t = __fadd2_rn(make_float2(a[v], a[v + 1]), make_float2(b[v], b[v + 1]));
            r[v] = t.x, r[v + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[v] = a[v] + b[v];
    }
}
template <int VEC>
__device__ __forceinline__ void fma_to(float (&r)[VEC], const float (&a)[VEC], const float (&b)[VEC], const float (&c)[VEC]) {
    if constexpr (VEC % 2 == 0) {
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
            const float2 t =
                __ffma2_rn(make_float2(a[v], a[v + 1]), make_float2(b[v], b[v + 1]), make_float2(c[v], c[v + 1]));
            r[v] = t.x, r[v + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[v] = fmaf(a[v], b[v], c[v]);
    }
}
template <int VEC>
__device__ __forceinline__ void fma_to(float (&r)[VEC], const float (&a)[VEC], float b, float c) {
    float bb[VEC], cc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) bb[v] = b, cc[v] = c;
    fma_to<VEC>(r, a, bb, cc);
}

// The values of VEC codes and their scale.  A code + 128 in the low byte of 2^23 is 2^23 + 128 + code: an addition makes it
// a float, where conversions would take the slow pipe.
template <int VEC>
__device__ __forceinline__ void code_values(raw_t<int8_t, VEC> raw, float scale, float (&v)[VEC]) {
    unsigned w[(VEC + 3) / 4] = {};
    memcpy(w, &raw, sizeof(raw));
    float off[VEC], s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const unsigned u = w[i / 4] ^ 0x80808080u;
        v[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650u | unsigned(i % 4)));
        off[i] = -8388736.f;
        s[i] = scale;
    }
    add_to<VEC>(v, v, off);
    mul_to<VEC>(v, v, s);
}

// a and 1 - a from the sigmoid's arguments g, both without cancellation: with z = exp(-g), a = 1 / (1 + z) and 1 - a = z a.
// The quotient is the approximate reciprocal with one Newton step, since a decay's relative error
// counts as often as the state remembers tokens.  FULL: the exponential of full accuracy, for FP32 arguments.
// Else the fast one, whose error grows with |g| (2^-20 of 1 - a at 8, 2^-19 at 16; of a small a
// likewise): 16-bit arguments carry 2^-12 |g| at best themselves.  Below 2^-126, 1 - a is then 0 and a is 2^-126.
// ZERO, the faster form: an a below 2^-126 is 0, and with it what is given for 1 - a, for use as a factor beside a alone.
template <bool FULL, int VEC, bool ZERO = false>
__device__ __forceinline__ void sigmoid_pair(float (&a)[VEC], float (&rest)[VEC]) {
    if constexpr (FULL) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float g = a[v], z = expf(-fabsf(g)), d = 1.f + z;
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
            r = fmaf(r, fmaf(-d, r, 1.f), r);
            const float s = z * r;
            a[v] = g >= 0.f ? r : s;                       // a NaN is in r and s already
            rest[v] = g >= 0.f ? s : r;
        }
    } else {
        float z[VEC], m[VEC], r[VEC], u[VEC], k[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) k[v] = -1.4426950408889634f;
        mul_to<VEC>(z, a, k);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            // 126: 1 + z stays finite, and its reciprocal a normal number; 127: which is flushed to 0
            if constexpr (ZERO) asm("min.NaN.f32 %0, %0, 0f42FE0000;" : "+f"(z[v]));
            else asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(z[v]));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(z[v]));
        }
        fma_to<VEC>(m, z, -1.f, -1.f);                     // -(1 + z)
#pragma unroll
        for (int v = 0; v < VEC; ++v) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[v]) : "f"(-m[v]));
#pragma unroll
        for (int v = 0; v < VEC; ++v) k[v] = 1.f;
        fma_to<VEC>(u, m, r, k);
        fma_to<VEC>(a, r, u, r);
        mul_to<VEC>(rest, z, a);
    }
}

// The decays of VEC values g (in a, then their decays) and, where the form has a use for it, 1 - a.  Log decays
// take the exponential of full accuracy, for the reason above.
template <bool FULL, int VEC>
__device__ __forceinline__ void decays(int form, float (&a)[VEC], float (&rest)[VEC]) {
    if (form & RECUR_SIGMOID) {
        sigmoid_pair<FULL, VEC>(a, rest);
        return;
    }
    float g[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) g[v] = a[v], a[v] = expf(a[v]);
    if (form & RECUR_COMPLEMENT) {
        // 1 - exp(g) = -g (1 + g/2! + g^2/3! + ...) near 0, where the difference would cancel: eight terms leave
        // 0.35^8 / 9! = 6e-10 of it
        float q[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) q[v] = 1.f / 40320.f;
        const float inverse[7] = {1.f / 5040.f, 1.f / 720.f, 1.f / 120.f, 1.f / 24.f, 1.f / 6.f, 0.5f, 1.f};
#pragma unroll
        for (int k = 0; k < 7; ++k) {
            float c[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) c[v] = inverse[k];
            fma_to<VEC>(q, q, g, c);
        }
        mul_to<VEC>(q, q, g);
#pragma unroll
        for (int v = 0; v < VEC; ++v) rest[v] = g[v] > -0.35f ? -q[v] : 1.f - a[v];
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

// ------------------------------------------------------------------- inputs
// One row operand of a warp: R rows of the block's columns, of type S (int8_t: codes, with their exponents), in a
// ring in shared memory of the warp's own.  It is filled by asynchronous copies of PIECE bytes (16, or 4 for rows of
// FP32 that 16 do not fit), or with PIECE 0 through registers, element by element, for any width and alignment (one
// channel to a lane).
template <typename S, int VEC, int R, int RING, int PIECE>
struct Source {
    static constexpr int ROW = 32 * VEC * int(sizeof(S)), BYTES = R * ROW;   // of a warp's rows
    static constexpr bool CODES = sizeof(S) == 1;
    static constexpr int BYTES_RING = RING * (BYTES + (CODES ? 128 : 0));
    static constexpr int PIECES = PIECE == 0 ? 32 : ROW / PIECE;             // of a row
    static constexpr int ROWS = PIECES < 32 ? 32 / PIECES : 1;               // of one copy of the warp
    static_assert(!CODES || R * VEC <= 32, "one scale to a lane");
    unsigned char *ring;
    const S *base;
    const char *from;           // the lane's first piece of the next tile
    int64_t ld, step, down;     // pitch; bytes from one tile of the warp to its next, and between the rows of two copies
    uint32_t to;                // the lane's place in the ring
    int own_row;
    bool own;                   // whether the lane has a piece: its row and column are there
    raw_t<S, VEC> raw[PIECE == 0 ? R : 1];
    unsigned exponent = 0;      // codes: of row lane / VEC, block lane % VEC of the warp's columns

    // the warp's tiles begin at row0 and are `rows` apart
    __device__ __forceinline__ void open(unsigned char *at, const void *tensor, int64_t pitch, int row0, int rows, int D, int slab,
                                         int lane) {
        ring = at;
        base = static_cast<const S *>(tensor);
        ld = pitch;
        step = rows * ld * int(sizeof(S));
        down = ROWS * ld * int(sizeof(S));
        to = smem_u32(ring) + lane * PIECE;
        own_row = PIECE == 0 ? 0 : lane / PIECES;
        const int col = slab + (PIECE == 0 ? lane * VEC : lane % PIECES * (PIECE / int(sizeof(S))));
        own = col < D && own_row < R;
        from = reinterpret_cast<const char *>(base + int64_t(row0 + own_row) * ld + col);
    }
    // A tile's rows row0 .. row0 + R take two steps: load() when the tile before it is put(), and put() into its place of
    // the ring.  Rows without their bit in `live` read as zeros.
    __device__ __forceinline__ void load(const uint8_t *exps, int row0, unsigned live, int D, int slab, int lane) {
        if constexpr (PIECE == 0) {
            const S *s = base + int64_t(row0) * ld + slab + lane * VEC;
#pragma unroll
            for (int j = 0; j < R; ++j) raw[j] = own && (live >> j & 1u) ? load_once<S, VEC>(s + j * ld) : raw_t<S, VEC>{};
        }
        if constexpr (CODES) {
            // 32 VEC columns are VEC blocks of 32; the block's first column is a multiple of 32
            const int j = lane / VEC, block = slab / CKPT_BLOCK + lane % VEC, blocks = (D + CKPT_BLOCK - 1) / CKPT_BLOCK;
            exponent = j < R && block < blocks && (live >> j & 1u) ? exps[int64_t(row0 + j) * blocks + block] : 0u;
        }
    }
    __device__ __forceinline__ static void copy(uint32_t at, const void *source, int bytes) {
        if constexpr (PIECE == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(source), "r"(bytes) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at), "l"(source), "r"(bytes) : "memory");
    }
    // BRANCH: whole tiles apart, which is quicker where the copies are all that a warp has to do at the time.
    template <bool BRANCH>
    __device__ __forceinline__ void put(unsigned live, int lane, int place) {
        if constexpr (PIECE == 0) {
#pragma unroll
            for (int j = 0; j < R; ++j)
                *reinterpret_cast<raw_t<S, VEC> *>(ring + place * BYTES + j * ROW + lane * VEC * int(sizeof(S))) = raw[j];
        } else {
            constexpr int COPIES = (R + ROWS - 1) / ROWS;
            const uint32_t at = to + place * BYTES;
            const char *s = from;
            const unsigned have = own ? live >> own_row : 0u;
            if (BRANCH && live == (1u << R) - 1u && own) {
#pragma unroll
                for (int i = 0; i < COPIES; ++i, s += down) copy(at + i * ROWS * ROW, s, PIECE);
            } else {
#pragma unroll
                for (int i = 0; i < COPIES; ++i, s += down) {
                    const bool ok = have >> (i * ROWS) & 1u;
                    if (R >= ROWS || own_row < R) copy(at + i * ROWS * ROW, ok ? s : reinterpret_cast<const char *>(base), ok ? PIECE : 0);
                }
            }
            from += step;
        }
        if constexpr (CODES) scales(place)[lane] = ckpt_scale(exponent);
    }
    __device__ __forceinline__ float *scales(int place) const {
        return reinterpret_cast<float *>(ring + RING * BYTES) + place * 32;
    }
    __device__ __forceinline__ void value(int j, float (&v)[VEC], int lane, int place) const {
        const raw_t<S, VEC> r =
            *reinterpret_cast<const raw_t<S, VEC> *>(ring + place * BYTES + j * ROW + lane * VEC * int(sizeof(S)));
        if constexpr (CODES) code_values<VEC>(r, scales(place)[j * VEC + lane * VEC / CKPT_BLOCK], v);
        else widen<S, VEC>(r, v);
    }
};
__device__ __forceinline__ void tile_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all tiles but the AHEAD ones sent last are there, for all lanes
template <int AHEAD>
__device__ __forceinline__ void tile_ready() {
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
    __syncwarp();
}

// The warp's number in the block, the same register for all lanes as far as the compiler sees.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0); }

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size() {
    int r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// N floats (2 or 4) to the same place in block `rank` of the cluster, counted there on its mbarrier `bar`.
template <int N>
__device__ __forceinline__ void send_floats(const float *at, uint64_t *bar, int rank, const float (&v)[N]) {
    if constexpr (N == 4)
        asm volatile(
            "{\n\t.reg .b32 a, b;\n\t"
            "mapa.shared::cluster.u32 a, %0, %2;\n\t"
            "mapa.shared::cluster.u32 b, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%3, %4, %5, %6}, [b];\n\t}" ::"r"(smem_u32(at)),
            "r"(smem_u32(bar)), "r"(rank), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .b32 a, b;\n\t"
            "mapa.shared::cluster.u32 a, %0, %2;\n\t"
            "mapa.shared::cluster.u32 b, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [a], {%3, %4}, [b];\n\t}" ::"r"(smem_u32(at)),
            "r"(smem_u32(bar)), "r"(rank), "f"(v[0]), "f"(v[1])
            : "memory");
}
// Wait for phase `parity` of `bar`, whose bytes come from other blocks of the cluster; false after a second.
__device__ __forceinline__ bool cluster_mbar_wait(uint64_t *bar, uint32_t parity) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
            : "memory");
        if (ok != 0) return true;
        if (it == 0) t0 = globaltimer();
        else if ((it & 63u) == 0u && globaltimer() - t0 > WAIT_LIMIT_NS) return false;
    }
}

constexpr int RECUR_CLUSTER = 16;             // most blocks of a cluster

// The map of a run of rows for K neighbouring channels: a and h' of each, for h -> a h + h', or with SET's bits in place of a
// for h -> h', whatever came before.  Arithmetic never gives these bits: its NaNs are all 0x7fffffff.
constexpr unsigned MAP_SET = 0x7fc0a5e7u;
template <int VEC>
struct Map {
    float m[2 * VEC];                         // a, h' of each channel
    __device__ __forceinline__ void read(const float *at) { widen<float, 2 * VEC>(*reinterpret_cast<const raw_t<float, 2 * VEC> *>(at), m); }
    __device__ __forceinline__ void write(float *at) const { store_raw<float, 2 * VEC>(at, narrow<float, 2 * VEC>(m)); }
    __device__ __forceinline__ bool set() const { return __float_as_uint(m[0]) == MAP_SET; }
    __device__ __forceinline__ void apply(float (&h)[VEC]) const {
        const bool s = set();
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = s ? m[2 * v + 1] : fmaf(m[2 * v], h[v], m[2 * v + 1]);
    }
};

// The maps that the W warps of a block hand to the warp that chains them, between two barriers of the block, and what
// their rows start from, which comes back in the maps' place.
template <int VEC, int W, bool BACK>
struct Chain {
    static constexpr int ROW = 64 * VEC, BYTES = W * ROW * int(sizeof(float));
    float *maps;                              // [W][32 lanes]

    static __device__ __forceinline__ int of(int i) { return BACK ? W - 1 - i : i; }
    __device__ __forceinline__ float *at(int warp, int lane) const { return maps + warp * ROW + lane * 2 * VEC; }

    __device__ __forceinline__ void put(int warp, int lane, const float (&a)[VEC], const float (&h)[VEC], bool set) const {
        Map<VEC> m;
#pragma unroll
        for (int v = 0; v < VEC; ++v) m.m[2 * v] = set ? __uint_as_float(MAP_SET) : a[v], m.m[2 * v + 1] = h[v];
        m.write(at(warp, lane));
    }
    __device__ __forceinline__ void get(int warp, int lane, float (&h)[VEC]) const {
        Map<VEC> m;
        m.read(at(warp, lane));
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = m.m[2 * v];
    }
    // K channels from number c on, by one thread: the map of all warps' rows in order; and what each warp's start
    // from, given h, which becomes what follows them.  Four maps are read at a time.
    template <int K>
    __device__ __forceinline__ Map<K> all(int c) const {
        float A[K], H[K];
        bool set = false;
#pragma unroll
        for (int v = 0; v < K; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            Map<K> m;
            m.read(maps + of(i) * ROW + 2 * c);
            m.apply(H);
#pragma unroll
            for (int v = 0; v < K; ++v) A[v] *= m.m[2 * v];
            set = set || m.set();
        }
        Map<K> r;
#pragma unroll
        for (int v = 0; v < K; ++v) r.m[2 * v] = set ? __uint_as_float(MAP_SET) : A[v], r.m[2 * v + 1] = H[v];
        return r;
    }
    template <int K>
    __device__ __forceinline__ void give(int c, float (&h)[K]) const {
#pragma unroll
        for (int base = 0; base < W; base += 4) {
            Map<K> m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (base + i < W) m[i].read(maps + of(base + i) * ROW + 2 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (base + i >= W) continue;
#pragma unroll
                for (int v = 0; v < K; ++v) maps[of(base + i) * ROW + 2 * (c + v)] = h[v];
                m[i].apply(h);
            }
        }
    }
};

// The same between the blocks of a cluster: every block's map of its tile to all of them, two tiles' worth in turn.
template <int VEC>
struct Blocks {
    static constexpr int ROW = 64 * VEC;
    float *maps;                              // [2][size][32 lanes]
    uint64_t *bar;                            // [2]
    bool dead = false;

    static int bytes(int size) { return size > 1 ? 2 * size * ROW * int(sizeof(float)) + 16 : 0; }
    // all threads, before the first tile and behind the last one
    __device__ __forceinline__ void open(int size) const {
        if (size == 1) return;
        if (threadIdx.x == 0) {
            mbar_init(&bar[0], 1);
            mbar_init(&bar[1], 1);
            fence_mbar_init();
        }
        cluster_barrier();
    }
    __device__ __forceinline__ void close(int size) const {
        if (size > 1) cluster_barrier();       // no block leaves while another may still write to it
    }
    // K channels from number c on, by one thread; tile number `turn`
    template <int K>
    __device__ __forceinline__ void send(int c, int rank, int size, int turn, const Map<K> &mine) const {
        const int buf = turn & 1;
        for (int to = 0; to < size; ++to) send_floats<2 * K>(maps + (buf * size + rank) * ROW + 2 * c, &bar[buf], to, mine.m);
        if (c == 0) mbar_arrive_expect_tx(&bar[buf], uint32_t(size * ROW * int(sizeof(float))));
    }
    // What this block's tile starts from; the carry is that of the cluster's tiles, and then of its next ones.  The place
    // and its phase are used again two tiles on: nobody sends there before it has this block's map of the
    // next tile, which goes out behind the barrier that ends this one.
    template <int K>
    __device__ __forceinline__ void receive(int c, int rank, int size, int turn, float (&carry)[K], float (&h)[K],
                                            unsigned *err) {
        const int buf = turn & 1;
        if (!dead && !cluster_mbar_wait(&bar[buf], uint32_t(turn >> 1) & 1u)) {
            dead = true;
            atomicOr(err, ERR_WAIT_TIMEOUT);
        }
        for (int base = 0; base < size; base += 4) {                         // four loads at a time
            Map<K> m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (base + i < size) m[i].read(maps + (buf * size + base + i) * ROW + 2 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (base + i == rank) {
#pragma unroll
                    for (int v = 0; v < K; ++v) h[v] = carry[v];
                }
                if (base + i < size) m[i].apply(carry);
            }
        }
    }
};

// ------------------------------------------------------------------ forward
// Many sequences of like lengths: one warp walks the rows of a part alone, nothing is chained, and every row is looked at
// once.  The warps of all blocks share the parts and columns.  Bound by HBM: 16 x 512 rows of 8192 channels, BF16, in 61 us,
// 360 MB at 74 % of the DRAM's peak (floor 59).  The ring hides the latency of the loads, which 7 warps
// to an SM would not.
template <typename T, typename G, int VEC>
struct WalkShape {
    static constexpr int R = 8, TILE_BYTES = 32 * VEC * R * int(sizeof(T) + sizeof(G)), RING = TILE_BYTES > 4096 ? 2 : 3;
    using X = Source<T, VEC, R, RING, 16>;
    using S = Source<G, VEC, R, RING, 16>;
    static constexpr int WARP = X::BYTES_RING + S::BYTES_RING;
};

template <typename T, typename G, int VEC, int R, int W, int RINGS, int PIECE>
struct ScanShape {
    static constexpr int RING = RINGS;        // tiles in a warp's ring
    using X = Source<T, VEC, R, RING, PIECE>;
    using S = Source<G, VEC, R, RING, PIECE>;
    using Warps = Chain<VEC, W, false>;
    using Cluster = Blocks<VEC>;
    static constexpr int WARP = X::BYTES_RING + S::BYTES_RING, THREADS = (W + 1) * 32, COLUMNS = 32 * VEC, TILE = R * W;
    // of a walking warp of the block, with 8 bytes of x to a lane; 4 take less
    static constexpr int WIDE = 8 / int(sizeof(T)), WALK = PIECE == 16 ? (W + 1) * WalkShape<T, G, WIDE>::WARP : 0;
    static int bytes(int cluster) {
        const int chained = W * WARP + Warps::BYTES + Cluster::bytes(cluster);
        return chained > WALK ? chained : WALK;
    }
};

template <typename T, typename G, int VEC>
__device__ __forceinline__ void walk(const RecurParams &p, const int form, int part, int slab, unsigned char *ring, int lane) {
    using Shape = WalkShape<T, G, VEC>;
    constexpr int R = Shape::R, RING = Shape::RING;
    constexpr bool FULL = sizeof(G) == 4;
    const int col = slab + lane * VEC;
    const bool in = col < p.D;
    int begin, end;
    part_rows(p, part, p.walk_parts, p.walk_part, lane, begin, end);
    const int tile0 = begin / R, tiles = end > begin ? (end - 1) / R + 1 - tile0 : 0;
    typename Shape::X xs;
    typename Shape::S gs;
    xs.open(ring, p.x, p.ldx, tile0 * R, R, p.D, slab, lane);
    gs.open(ring + xs.BYTES_RING, p.g, p.ldg, tile0 * R, R, p.D, slab, lane);
    auto put = [&](int tile, int place) {
        if (tile < tiles) {
            const unsigned live = live_bits<R>((tile0 + tile) * R, begin, end);
            xs.template put<true>(live, lane, place);
            gs.template put<true>(live, lane, place);
        }
        tile_sent();
    };
    for (int i = 0; i < RING; ++i) put(i, i);
    Near near;
    float h[VEC] = {};
    int place = 0;
    T *y = static_cast<T *>(p.y) + int64_t(tile0) * R * p.D + col;
    for (int tile = 0; tile < tiles; ++tile) {
        const int row0 = (tile0 + tile) * R;
        const Rows rows = look_at<R>(p, near, row0, live_bits<R>(row0, begin, end), end, lane);
        tile_ready<RING - 1>();
        auto row = [&](int j) {
            float a[VEC], b[VEC], c[VEC];
            xs.value(j, b, lane, place);
            gs.value(j, a, lane, place);
            decays<FULL, VEC>(form, a, c);
            if (form & RECUR_COMPLEMENT) mul_to<VEC>(b, b, c);
            fma_to<VEC>(h, a, h, b);
        };
        if (row0 % RECUR_CHUNK == 0 && (rows.live & 1u) && !(rows.starts & 1u))
            store_state<VEC>(h, p.chunk, row0 / RECUR_CHUNK, p.D, col);
        if ((rows.starts | rows.lasts) == 0 && rows.live == (1u << R) - 1u) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                row(j);
                if (in) store_raw<T, VEC>(y, narrow<T, VEC>(h));
                y += p.D;
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < R; ++j, y += p.D) {
                if (!(rows.live >> j & 1u)) continue;
                if (rows.starts >> j & 1u) {
                    load_state<VEC>(h, p.state_in, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
                    if (j == 0 && row0 % RECUR_CHUNK == 0) store_state<VEC>(h, p.chunk, row0 / RECUR_CHUNK, p.D, col);
                }
                row(j);
                if (in) store_raw<T, VEC>(y, narrow<T, VEC>(h));
                if (rows.lasts >> j & 1u) store_state<VEC>(h, p.state_out, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
            }
        }
        __syncwarp();
        put(tile + RING, place);
        place = place + 1 == RING ? 0 : place + 1;
    }
    copy_empty<VEC>(p, p.state_in, p.state_out, part, p.walk_parts, lane, col);
    __syncwarp();                                           // the ring may go to the next part
}

template <typename T, typename G, int VEC>
__device__ __forceinline__ void walk_all(const RecurParams &p, int form, unsigned char *shared, int warp, int warps, int lane) {
    const int slabs = (p.D + 32 * VEC - 1) / (32 * VEC), units = slabs * p.walk_parts;
    const int blocks = int(gridDim.x), block = int(blockIdx.x);
    for (int u = warp * blocks + block; u < units; u += warps * blocks)
        walk<T, G, VEC>(p, form, u / slabs, u % slabs * 32 * VEC, shared + warp * WalkShape<T, G, VEC>::WARP, lane);
}

// FORM: RECUR_ bits, or -1 for those of the parameters.  W warps take the rows, one more chains their maps: it would
// not find the registers in theirs.
//
// One sequence of 65536 rows of 2048 channels, BF16, chunk states kept: 175 us by 32 clusters of 8 (floor 120; 41 % of the issue
// slots).  What bounds it is the exchange between the blocks of a cluster, one tile after the other: the same work
// without it, by parts that are each a sequence, takes 145 us, and 131 by 9 parts, for which there is no room in
// clusters.  Two tiles in the ring: 164 us for 16384 rows of 8192 channels, 170 with one.  16 rows to a warp are what the
// registers of two blocks hold; half as many double the exchanges.
template <typename T, typename G, int FORM, int VEC, int R, int W, int RING, int PIECE, int MIN>
__global__ void __launch_bounds__((W + 1) * 32, MIN) kda_gated_scan_kernel(const __grid_constant__ RecurParams p) {
    constexpr int TILE = R * W;
    constexpr bool FULL = sizeof(G) == 4;
    static_assert(RECUR_CHUNK % R == 0 && R <= 16, "chunk states lie at warps' first rows");
    using Shape = ScanShape<T, G, VEC, R, W, RING, PIECE>;
    extern __shared__ __align__(16) unsigned char shared[];
    const int lane = threadIdx.x & 31, warp = warp_index(), all = cluster_size();
    const typename Shape::Warps chain{reinterpret_cast<float *>(shared + W * Shape::WARP)};
    typename Shape::Cluster cluster;
    cluster.maps = reinterpret_cast<float *>(shared + W * Shape::WARP + Shape::Warps::BYTES);
    cluster.bar = reinterpret_cast<uint64_t *>(cluster.maps + 2 * all * cluster.ROW);
    const int slab = int(blockIdx.x) / all % p.slabs * 32 * VEC, col = slab + lane * VEC;
    const int form = FORM < 0 ? p.form : FORM;
    const bool in = col < p.D;
    pdl_wait();
    const int longest = p.cu != nullptr && (p.walk_parts > 0 || p.solo_part > 0) ? longest_of(p) : 0;
    if constexpr (PIECE == 16) {
        if (p.walk_parts > 0 && longest <= p.walk_most) {   // the same for all blocks
            if (p.walk_wide) walk_all<T, G, Shape::WIDE>(p, form, shared, warp, W + 1, lane);
            else walk_all<T, G, Shape::WIDE / 2>(p, form, shared, warp, W + 1, lane);
            pdl_launch_dependents();
            return;
        }
    }
    const Place at(p, cluster_rank(), all, longest);
    if (at.part >= at.parts) return;                        // the whole cluster
    const int rank = at.rank, size = at.size;
    int begin, end;
    part_rows(p, at.part, at.parts, at.length, lane, begin, end);
    const int tile0 = begin / TILE, tiles = end > begin ? (end - 1) / TILE + 1 - tile0 : 0;
    const int turns = (tiles + size - 1) / size;
    if (warp == W) {
        float h[VEC] = {}, carry[VEC] = {};                 // what the block's and the cluster's tiles start from
        const int c = lane * VEC;
        cluster.open(size);
        for (int turn = 0; turn < turns; ++turn) {
            __syncthreads();
            if (size > 1) {
                cluster.template send<VEC>(c, rank, size, turn, chain.template all<VEC>(c));
                cluster.template receive<VEC>(c, rank, size, turn, carry, h, p.err);
            }
            chain.template give<VEC>(c, h);
            __syncthreads();
        }
        cluster.close(size);
        return;
    }
    typename Shape::X xs;
    typename Shape::S gs;
    auto first_row = [&](int turn) { return (tile0 + turn * size + rank) * TILE + warp * R; };
    xs.open(shared + warp * Shape::WARP, p.x, p.ldx, first_row(0), size * TILE, p.D, slab, lane);
    gs.open(xs.ring + xs.BYTES_RING, p.g, p.ldg, first_row(0), size * TILE, p.D, slab, lane);
    auto live_of = [&](int turn) { return turn < turns ? live_bits<R>(first_row(turn), begin, end) : 0u; };
    auto load = [&](int turn) {
        if (PIECE != 0) return;
        xs.load(nullptr, first_row(turn), live_of(turn), p.D, slab, lane);
        gs.load(nullptr, first_row(turn), live_of(turn), p.D, slab, lane);
    };
    auto put = [&](int turn, int place) {
        if (turn < turns) {
            const unsigned live = live_of(turn);
            xs.template put<true>(live, lane, place);
            gs.template put<true>(live, lane, place);
        }
        tile_sent();
    };
    // decay and input of row j
    auto row_of = [&](int j, int place, float (&a)[VEC], float (&b)[VEC]) {
        float c[VEC];
        xs.value(j, b, lane, place);
        gs.value(j, a, lane, place);
        decays<FULL, VEC>(form, a, c);
        if (form & RECUR_COMPLEMENT) mul_to<VEC>(b, b, c);
    };
    T *const y = static_cast<T *>(p.y) + col;
    load(0);
    for (int i = 0; i < RING; ++i) {
        put(i, i);
        load(i + 1);
    }
    cluster.open(size);
    Near near;
    int place = 0;
    for (int turn = 0; turn < turns; ++turn) {
        const int row0 = first_row(turn);
        float a[R][VEC], b[R][VEC], h[VEC], A[VEC], H[VEC];
        tile_ready<RING - 1>();
#pragma unroll
        for (int j = 0; j < R; ++j) {
            row_of(j, place, a[j], b[j]);
            if (j == 0) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) A[v] = a[0][v], H[v] = b[0][v];
            } else {
                fma_to<VEC>(H, a[j], H, b[j]);
                mul_to<VEC>(A, A, a[j]);
            }
        }
        const Rows rows = look_at<R>(p, near, row0, live_bits<R>(row0, begin, end), end, lane);
        if (rows.starts != 0) {
            // from the first row that begins a sequence on, nothing depends on what came before: these rows
            // are finished here, before state_in can be overwritten
#pragma unroll 1
            for (int j = __ffs(rows.starts) - 1; j < R; ++j) {
                if (!(rows.live >> j & 1u)) break;
                float aj[VEC], bj[VEC];
                row_of(j, place, aj, bj);
                if (rows.starts >> j & 1u) {
                    load_state<VEC>(H, p.state_in, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
                    if (j == 0 && row0 % RECUR_CHUNK == 0) store_state<VEC>(H, p.chunk, row0 / RECUR_CHUNK, p.D, col);
                }
                fma_to<VEC>(H, aj, H, bj);
                if (in) store_raw<T, VEC>(y + int64_t(row0 + j) * p.D, narrow<T, VEC>(H));
                if (rows.lasts >> j & 1u) store_state<VEC>(H, p.state_out, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
            }
        }
        chain.put(warp, lane, A, H, rows.starts != 0);
        __syncthreads();
        put(turn + RING, place);                            // all lanes are through with the tile's place
        load(turn + RING + 1);
        place = place + 1 == RING ? 0 : place + 1;
        __syncthreads();
        if (rows.live == 0) continue;
        chain.get(warp, lane, h);
        if (row0 % RECUR_CHUNK == 0 && (rows.live & 1u) && !(rows.starts & 1u))
            store_state<VEC>(h, p.chunk, row0 / RECUR_CHUNK, p.D, col);
        T *const to = static_cast<T *>(p.y) + int64_t(row0) * p.D + slab;
        // rows that begin or end a sequence have code of their own: branches in the unrolled rows would keep them apart
        if (__builtin_expect((rows.starts | rows.lasts) == 0 && rows.live == (1u << R) - 1u, 1)) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                fma_to<VEC>(h, a[j], h, b[j]);
                if (in) store_raw<T, VEC>(to + unsigned(j * p.D + lane * VEC), narrow<T, VEC>(h));
            }
        } else {
            const unsigned mine = rows.starts != 0 ? rows.live & ((rows.starts & (0u - rows.starts)) - 1u) : rows.live;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (!(mine >> j & 1u)) continue;
                fma_to<VEC>(h, a[j], h, b[j]);
                if (in) store_raw<T, VEC>(to + unsigned(j * p.D + lane * VEC), narrow<T, VEC>(h));
                if (rows.lasts >> j & 1u) store_state<VEC>(h, p.state_out, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
            }
        }
    }
    pdl_launch_dependents();
    copy_empty<VEC>(p, p.state_in, p.state_out, (at.part * size + rank) * W + warp, at.parts * size * W, lane, col);
    cluster.close(size);
}

// ----------------------------------------------------------------- backward
template <typename T, typename X, typename S, int VEC, int R, int W, int RINGS, int PIECE>
struct GradShape {
    static constexpr int RING = RINGS;
    using Xs = Source<X, VEC, R, RING, PIECE>;
    using Gs = Source<S, VEC, R, RING, PIECE>;
    using Ds = Source<T, VEC, R, RING, PIECE>;
    using Forth = Chain<VEC, W, false>;       // of h within the tile, which is a chunk
    using Back = Chain<VEC, W, true>;         // of a d
    using Cluster = Blocks<VEC>;
    static constexpr int WARP = Xs::BYTES_RING + Gs::BYTES_RING + Ds::BYTES_RING, THREADS = W * 32;
    static constexpr int COLUMNS = 32 * VEC, TILE = R * W;
    static int bytes(int cluster) { return W * WARP + Forth::BYTES + Back::BYTES + Cluster::bytes(cluster); }
};

// T: dy, dx; X, S: x and g, or int8_t for codes; G: dg.
//
// 16 x 512 rows of 8192 channels, BF16: 122 us (floor 100), 635 MB at 63 % of the DRAM's peak and 55 % of the issue slots, which
// two blocks of 8 warps to an SM with a barrier twice to a tile do not use better.  One sequence of 16384 rows of 2048
// channels from codes: 92 us (floor 40; 228 MB, 30 % and 48 %): nothing is saturated, 16 warps to an SM wait for one another
// twice a tile; from tensors it takes 86.  Eight rows and two channels to a lane: with four channels and
// four rows, one block to an SM, 16 x 512 takes 167 us (from codes 186, here 139).
template <typename T, typename X, typename S, typename G, int FORM, int VEC, int R, int W, int RING, int PIECE, int MIN>
__global__ void __launch_bounds__(W * 32, MIN) kda_gated_scan_backward_kernel(const __grid_constant__ RecurParams p) {
    constexpr int TILE = R * W;
    constexpr bool FULL = sizeof(S) == 4;
    // Gradients of 16 x 512 x 8192 BF16: from tensors 125 us with one tile ahead, fetched at once, 120 with two, fetched
    // behind the barrier; from codes 139 and 155.
    constexpr bool LATE = RING > 1;
    static_assert(TILE == RECUR_CHUNK, "a tile is a chunk");
    using Shape = GradShape<T, X, S, VEC, R, W, RING, PIECE>;
    extern __shared__ __align__(16) unsigned char shared[];
    const int lane = threadIdx.x & 31, warp = warp_index(), all = cluster_size();
    const typename Shape::Forth forth{reinterpret_cast<float *>(shared + W * Shape::WARP)};
    const typename Shape::Back back{forth.maps + Shape::Forth::BYTES / int(sizeof(float))};
    typename Shape::Cluster cluster;
    cluster.maps = back.maps + Shape::Back::BYTES / int(sizeof(float));
    cluster.bar = reinterpret_cast<uint64_t *>(cluster.maps + 2 * all * cluster.ROW);
    const int slab = int(blockIdx.x) / all % p.slabs * 32 * VEC, col = slab + lane * VEC;
    const int form = FORM < 0 ? p.form : FORM;
    const bool in = col < p.D, complement = form & RECUR_COMPLEMENT;
    pdl_wait();
    const Place at(p, cluster_rank(), all, p.cu != nullptr && p.solo_part > 0 ? longest_of(p) : 0);
    const int rank = at.rank, size = at.size;
    int begin, end;
    part_rows(p, at.part, at.parts, at.length, lane, begin, end);
    const int tile0 = begin / TILE, tiles = end > begin ? (end - 1) / TILE + 1 - tile0 : 0;
    const int turns = (tiles + size - 1) / size;
    typename Shape::Xs xs;
    typename Shape::Gs gs;
    typename Shape::Ds ds;
    // tiles from the last one back; those before the part's first have no live rows
    auto tile_of = [&](int turn) { return tile0 + tiles - 1 - (turn * size + rank); };
    auto first_row = [&](int turn) { return tile_of(turn) * TILE + warp * R; };
    xs.open(shared + warp * Shape::WARP, p.x, p.ldx, first_row(0), -size * TILE, p.D, slab, lane);
    gs.open(xs.ring + xs.BYTES_RING, p.g, p.ldg, first_row(0), -size * TILE, p.D, slab, lane);
    ds.open(gs.ring + gs.BYTES_RING, p.dy, p.lddy, first_row(0), -size * TILE, p.D, slab, lane);
    auto live_of = [&](int turn) {
        return turn < turns && tile_of(turn) >= tile0 ? live_bits<R>(first_row(turn), begin, end) : 0u;
    };
    auto load = [&](int turn) {
        if (PIECE != 0 && !xs.CODES && !gs.CODES) return;
        const int row0 = first_row(turn);
        const unsigned live = live_of(turn);
        xs.load(p.xe, row0, live, p.D, slab, lane);
        gs.load(p.ge, row0, live, p.D, slab, lane);
        ds.load(nullptr, row0, live, p.D, slab, lane);
    };
    auto put = [&](int turn, int place) {
        if (turn < turns) {
            const unsigned live = live_of(turn);
            xs.template put<false>(live, lane, place);
            gs.template put<false>(live, lane, place);
            ds.template put<false>(live, lane, place);
        }
        tile_sent();
    };
    // a thread to a channel chains the maps: the first C of them backwards, the next C forwards, from the state before the
    // chunk; where the part begins inside the chunk, a row that begins a sequence makes that void
    constexpr int C = 32 * VEC;
    auto chunk_of = [&](int turn, float (&h)[1]) {
        const int t = tile_of(turn), c = slab + int(threadIdx.x) - C;
        const bool mine = threadIdx.x >= C && threadIdx.x < 2 * C && c < p.D;
        h[0] = mine && turn < turns && t >= tile0 && t * TILE >= begin ? p.chunk[int64_t(t) * p.D + c] : 0.f;
    };
    load(0);
    for (int i = 0; i < RING; ++i) {
        put(i, i);
        load(i + 1);
    }
    float chunk[1], carry[1] = {};
    chunk_of(0, chunk);
    cluster.open(size);
    Near near;
    int place = 0;
    auto refill = [&](int turn) {
        put(turn + RING, place);
        load(turn + RING + 1);
        place = place + 1 == RING ? 0 : place + 1;
    };
    for (int turn = 0; turn < turns; ++turn) {
        const int row0 = first_row(turn);
        // x: in the end h before the row, less x where c = 1 - a
        float a[R][VEC], rest[R][VEC], x[R][VEC], d[R][VEC], h[VEC], e[VEC], A[VEC], H[VEC], E[VEC];
        tile_ready<RING - 1>();
#pragma unroll
        for (int j = 0; j < R; ++j) {
            xs.value(j, x[j], lane, place);
            gs.value(j, a[j], lane, place);
            ds.value(j, d[j], lane, place);
            decays<FULL, VEC>(form, a[j], rest[j]);
        }
        if (!LATE) {
            __syncwarp();
            refill(turn);
        }
        const Rows rows = look_at<R>(p, near, row0, live_of(turn), end, lane);
        // h after row j, from h before it
        auto step = [&](float (&s)[VEC], int j) {
            if (complement) {
                float b[VEC];
                mul_to<VEC>(b, rest[j], x[j]);
                fma_to<VEC>(s, a[j], s, b);
            } else {
                fma_to<VEC>(s, a[j], s, x[j]);
            }
        };
        // a sequence's state before its first row, or its state's gradient behind its last
        auto edge = [&](float (&s)[VEC], const float *states, int j) {
            load_state<VEC>(s, states, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
        };
        // the rows' maps, forwards and backwards
        // rows that begin or end a sequence have code of their own: branches in the unrolled rows would keep them apart
        auto sum_up = [&](auto edges) {
            constexpr bool EDGES = decltype(edges)::value;
#pragma unroll
            for (int v = 0; v < VEC; ++v) A[v] = a[0][v], H[v] = E[v] = 0.f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (EDGES && (rows.starts >> j & 1u)) edge(H, p.state_in, j);
                step(H, j);
                if (j > 0) mul_to<VEC>(A, A, a[j]);
            }
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                if (EDGES && (rows.lasts >> j & 1u)) edge(E, p.dfinal, j);
                add_to<VEC>(E, E, d[j]);
                mul_to<VEC>(E, E, a[j]);
            }
        };
        if (__builtin_expect((rows.starts | rows.lasts) == 0, 1)) sum_up(std::false_type{});
        else sum_up(std::true_type{});
        forth.put(warp, lane, A, H, rows.starts != 0);
        back.put(warp, lane, A, E, rows.lasts != 0);
        __syncthreads();
        if (threadIdx.x < C) {
            const int c = threadIdx.x;
            float t[1] = {carry[0]};
            if (size > 1) {
                cluster.template send<1>(c, rank, size, turn, back.template all<1>(c));
                cluster.template receive<1>(c, rank, size, turn, carry, t, p.err);
                back.template give<1>(c, t);
            } else {
                back.template give<1>(c, carry);
            }
        } else if (threadIdx.x < 2 * C) {
            forth.template give<1>(int(threadIdx.x) - C, chunk);
            chunk_of(turn + 1, chunk);
        }
        if (LATE) refill(turn);                             // behind the barrier, while the chain is worked on
        __syncthreads();
        if (rows.live == 0) continue;
        forth.get(warp, lane, h);
        back.get(warp, lane, e);
        const int64_t first = int64_t(row0) * p.D + slab;
        T *const dx = static_cast<T *>(p.dx) + first;
        G *const dg = static_cast<G *>(p.dg) + first;
        auto finish = [&](auto edges) {
            constexpr bool EDGES = decltype(edges)::value;
            float minus[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) minus[v] = -1.f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (EDGES && (rows.starts >> j & 1u)) edge(h, p.state_in, j);
                float was[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) was[v] = h[v];
                if (j < R - 1) step(h, j);
                if (complement) fma_to<VEC>(x[j], x[j], minus, was);
                else {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) x[j][v] = was[v];
                }
            }
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                if (EDGES && (rows.lasts >> j & 1u)) edge(e, p.dfinal, j);
                float dh[VEC], g[VEC];
                add_to<VEC>(dh, d[j], e);
                mul_to<VEC>(e, a[j], dh);
                mul_to<VEC>(g, e, x[j]);
                if (form & RECUR_SIGMOID) mul_to<VEC>(g, g, rest[j]);
                if (complement) mul_to<VEC>(dh, rest[j], dh);
                if (in && (!EDGES || (rows.live >> j & 1u))) {
                    const unsigned at = unsigned(j * p.D + lane * VEC);
                    store_raw<T, VEC>(dx + at, narrow<T, VEC>(dh));
                    store_raw<G, VEC>(dg + at, narrow<G, VEC>(g));
                }
                if (EDGES && p.dinitial != nullptr && (rows.starts >> j & 1u))
                    store_state<VEC>(e, p.dinitial, __shfl_sync(0xffffffffu, rows.entry, j), p.D, col);
            }
        };
        if (__builtin_expect((rows.starts | rows.lasts) == 0 && rows.live == (1u << R) - 1u, 1)) finish(std::false_type{});
        else finish(std::true_type{});
    }
    pdl_launch_dependents();
    copy_empty<VEC>(p, p.dfinal, p.dinitial, (at.part * size + rank) * W + warp, at.parts * size * W, lane, col);
    cluster.close(size);
}

}  // namespace kda
