// kda_recur.cuh -- the gated linear recurrence over whole sequences, and its gradients.
//
// Every channel keeps a state h; with its decay a and its input's factor c (1 or 1 - a),
//
//     h_t = a_t h_{t-1} + c_t x_t,   y_t = h_t.
//
// The sequences lie one after the other in a stream of rows.  A row maps the state before it to the
// state after it, h -> A h + H, and so does any run of rows; a sequence's first row maps everything
// to one state.  A cluster of blocks takes 32 lanes' channels of one part of the stream, tile after tile
// in turn: each warp takes R consecutive rows of its block's tile into registers and works out their map; a
// thread for each channel chains the maps of the block's warps, and those of the cluster's blocks, which
// it sends and receives through their shared memory, to the state that every warp's rows start from; then
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
    unsigned *err;              // device error word
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

// Boundaries of sequences near a warp's rows.  Between `low` and `high`, both exclusive, there is none.
struct Near {
    int low = INT_MAX, high = INT_MIN;
    int first = 0, bound = INT_MAX;   // packed: boundary number `lane` from the last search is entry first + lane of cu
};

// What a warp knows of its R rows: which are its part's, which begin a sequence, which end one.
struct Rows {
    unsigned live, starts, lasts;
};

template <int R>
__device__ __forceinline__ unsigned live_bits(int row0, int begin, int end) {
    const int lo = max(begin - row0, 0), hi = min(end - row0, R);
    return hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
}

template <int R>
__device__ __forceinline__ Rows look_at(const RecurParams &p, Near &near, int row0, int begin, int end, int lane) {
    Rows r{live_bits<R>(row0, begin, end), 0, 0};
    if (r.live == 0) return r;
    unsigned s = 0;                                        // bits 0 .. R: rows at which a sequence begins
    if (!(near.low < row0 && row0 + R < near.high)) {
        if (p.cu == nullptr) {
            const unsigned t = unsigned(p.T), before = unsigned(row0) / t * t;
            s = __ballot_sync(0xffffffffu, lane <= R && unsigned(row0 + lane) % t == 0);
            near.low = int(before) - (before == unsigned(row0) ? 1 : 0);
            near.high = int(before == unsigned(row0) ? before : before + t);
        } else {
            near.first = count_until(p.cu, p.nseq + 1, row0 - 1, lane);
            int at = near.first + lane;
            near.bound = at <= p.nseq ? p.cu[at] : INT_MAX;
            near.low = near.first > 0 ? p.cu[near.first - 1] : -1;
            near.high = __shfl_sync(0xffffffffu, near.bound, 0);
            unsigned bits = 0;
            for (int v = near.bound;;) {
                const int d = v - row0;
                if (d >= 0 && d <= R) bits |= 1u << d;
                if (__shfl_sync(0xffffffffu, v, 31) > row0 + R) break;
                at += 32;                                  // only where sequences are short or empty
                v = at <= p.nseq ? p.cu[at] : INT_MAX;
            }
            s = __reduce_or_sync(0xffffffffu, bits);
        }
    }
    r.starts = s & r.live;
    r.lasts = s >> 1;
    if (end - 1 - row0 < R) r.lasts |= 1u << (end - 1 - row0);
    r.lasts &= r.live;
    return r;
}

// The sequence that `row` belongs to, for a live row that begins or ends one, after look_at; all lanes call it.
__device__ __forceinline__ int sequence_of(const RecurParams &p, const Near &near, int row, int lane) {
    if (p.cu == nullptr) return row / p.T;
    const int k = __popc(__ballot_sync(0xffffffffu, near.bound <= row));
    return (k < 32 ? near.first + k : count_until(p.cu, p.nseq + 1, row, lane)) - 1;
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

// ---------------------------------------------------------------- arithmetic
// VEC channels at once; two of them by the paired instructions, which halves what is issued.
template <int VEC>
__device__ __forceinline__ void mul_to(float (&r)[VEC], const float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC == 2) {
        const float2 t = __fmul2_rn(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
        r[0] = t.x, r[1] = t.y;
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[v] = a[v] * b[v];
    }
}
template <int VEC>
__device__ __forceinline__ void add_to(float (&r)[VEC], const float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC == 2) {
        const float2 t = __fadd2_rn(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
        r[0] = t.x, r[1] = t.y;
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[v] = a[v] + b[v];
    }
}
template <int VEC>
__device__ __forceinline__ void fma_to(float (&r)[VEC], const float (&a)[VEC], const float (&b)[VEC], const float (&c)[VEC]) {
    if constexpr (VEC == 2) {
        const float2 t = __ffma2_rn(make_float2(a[0], a[1]), make_float2(b[0], b[1]), make_float2(c[0], c[1]));
        r[0] = t.x, r[1] = t.y;
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

// a and 1 - a from the sigmoid's arguments g, both without cancellation: with z = exp(-g), a = 1 / (1 + z) and 1 - a = z a.
// The quotient is the approximate reciprocal with one Newton step, since a decay's relative error
// counts as often as the state remembers tokens.  FULL: the exponential of full accuracy, for FP32 arguments.
// Else the fast one, whose error grows with |g| (2^-20 of 1 - a at 8, 2^-19 at 16; of a small a
// likewise): 16-bit arguments carry 2^-12 |g| at best themselves.  Below 2^-126, 1 - a is then 0 and a is 2^-126.
template <bool FULL, int VEC>
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
            asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(z[v]));   // 126: 1 + z stays finite
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
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (form & RECUR_COMPLEMENT) rest[v] = -expm1f(a[v]);
            a[v] = expf(a[v]);
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

// ------------------------------------------------------------------- inputs
// One row operand of a warp: R rows of the block's columns, of type S (int8_t: codes, with their exponents).
//
// Staged: every warp has a ring of its own in shared memory, filled by asynchronous copies of 16 bytes
// whose place in the rows is not the lane that uses them, so a warp's barrier lies between.  It takes two channels to a
// lane and rows of whole, aligned 16-byte pieces.  Direct: each lane loads its own elements into registers
// one tile ahead; for any width and alignment.
template <typename S, int VEC, int R, int STAGES>
struct Source {
    static constexpr bool STAGED = STAGES > 0;
    static constexpr int ROW = 32 * VEC * int(sizeof(S)), BYTES = R * ROW;   // of a warp's rows
    static constexpr int RING = BYTES * STAGES;
    raw_t<S, VEC> raw[STAGED ? 1 : R];
    unsigned scales = 0;        // codes: the exponent of row lane / VEC, block lane % VEC of the warp's columns
    unsigned char *ring = nullptr;

    // rows row0 .. row0 + R of [rows, D] at pitch ld, into place `stage`; rows without their bit in `live` read as zeros
    __device__ __forceinline__ void fetch(const void *base, int64_t ld, int row0, unsigned live, int D, int slab, int lane,
                                          int stage) {
        const S *s = static_cast<const S *>(base);
        if constexpr (STAGED) {
            constexpr int PIECES = ROW / 16, ROWS = 32 / PIECES;             // rows of one copy of the warp
            const int j0 = lane / PIECES, col = slab + lane % PIECES * (16 / int(sizeof(S)));
            const S *from = s + int64_t(row0 + j0) * ld + col;
            const uint32_t to = smem_u32(ring) + stage * BYTES + lane * 16;
            const unsigned have = col < D ? live >> j0 : 0u;
#pragma unroll
            for (int i = 0; i < R / ROWS; ++i) {
                const bool ok = have >> (i * ROWS) & 1u;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 512),
                             "l"(ok ? from + i * ROWS * ld : s), "r"(ok ? 16 : 0) : "memory");
            }
        } else {
            const int col = slab + lane * VEC;
#pragma unroll
            for (int j = 0; j < R; ++j)
                raw[j] = col < D && (live >> j & 1u) ? load_once<S, VEC>(s + int64_t(row0 + j) * ld + col) : raw_t<S, VEC>{};
        }
    }
    __device__ __forceinline__ unsigned fetch_scales(const uint8_t *exps, int row0, unsigned live, int D, int slab, int lane) {
        if constexpr (sizeof(S) == 1) {
            // 32 VEC columns are VEC blocks of 32; the block's first column is a multiple of 32
            const int j = lane / VEC, block = slab / CKPT_BLOCK + lane % VEC, blocks = (D + CKPT_BLOCK - 1) / CKPT_BLOCK;
            return j < R && block < blocks && (live >> j & 1u) ? exps[int64_t(row0 + j) * blocks + block] : 0u;
        }
        return 0u;
    }
    __device__ __forceinline__ void set_scales(unsigned exponents) {
        if constexpr (sizeof(S) == 1) scales = __float_as_uint(ckpt_scale(exponents));
    }
    __device__ __forceinline__ void value(int j, float (&v)[VEC], int lane, int stage) const {
        if constexpr (STAGED)
            widen<S, VEC>(*reinterpret_cast<const raw_t<S, VEC> *>(ring + stage * BYTES + j * ROW + lane * VEC * int(sizeof(S))), v);
        else
            widen<S, VEC>(raw[j], v);
        if constexpr (sizeof(S) == 1) {
            const float s = __uint_as_float(__shfl_sync(0xffffffffu, scales, j * VEC + lane * VEC / CKPT_BLOCK));
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] *= s;
        }
    }
};
template <int STAGES>
__device__ __forceinline__ void tile_sent() {
    if constexpr (STAGES > 0) asm volatile("cp.async.commit_group;" ::: "memory");
}
// the oldest tile in the ring is there, for all lanes
template <int STAGES>
__device__ __forceinline__ void tile_ready() {
    if constexpr (STAGES > 0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();
    }
}

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
// Two floats to the same place in block `rank` of the cluster, counted there on its mbarrier `bar`.
__device__ __forceinline__ void send_pair(const float2 *at, uint64_t *bar, int rank, float2 v) {
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %2;\n\t"
        "mapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [a], {%3, %4}, [b];\n\t}" ::"r"(smem_u32(at)),
        "r"(smem_u32(bar)), "r"(rank), "f"(v.x), "f"(v.y)
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

constexpr int RECUR_CLUSTER = 8;              // most blocks of a cluster

// The map of a run of rows for one channel: (A, H) for h -> A h + H, or with SET's bits in place of A for
// h -> H, whatever came before.  Arithmetic never gives these bits: its NaNs are all 0x7fffffff.
constexpr unsigned MAP_SET = 0x7fc0a5e7u;
__device__ __forceinline__ bool map_set(float2 m) { return __float_as_uint(m.x) == MAP_SET; }
__device__ __forceinline__ float map_apply(float2 m, float h) { return map_set(m) ? m.y : fmaf(m.x, h, m.y); }

// What the blocks exchange for one direction of the recurrence.
template <int VEC, int W, bool BACK>
struct Exchange {
    static constexpr int C = 32 * VEC;
    float2 maps[W][C];                        // of the block's warps
    float in[W][C];                           // what each warp's rows start from
    // the rest for clusters alone: the blocks' maps, two tiles' worth in turn
    float2 blocks[2][RECUR_CLUSTER][C];
    uint64_t bar[2];

    static __host__ __device__ constexpr int bytes(bool cluster) {
        return cluster ? int(sizeof(Exchange)) : W * C * int(sizeof(float2) + sizeof(float));
    }
    static __device__ __forceinline__ int of(int i) { return BACK ? W - 1 - i : i; }

    __device__ __forceinline__ void put(int warp, int lane, const float (&a)[VEC], const float (&h)[VEC], bool set) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) maps[warp][lane * VEC + v] = make_float2(set ? __uint_as_float(MAP_SET) : a[v], h[v]);
    }
    __device__ __forceinline__ void get(int warp, int lane, float (&h)[VEC]) const {
        widen<float, VEC>(*reinterpret_cast<const raw_t<float, VEC> *>(&in[warp][lane * VEC]), h);
    }
    // Channel c, by one thread of the block, between two barriers of the block: what every warp's rows
    // start from, given the carry before the cluster's tiles; the carry becomes the one after them.
    // `turn` counts the cluster's tiles.
    __device__ __forceinline__ void chain(int c, float &carry, int rank, int size, int turn, bool &dead, unsigned *err) {
        float h = carry;
        if (size > 1) {
            float A = 1.f, H = 0.f;
            bool set = false;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float2 m = maps[of(i)][c];
                H = map_apply(m, H);
                A *= m.x;
                set = set || map_set(m);
            }
            const int buf = turn & 1;
            const float2 mine = make_float2(set ? __uint_as_float(MAP_SET) : A, H);
            for (int to = 0; to < size; ++to) send_pair(&blocks[buf][rank][c], &bar[buf], to, mine);
            if (c == 0) mbar_arrive_expect_tx(&bar[buf], uint32_t(size * C * int(sizeof(float2))));
            // The next use of this place and of its phase is two tiles on: nobody sends there before it has
            // this block's maps of the next tile, which go out behind the barrier that ends this tile.
            if (!dead && !cluster_mbar_wait(&bar[buf], uint32_t(turn >> 1) & 1u)) {
                dead = true;
                atomicOr(err, ERR_WAIT_TIMEOUT);
            }
            float next = carry;
            for (int i = 0; i < size; ++i) {
                if (i == rank) h = next;
                next = map_apply(blocks[buf][i][c], next);
            }
            carry = next;
        }
        float t = h;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            in[of(i)][c] = t;
            t = map_apply(maps[of(i)][c], t);
        }
        if (size == 1) carry = t;
    }
    // all threads, before the first tile and behind the last one
    __device__ __forceinline__ void open(int size) {
        if (size == 1) return;
        if (threadIdx.x == 0) {
            mbar_init(&bar[0], 1);
            mbar_init(&bar[1], 1);
            fence_mbar_init();
        }
        cluster_barrier();
    }
    __device__ __forceinline__ void close(int size) {
        if (size > 1) cluster_barrier();       // no block leaves while another may still write to it
    }
};

// ------------------------------------------------------------------ forward
// Bytes of shared memory: the warps' rings, then the exchange.
template <typename T, typename G, int VEC, int R, int W, int STAGES>
struct ScanShared {
    static constexpr int RINGS = W * (Source<T, VEC, R, STAGES>::RING + Source<G, VEC, R, STAGES>::RING);
    static int bytes(int cluster) { return RINGS + Exchange<VEC, W, false>::bytes(cluster > 1); }
};

// FORM: RECUR_ bits, or -1 for those of the parameters.
template <typename T, typename G, int FORM, int VEC, int R, int W, int STAGES, int MIN>
__global__ void __launch_bounds__(W * 32, MIN) kda_gated_scan_kernel(const RecurParams p) {
    constexpr int TILE = R * W, AHEAD = STAGES > 0 ? STAGES - 1 : 1;
    constexpr bool FULL = sizeof(G) == 4;
    static_assert(RECUR_CHUNK % R == 0 && R <= 16, "chunk states lie at warps' first rows");
    using Ex = Exchange<VEC, W, false>;
    extern __shared__ __align__(16) unsigned char shared[];
    Ex &ex = *reinterpret_cast<Ex *>(shared + ScanShared<T, G, VEC, R, W, STAGES>::RINGS);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = cluster_rank(), size = cluster_size();
    const int slab = int(blockIdx.y) * 32 * VEC, col = slab + lane * VEC, part = blockIdx.z, parts = gridDim.z;
    const int form = FORM < 0 ? p.form : FORM;
    const bool in = col < p.D;
    pdl_wait();
    int begin, end;
    part_rows(p, part, parts, lane, begin, end);
    const int tile0 = begin / TILE, tiles = end > begin ? (end - 1) / TILE + 1 - tile0 : 0;
    const int turns = (tiles + size - 1) / size;
    Source<T, VEC, R, STAGES> xs;
    Source<G, VEC, R, STAGES> gs;
    xs.ring = shared + warp * (xs.RING + gs.RING);
    gs.ring = xs.ring + xs.RING;
    auto first_row = [&](int turn) { return (tile0 + turn * size + rank) * TILE + warp * R; };
    auto fetch = [&](int turn, int stage) {
        if (turn < turns) {
            const int row0 = first_row(turn);
            const unsigned live = live_bits<R>(row0, begin, end);
            xs.fetch(p.x, p.ldx, row0, live, p.D, slab, lane, stage);
            gs.fetch(p.g, p.ldg, row0, live, p.D, slab, lane, stage);
        }
        tile_sent<STAGES>();
    };
    Near near;
    float carry = 0.f;                                      // of channel threadIdx.x
    bool dead = false;
    for (int i = 0; i < AHEAD; ++i) fetch(i, i);
    ex.open(size);
    int stage = 0, next = AHEAD % (STAGES > 0 ? STAGES : 1);
    for (int turn = 0; turn < turns; ++turn) {
        const int row0 = first_row(turn);
        float a[R][VEC], b[R][VEC];
        if constexpr (STAGES > 0) {                        // the tile read in the last turn makes room
            fetch(turn + AHEAD, next);
            next = next + 1 == STAGES ? 0 : next + 1;
        }
        tile_ready<STAGES>();
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float c[VEC];
            xs.value(j, b[j], lane, stage);
            gs.value(j, a[j], lane, stage);
            decays<FULL, VEC>(form, a[j], c);
            if (form & RECUR_COMPLEMENT) mul_to<VEC>(b[j], b[j], c);
        }
        if constexpr (STAGES > 0) {
            __syncwarp();
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        } else {
            fetch(turn + 1, 0);
        }
        const Rows rows = look_at<R>(p, near, row0, begin, end, lane);
        float start[VEC] = {};                              // the state before the first row, where that starts a sequence
        float A[VEC], H[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = a[0][v], H[v] = b[0][v];
        if (rows.starts != 0) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) H[v] = 0.f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const bool starts = rows.starts >> j & 1u;
                if (starts) {
                    load_state<VEC>(H, p.state_in, recur_entry(p, sequence_of(p, near, row0 + j, lane)), p.D, col);
                    if (j == 0) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) start[v] = H[v];
                    }
                }
                fma_to<VEC>(H, a[j], H, b[j]);
                if (starts) {                              // what follows takes b as the row's state: state_in may be
#pragma unroll                                                     // overwritten by then
                    for (int v = 0; v < VEC; ++v) b[j][v] = H[v];
                }
            }
        } else {
#pragma unroll
            for (int j = 1; j < R; ++j) {
                fma_to<VEC>(H, a[j], H, b[j]);
                mul_to<VEC>(A, A, a[j]);
            }
        }
        ex.put(warp, lane, A, H, rows.starts != 0);
        __syncthreads();
        if (threadIdx.x < Ex::C) ex.chain(threadIdx.x, carry, rank, size, turn, dead, p.err);
        __syncthreads();
        if (rows.live == 0) continue;
        float h[VEC];
        ex.get(warp, lane, h);
        if (p.chunk != nullptr && row0 % RECUR_CHUNK == 0 && (rows.live & 1u))
            store_state<VEC>(rows.starts & 1u ? start : h, p.chunk, row0 / RECUR_CHUNK, p.D, col);
        T *y = static_cast<T *>(p.y) + int64_t(row0) * p.D + col;
        if ((rows.starts | rows.lasts) == 0 && rows.live == (1u << R) - 1u) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                fma_to<VEC>(h, a[j], h, b[j]);
                if (in) store_raw<T, VEC>(y, narrow<T, VEC>(h));
                y += p.D;
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool starts = rows.starts >> j & 1u;
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = starts ? b[j][v] : fmaf(a[j][v], h[v], b[j][v]);
            if (in && (rows.live >> j & 1u)) store_raw<T, VEC>(y + int64_t(j) * p.D, narrow<T, VEC>(h));
            if (rows.lasts >> j & 1u)
                store_state<VEC>(h, p.state_out, recur_entry(p, sequence_of(p, near, row0 + j, lane)), p.D, col);
        }
    }
    pdl_launch_dependents();
    copy_empty<VEC>(p, p.state_in, p.state_out, (part * size + rank) * W + warp, parts * size * W, lane, col);
    ex.close(size);
}

// ----------------------------------------------------------------- backward
// Forwards the exchange stays in the block, since a tile is a chunk.
template <typename T, typename X, typename S, int VEC, int R, int W, int STAGES>
struct GradShared {
    static constexpr int RINGS = W * (Source<X, VEC, R, STAGES>::RING + Source<S, VEC, R, STAGES>::RING +
                                      Source<T, VEC, R, STAGES>::RING);
    static constexpr int FORTH = Exchange<VEC, W, false>::bytes(false);
    static int bytes(int cluster) { return RINGS + FORTH + Exchange<VEC, W, true>::bytes(cluster > 1); }
};

// T: dy, dx; X, S: x and g, or int8_t for codes; G: dg.
template <typename T, typename X, typename S, typename G, int FORM, int VEC, int R, int W, int STAGES, int MIN>
__global__ void __launch_bounds__(W * 32, MIN) kda_gated_scan_backward_kernel(const RecurParams p) {
    constexpr int TILE = R * W, AHEAD = STAGES > 0 ? STAGES - 1 : 1;
    constexpr bool FULL = sizeof(S) == 4;
    static_assert(TILE == RECUR_CHUNK && R * VEC <= 32, "a tile is a chunk");
    using Shared = GradShared<T, X, S, VEC, R, W, STAGES>;
    using Forth = Exchange<VEC, W, false>;
    using Ex = Exchange<VEC, W, true>;
    extern __shared__ __align__(16) unsigned char shared[];
    Forth &forth = *reinterpret_cast<Forth *>(shared + Shared::RINGS);
    Ex &ex = *reinterpret_cast<Ex *>(shared + Shared::RINGS + Shared::FORTH);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = cluster_rank(), size = cluster_size();
    const int slab = int(blockIdx.y) * 32 * VEC, col = slab + lane * VEC, part = blockIdx.z, parts = gridDim.z;
    const int form = FORM < 0 ? p.form : FORM;
    const bool in = col < p.D, complement = form & RECUR_COMPLEMENT;
    pdl_wait();
    int begin, end;
    part_rows(p, part, parts, lane, begin, end);
    const int tile0 = begin / TILE, tiles = end > begin ? (end - 1) / TILE + 1 - tile0 : 0;
    const int turns = (tiles + size - 1) / size;
    Source<X, VEC, R, STAGES> xs;
    Source<S, VEC, R, STAGES> gs;
    Source<T, VEC, R, STAGES> ds;
    xs.ring = shared + warp * (xs.RING + gs.RING + ds.RING);
    gs.ring = xs.ring + xs.RING;
    ds.ring = gs.ring + gs.RING;
    // tiles from the last one back; those before the part's first have no live rows
    auto tile_of = [&](int turn) { return tile0 + tiles - 1 - (turn * size + rank); };
    auto live_of = [&](int turn) {
        return turn < turns && tile_of(turn) >= tile0 ? live_bits<R>(tile_of(turn) * TILE + warp * R, begin, end) : 0u;
    };
    auto fetch = [&](int turn, int stage) {
        if (turn < turns) {
            const int row0 = tile_of(turn) * TILE + warp * R;
            const unsigned live = live_of(turn);
            xs.fetch(p.x, p.ldx, row0, live, p.D, slab, lane, stage);
            gs.fetch(p.g, p.ldg, row0, live, p.D, slab, lane, stage);
            ds.fetch(p.dy, p.lddy, row0, live, p.D, slab, lane, stage);
        }
        tile_sent<STAGES>();
    };
    // one turn ahead: exponents, and the chunk's state for the tile's first warp
    unsigned xscales = 0, gscales = 0;
    float chunk[VEC];
    auto fetch_small = [&](int turn) {
        const int row0 = tile_of(turn) * TILE + warp * R;
        const unsigned live = live_of(turn);
        xscales = xs.fetch_scales(p.xe, row0, live, p.D, slab, lane);
        gscales = gs.fetch_scales(p.ge, row0, live, p.D, slab, lane);
        load_state<VEC>(chunk, p.chunk, warp == 0 && (live & 1u) ? tile_of(turn) : -1, p.D, col);
    };
    Near near;
    float carry = 0.f, none = 0.f;                          // of channel threadIdx.x
    bool dead = false;
    for (int i = 0; i < AHEAD; ++i) fetch(i, i);
    fetch_small(0);
    ex.open(size);
    int stage = 0, next = AHEAD % (STAGES > 0 ? STAGES : 1);
    for (int turn = 0; turn < turns; ++turn) {
        const int row0 = tile_of(turn) * TILE + warp * R;
        // x: in the end h before the row, less x where c = 1 - a
        float a[R][VEC], rest[R][VEC], x[R][VEC], d[R][VEC], h[VEC];
        if constexpr (STAGES > 0) {
            fetch(turn + AHEAD, next);
            next = next + 1 == STAGES ? 0 : next + 1;
        }
        tile_ready<STAGES>();
        xs.set_scales(xscales);
        gs.set_scales(gscales);
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = chunk[v];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            xs.value(j, x[j], lane, stage);
            gs.value(j, a[j], lane, stage);
            ds.value(j, d[j], lane, stage);
            decays<FULL, VEC>(form, a[j], rest[j]);
        }
        if constexpr (STAGES > 0) {
            __syncwarp();
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        } else {
            fetch(turn + 1, 0);
        }
        fetch_small(turn + 1);
        Rows rows{0, 0, 0};
        if (live_of(turn) != 0) rows = look_at<R>(p, near, row0, begin, end, lane);
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
        auto edge = [&](float (&s)[VEC], const float *base, int j) {
            load_state<VEC>(s, base, recur_entry(p, sequence_of(p, near, row0 + j, lane)), p.D, col);
        };
        float A[VEC], H[VEC], E[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = a[0][v], H[v] = h[v], E[v] = 0.f;
        // forwards; a first row's state is looked up here and once more below, where it is in the cache
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (rows.starts >> j & 1u) edge(H, p.state_in, j);
            step(H, j);
            if (j > 0) mul_to<VEC>(A, A, a[j]);
        }
        // backwards
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            if (rows.lasts >> j & 1u) edge(E, p.dfinal, j);
            add_to<VEC>(E, E, d[j]);
            mul_to<VEC>(E, E, a[j]);
        }
        forth.put(warp, lane, A, H, warp == 0 || rows.starts != 0);
        ex.put(warp, lane, A, E, rows.lasts != 0);
        __syncthreads();
        if (threadIdx.x < Ex::C) ex.chain(threadIdx.x, carry, rank, size, turn, dead, p.err);
        else if (threadIdx.x < 2 * Ex::C) forth.chain(threadIdx.x - Ex::C, none, 0, 1, 0, dead, p.err);
        __syncthreads();
        if (rows.live == 0) continue;
        float e[VEC];
        ex.get(warp, lane, e);
        if (warp > 0) forth.get(warp, lane, h);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (rows.starts >> j & 1u) edge(h, p.state_in, j);
            float was[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) was[v] = h[v];
            if (j < R - 1) step(h, j);
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[j][v] = complement ? was[v] - x[j][v] : was[v];
        }
        T *dx = static_cast<T *>(p.dx) + int64_t(row0) * p.D + col;
        G *dg = static_cast<G *>(p.dg) + int64_t(row0) * p.D + col;
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            if (rows.lasts >> j & 1u) edge(e, p.dfinal, j);
            float dh[VEC], og[VEC];
            add_to<VEC>(dh, d[j], e);
            mul_to<VEC>(e, a[j], dh);
            mul_to<VEC>(og, e, x[j]);
            if (form & RECUR_SIGMOID) mul_to<VEC>(og, og, rest[j]);
            if (complement) mul_to<VEC>(dh, rest[j], dh);
            if (in && (rows.live >> j & 1u)) {
                store_raw<T, VEC>(dx + int64_t(j) * p.D, narrow<T, VEC>(dh));
                store_raw<G, VEC>(dg + int64_t(j) * p.D, narrow<G, VEC>(og));
            }
            if (p.dinitial != nullptr && (rows.starts >> j & 1u))
                store_state<VEC>(e, p.dinitial, recur_entry(p, sequence_of(p, near, row0 + j, lane)), p.D, col);
        }
    }
    pdl_launch_dependents();
    copy_empty<VEC>(p, p.dfinal, p.dinitial, (part * size + rank) * W + warp, parts * size * W, lane, col);
    ex.close(size);
}

}  // namespace kda
