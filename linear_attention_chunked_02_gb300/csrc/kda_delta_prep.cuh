// kda_delta_prep.cuh -- what the chunked gated delta rule needs of a chunk before
// its state is known: for every 64-token chunk and head, from q, k, g and beta,
//
//   A_ij = beta_i sum_d k_id k_jd e^{G_id - G_jd}  (j < i),   M = (I + A)^-1 diag(beta),
//   P_ij = scale sum_d q_id k_jd e^{G_id - G_jd}   (j <= i),
//
// with G the cumulative log decay inside the chunk.  All chunk-heads are
// independent.  M and P go to the workspace as the operand images that
// kda_delta_scan.cuh multiplies with.
//
// One product for both.  With E = G - G_31 (the reference in the chunk's middle),
//   [A; P] = [K e^E; Q e^E] (K e^{-E})^T,
// a 128 x 64 product over the channels on tcgen05, FP32 accuracy from TF32 as in the
// fused construction kernel (hi hi + hi lo + lo hi).  E is summed outward from the
// middle, so that it is exact to FP32 of its own size where it matters.  A channel
// whose decay over either half of the chunk exceeds PREP_SAFE nats is left out of
// the product and its terms are added one by one, with running products of e^g.
//
// Shared memory is what bounds this: a version with both operands there moved 7000
// 128-byte wavefronts for a chunk-head, a third of them the tensor core's reads of the
// 128-row side.  So that side goes to tensor memory, written by threads that own its
// rows, and the images leave by bulk copies from shared memory (stores of 16 bytes
// a lane had taken 50 of 320 us at 16 x 512 tokens x 64 heads).
//
// One persistent CTA of seven warpgroups per SM; every role walks the same chunk-heads:
//   * warps 2 and 3 of the first CTA: the scan's list of segments, from cu_seqlens;
//   * warp 0: MMA issue; warp 1: TMA loads of k, q and g in slices of 32 channels into a
//     ring, swizzled so that both passes of the transform read them without conflicts;
//   * warps 8-15 and 16-23 (transform): every second slice each.  First a thread has four rows of two
//     channels: E, summed in registers with one exchange of eight totals to a channel, takes
//     g's place.  Then lane = row: K e^E and Q e^E to tensor memory, K e^{-E} to shared;
//   * warps 4, 5 (A) and 6, 7 (P): the accumulator's rows out of tensor memory; A
//     with beta and the mask into the solve's tile, P into its image;
//   * warps 24-27: two pairs, each the 64-token solve of every second chunk-head,
//     and M's image.
// 16 x 512 tokens x 64 heads of BF16, K = 128: 203 us and 770 MB, 3.8 TB/s.  What bounds it is issue: 162
// million warp instructions, 70 % of the slots; the transform groups and the solve pairs
// are both busy nearly all the time (7400 and 6500 cycles to a chunk-head).
// Five kinds of code run at once on an SM whose instruction cache holds about 32 KB of
// them: with everything unrolled (100 KB) half the cache's requests missed and
// that, not any pipe, set the time (424 us under the profiler, 16 x 512 tokens x 64
// heads).  So the loops here are kept rolled wherever registers allow it.
#pragma once

#include "kda_delta_rec.cuh"
#include "kda_kgb.cuh"

namespace kda {

// Image of one chunk-head in the workspace.  M and P are FP16 pairs hi + lo (22
// bits) scaled by a power of two for each half of 32 rows, 64 rows of 128
// bytes with the 128-byte swizzle: the B operands of the scan's products.
constexpr int IMG_MHI = 0, IMG_MLO = 8192, IMG_PHI = 16384, IMG_PLO = 24576, IMG_HDR = 32768;
constexpr int IMG_HDR_BYTES = 128, IMG_BYTES = IMG_HDR + IMG_HDR_BYTES;
// header (floats): 1 / scale of M rows 0-31, 32-63; largest row sum of |M| in the halves;
// 1 / scale of P in the halves; largest |k|, |q|; and, from the walk that finds a segment's M, the largest
// channel's decay over the chunk
constexpr int HDR_MINV = 0, HDR_MSUM = 2, HDR_PINV = 4, HDR_KMAX = 6, HDR_QMAX = 7, HDR_GMAX = 8;

constexpr int PREP_THREADS = 28 * 32, PREP_REGISTERS = 72;     // per thread at launch
constexpr int PREP_TW = 8;                         // transform warps of a group
constexpr float PREP_SAFE = 48.0f;
// The slices of a chunk go to the two transform groups in turn.  Each group has buffers of
// its own, so that all who wait on a buffer's barrier take part in every one of its phases
// (a group that skipped two phases would take the barrier's parity for its turn).
constexpr int PREP_NOPS = 2;                       // slices' operands, a group's: 64 TMEM columns and, in shared memory,
constexpr int PREP_OPS_BYTES = 16 * 1024;          // K e^{-E} hi and lo, 64 rows of 128 bytes each
// staging ring: a slice of 64 rows x 32 channels of k, q and g
template <typename T>
constexpr int prep_stage_bytes() { return 2 * 64 * 32 * int(sizeof(T)) + 8192; }
template <typename T>
constexpr int prep_stages() { return sizeof(T) == 2 ? 2 : 1; }     // of a group
constexpr int PB_OPS_FULL = 0, PB_OPS_EMPTY = PREP_NOPS, PB_D_FULL = 2 * PREP_NOPS, PB_D_EMPTY = PB_D_FULL + 2,
              PB_AT_FULL = PB_D_EMPTY + 2, PB_AT_EMPTY = PB_AT_FULL + 2, PB_ST_FULL = PB_AT_EMPTY + 2,
              PB_ST_EMPTY = PB_ST_FULL + 4, PREP_NBARS = PB_ST_EMPTY + 4;
constexpr int PREP_OFF_TMEM = PREP_NBARS * 8;
constexpr int PREP_OFF_STEEP = 256;                // [8 chunk-heads][4 slices]
constexpr int PREP_OFF_KQ = PREP_OFF_STEEP + 8 * 4 * 4;        // [8 chunk-heads][16 warps] largest |k| or |q|
constexpr int PREP_OFF_HALF = PREP_OFF_KQ + 8 * 16 * 4;        // [2 groups][2] steep channels by half
constexpr int PREP_OFF_META = PREP_OFF_HALF + 2 * 2 * 4;       // [4 stages] rows, first row, head
constexpr int PREP_OFF_TOT = 1024;                 // [2 groups][8 warps][32 channels] sums of g
constexpr int PREP_OFF_SC = PREP_OFF_TOT + 2 * 8 * 32 * 4;     // slow path: e^g, k of a channel, for A and for P
constexpr int PREP_OFF_BETA = PREP_OFF_SC + 2 * 64 * 8;        // [pairs][64]
constexpr int PREP_OFF_CU = PREP_OFF_BETA + 2 * 64 * 4;
constexpr int PREP_OFF_OPS = 6 * 1024;
constexpr int PREP_OFF_ST = PREP_OFF_OPS + PREP_NOPS * PREP_OPS_BYTES;
constexpr int PREP_XP = 68;                        // pitch of the solved tile (floats)
constexpr int PREP_X_FLOATS = 6 * XTS + 3 * XRS;   // transposed inverse blocks, negated diagonal ones
// after the staging ring: the solve's tiles, its inverse tiles, the solved tiles, M's images, P's image
template <typename T>
constexpr int prep_off_at() { return PREP_OFF_ST + 2 * prep_stages<T>() * prep_stage_bytes<T>(); }
template <typename T>
constexpr int prep_off_x() { return prep_off_at<T>() + 2 * 10 * 256 * 4; }
template <typename T>
constexpr int prep_off_xs() { return prep_off_x<T>() + 2 * PREP_X_FLOATS * 4; }
template <typename T>
constexpr int prep_off_m() { return prep_off_xs<T>() + 2 * 64 * PREP_XP * 4; }
template <typename T>
constexpr int prep_off_p() { return prep_off_m<T>() + 2 * 16384; }
template <typename T>
constexpr int prep_bytes() { return prep_off_p<T>() + 16384 + 1024; }
static_assert(PREP_OFF_TMEM + 4 <= PREP_OFF_STEEP && PREP_OFF_META + 4 * 16 <= PREP_OFF_TOT, "header fits");
static_assert(PREP_OFF_CU + CU_CAP * 4 <= PREP_OFF_OPS, "cu_seqlens fits");
static_assert(prep_stage_bytes<float>() % 1024 == 0 && prep_stage_bytes<__half>() % 1024 == 0 &&
                  prep_bytes<float>() <= 227 * 1024 && prep_bytes<__half>() <= 227 * 1024,
              "fits the shared memory of one CTA");
constexpr uint32_t PREP_TM_D = 0, PREP_TM_A = 128; // accumulators [2][64], operands [PREP_NOPS]{hi 32, lo 32}
constexpr uint32_t PREP_TM_FINE = 256;             // from an accumulator to its own for the small products

// Tensor maps of q, k [rows, Hk, K] and g [rows, H, K] as {channels, heads, rows}: boxes of 32
// channels x 64 rows here, swizzled over their row's bytes; of all channels (and of v's
// values) in the scan.
struct DeltaMaps {
    CUtensorMap q, k, g, v;
};

// Power-of-two scale that brings values of at most `bound` below 2^15, within FP16;
// the exponent is kept in [lo, hi] so that products of two scales and their
// inverses stay normal.  `inv` is its exact inverse.
__device__ __forceinline__ float pow2_scale(float bound, int lo, int hi, float &inv) {
    int e = 14 - (int((__float_as_uint(bound) >> 23) & 255u) - 127);
    e = e < lo ? lo : e > hi ? hi : e;
    inv = __uint_as_float(uint32_t(127 - e) << 23);
    return __uint_as_float(uint32_t(127 + e) << 23);
}
constexpr int KQ_LO = -26, KQ_HI = 40;             // exponents for keys, queries, M and P
constexpr int VS_LO = -100, VS_HI = 80;            // for states and values

// Two values as FP16 hi and lo parts, x ~ hi + lo to 2^-22 (x - hi is exact).
__device__ __forceinline__ void split_f16(float a, float b, uint32_t &hi, uint32_t &lo) {
    asm("{\n\t.reg .b16 h0, h1, m;\n\t.reg .f32 x, y;\n\t"
        "cvt.rn.f16x2.f32 %0, %3, %2;\n\t"
        "mov.b32 {h0, h1}, %0;\n\t"
        "mov.b16 m, 0xBC00;\n\t"                    // -1
        "fma.rn.f32.f16 x, h0, m, %2;\n\t"
        "fma.rn.f32.f16 y, h1, m, %3;\n\t"
        "cvt.rn.f16x2.f32 %1, y, x;\n\t}"
        : "=r"(hi), "=r"(lo)
        : "f"(a), "f"(b));
}

// Largest of m and |a|, |b|.
__device__ __forceinline__ float max3(float m, float a, float b) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

// Eight channels d .. d + 7 (a multiple of 8) of row r of a staged slice, as the tensor map's
// swizzle over the row's bytes (64 or 128) left them.
template <typename T>
__device__ __forceinline__ void load_row(const unsigned char *tile, int r, int d, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 t = *reinterpret_cast<const uint4 *>(tile + r * 64 + 16 * ((d >> 3) ^ ((r >> 1) & 3)));
        Elt<T>::widen(t, x);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 t = *reinterpret_cast<const float4 *>(tile + r * 128 + 16 * (((d >> 2) + j) ^ (r & 7)));
            x[4 * j] = t.x; x[4 * j + 1] = t.y; x[4 * j + 2] = t.z; x[4 * j + 3] = t.w;
        }
    }
}

__device__ __forceinline__ float warp_max(float v) {   // v >= 0
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// Columns 8 c .. + 7 of row i of an image tile, times s: hi and lo.
__device__ __forceinline__ void image_put(unsigned char *hi, unsigned char *lo, int i, int c, const float (&x)[8], float s) {
    uint4 h, l;
    split_f16(x[0] * s, x[1] * s, h.x, l.x);
    split_f16(x[2] * s, x[3] * s, h.y, l.y);
    split_f16(x[4] * s, x[5] * s, h.z, l.z);
    split_f16(x[6] * s, x[7] * s, h.w, l.w);
    const int at = i * 128 + 16 * (c ^ (i & 7));
    *reinterpret_cast<uint4 *>(hi + at) = h;
    *reinterpret_cast<uint4 *>(lo + at) = l;
}

// The 64-token solve of the A tile (blocks (i, j) at Ab + 256 blk(i, j)) by two warps: the row-major
// M = (I + A)^-1 diag(beta) into xs (its blocks above the diagonal are not written); `beta` is row pt's,
// sbeta all of them from the first barrier on.  Block by block along
// the diagonals, X_rc = -X_rr sum_k A_rk X_kc, transposed and in split TF32 as in the chunk
// solver; one loop body does every product, where the chunk solver unrolls its two levels.
__device__ __forceinline__ void prep_solve(const float *Ab, float *X, float *xs, float beta, const float *sbeta, int pt,
                                           int bar) {
    const int warp = pt >> 5, lane = pt & 31, g = lane >> 2, t = lane & 3;
    float *Xn = X + 6 * XTS;
    {
        const int b = pt >> 4, l = pt & 15;
        float x[16];
        diag_invert<true>(Ab + blk(b, b) * 256, 16, l, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) xs[(16 * b + i) * PREP_XP + 16 * b + l] = x[i] * beta;
        if (b != 3) {                                      // X_bb^T row-major (row = lane)
            float4 *d = reinterpret_cast<float4 *>(X + blk(b, b) * XTS + l * XTP);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i ^ xt_swz(l)] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
        if (b != 0) {                                      // -X_bb row-major (column = lane)
            float *d = Xn + (b - 1) * XRS + l;
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i * XRP] = -x[i];
        }
    }
    bar64(bar);
#pragma unroll 1
    for (int c = warp; c < 3; c += warp == 0 ? 3 : 1) {    // 9 tile products against 7
#pragma unroll 1
        for (int r = c + 1; r < 4; ++r) {
            TileA la;
            TileB rb;
            TileC acc, out;
            zero(acc);
            zero(out);
#pragma unroll 1
            for (int k = c; k < r; ++k) {
                left_smem<true>(la, X + blk(k, c) * XTS, XTP, g, t);
                right4<false>(rb, Ab + blk(r, k) * 256, 16, g, t);
                mma_tile<false>(acc, la, rb);
            }
            left_regs(la, acc);
            right2(rb, Xn + (r - 1) * XRS, XRP, g, t);
            mma_tile<false>(out, la, rb);
            if (r < 3) smem_tile_t<true>(X + blk(r, c) * XTS, out, g, t);
            const float b0 = sbeta[16 * c + g], b1 = sbeta[16 * c + g + 8];    // the tile is transposed
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) out.c[nt][e] *= e < 2 ? b0 : b1;
            out_tile_t(xs, PREP_XP, BT, r, c, out, g, t);
            __syncwarp();
        }
    }
    bar64(bar);
}

// A wait that gives up once, after WAIT_TRIES tries: the thread then records it and waits no more, but
// keeps arriving, so that no other thread is stranded.  A try suspends the warp until the phase ends
// or some 4 us have passed (polling takes issue slots from the warps at work), so that the tries make
// about a second; each of these waits ends within microseconds, or some hundred where a chunk goes the
// slow way.  No clock is read: a wait is a few instructions, which matters here (the kernels' loops
// fill the instruction cache; with a clock in every wait the two
// kernels of 16 x 512 x 64 heads took 221 and 265 us, without 204 and 257).
constexpr uint32_t WAIT_TRIES = 1u << 18;
__device__ __forceinline__ void prep_wait(bool &ok, uint64_t *bar, uint32_t parity, unsigned *err) {
    if (!ok) return;
    uint32_t left = WAIT_TRIES;
#pragma unroll 1
    while (!mbar_try_wait_suspend(bar, parity, 100000u))
        if (--left == 0u) {
            ok = false;
            atomicOr(err, ERR_WAIT_TIMEOUT);
            return;
        }
}

// The segments that the scan walks, {sequence, segment of it, chunks before the sequence, its
// segments} each (the last is 0 past the end), from cu_seqlens by threads t = 0 .. 63.  Whole
// sequences go longest first where there are at most SORTED of them, so that a
// long one does not start last; segments stay in order.
constexpr int PREP_SORTED = 128;
__device__ __forceinline__ void list_units(const DeltaParams &p, int t) {
    const int lane = t & 31;
    if (p.seg == 0 && p.nseq <= PREP_SORTED) {
#pragma unroll 1
        for (int i = t; i < p.nseq; i += 64) {
            const int32_t mine = max(0, p.cu[i + 1] - p.cu[i]);
            int32_t rank = 0, before = 0, a = p.cu[0];
#pragma unroll 1
            for (int j = 0; j < p.nseq; ++j) {
                const int32_t b = p.cu[j + 1], len = max(0, b - a);
                rank += len > mine || (len == mine && j < i);
                before += j < i ? (len + BT - 1) / BT : 0;
                a = b;
            }
            p.units[rank] = make_int4(i, 0, before, 1);
        }
        return;
    }
    if (t >= 32) return;
    // a lane has consecutive sequences; first their totals, then the entries
    const int per = (p.nseq + 31) / 32, i0 = min(p.nseq, lane * per), i1 = min(p.nseq, i0 + per);
    int32_t units = 0, chunks = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const int32_t nc = nchunks<BT>(p.cu[i], p.cu[i + 1]), nu = p.seg > 0 ? max(1, (nc + p.seg - 1) / p.seg) : 1;
            if (pass == 1)
                for (int j = 0; j < nu; ++j)
                    if (units + j < p.n_units) p.units[units + j] = make_int4(i, j, chunks, nu);
            units += nu;
            chunks += nc;
        }
        if (pass == 0) {
            int32_t su = units, sc = chunks;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t a = __shfl_up_sync(0xffffffffu, su, o), b = __shfl_up_sync(0xffffffffu, sc, o);
                if (lane >= o) {
                    su += a;
                    sc += b;
                }
            }
            const int32_t all = __shfl_sync(0xffffffffu, su, 31);
            for (int32_t i = max(0, all) + lane; i < p.n_units; i += 32) p.units[i] = make_int4(0, 0, 0, 0);
            units = su - units;
            chunks = sc - chunks;
            if (units < 0) return;                         // malformed cu_seqlens
        }
    }
}

// FP32 inputs need more of the TF32 products than 16-bit ones, whose own rounding is far above this:
// the instruction cuts the operands that it reads and cuts its sums as it adds to them, so that all
// parts err toward zero.  FINE rounds high and low parts to nearest, and gives the small products an
// accumulator of their own (16 sums at the accumulator's full size for K = 128, not 48).  P, 64 tokens
// of K = 128, against 64 bits: 1.0e-6 with rounded parts alone, 3.6e-7 with both.
template <typename T>
constexpr bool prep_fine() { return sizeof(T) == 4; }
template <bool FINE>
__device__ __forceinline__ void prep_split(float2 v, uint32_t &h0, uint32_t &h1, uint32_t &l0, uint32_t &l1) {
    if (!FINE) return split2(v, h0, h1, l0, l1);
    h0 = (__float_as_uint(v.x) + 0x1000u) & 0xffffe000u;
    h1 = (__float_as_uint(v.y) + 0x1000u) & 0xffffe000u;
    const float2 lo = __fadd2_rn(v, make_float2(-__uint_as_float(h0), -__uint_as_float(h1)));
    l0 = __float_as_uint(lo.x) + 0x1000u;
    l1 = __float_as_uint(lo.y) + 0x1000u;
}

template <typename T>
__global__ void __launch_bounds__(PREP_THREADS, 1) kda_delta_prep_kernel(const __grid_constant__ DeltaMaps maps, const DeltaParams p) {
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + PREP_OFF_TMEM);
    uint32_t *steep_m = reinterpret_cast<uint32_t *>(sm + PREP_OFF_STEEP);
    float *kq_m = reinterpret_cast<float *>(sm + PREP_OFF_KQ);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int NST = prep_stages<T>(), STB = prep_stage_bytes<T>(), ST_Q = 64 * 32 * int(sizeof(T)), ST_G = 2 * ST_Q;
    const int nsl = p.K / 32;
    const int32_t G = gridDim.x;
    const int group = p.H / p.Hk;
    pdl_launch_dependents();

    if (tid == 0) {
        for (int b = 0; b < 2 * NST; ++b) {
            mbar_init(&bars[PB_ST_FULL + b], 1);
            mbar_init(&bars[PB_ST_EMPTY + b], PREP_TW);
        }
        for (int b = 0; b < PREP_NOPS; ++b) {
            mbar_init(&bars[PB_OPS_FULL + b], PREP_TW);
            mbar_init(&bars[PB_OPS_EMPTY + b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars[PB_D_FULL + b], 2);
            mbar_init(&bars[PB_D_EMPTY + b], 4);
            mbar_init(&bars[PB_AT_FULL + b], 2);
            mbar_init(&bars[PB_AT_EMPTY + b], 2);
        }
        fence_mbar_init();
    }
    pdl_wait();
    DeltaParams ps = p;
    if (p.cu != nullptr && p.nseq < CU_CAP) {
        int32_t *cs = reinterpret_cast<int32_t *>(sm + PREP_OFF_CU);
        for (int i = tid; i <= p.nseq; i += PREP_THREADS) cs[i] = __ldg(p.cu + i);
        ps.cu = cs;
    }
    if (warp == 4) {
        tc::tmem_alloc(smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    static_assert(32 + 104 + 4 * 64 + 112 <= PREP_THREADS / 128 * PREP_REGISTERS, "the groups' shares");
    if (warp < 4) {
        tc::fewer_registers<32>();
        if (warp == 0) {
            // ------------------------------------------------------------- MMA issue
            TaskWalk w(ps, blockIdx.x, G);
            uint32_t turn[2] = {0u, 0u};                   // slices of each group so far
            for (uint32_t c = 0; w.next(ps).valid; ++c) {
                const int db = c & 1;
                prep_wait(ok, &bars[PB_D_EMPTY + db], ((c >> 1) & 1) ^ 1, p.err);
                for (int s = 0; s < nsl; ++s) {
                    const int ob = s & 1;
                    prep_wait(ok, &bars[PB_OPS_FULL + ob], (ob ? turn[1]++ : turn[0]++) & 1, p.err);
                    __syncwarp();
                    tc::fence_after_sync();
                    const uint32_t bh = smem_u32(sm + PREP_OFF_OPS + ob * PREP_OPS_BYTES);
                    const uint32_t d = tmem + PREP_TM_D + db * 64;
                    if (tc::elect_one()) {
                        // K = 8 channels: 8 columns of A, 32 bytes along B's rows
                        uint32_t ta = tmem + PREP_TM_A + ob * 64;
                        uint64_t dbh = tc::sw128_desc(bh), dbl = tc::sw128_desc(bh + 8192);
#pragma unroll 1
                        for (int kk = 0; kk < 4; ++kk) {
                            tc::mma_tf32_ts(d, ta, dbh, KGB_IDESC, s > 0 || kk > 0);
                            if (prep_fine<T>()) {
                                tc::mma_tf32_ts(d + PREP_TM_FINE, ta, dbl, KGB_IDESC, s > 0 || kk > 0);
                                tc::mma_tf32_ts(d + PREP_TM_FINE, ta + 32, dbh, KGB_IDESC, true);
                            } else {
                                tc::mma_tf32_ts(d, ta, dbl, KGB_IDESC, true);
                                tc::mma_tf32_ts(d, ta + 32, dbh, KGB_IDESC, true);
                            }
                            ta += 8;
                            dbh += 2;
                            dbl += 2;
                        }
                        tc::commit(smem_u32(&bars[PB_OPS_EMPTY + ob]));
                        if (s == nsl - 1) {
                            tc::commit(smem_u32(&bars[PB_D_FULL + db]));
                            mbar_arrive(&bars[PB_D_FULL + db]);    // releases the steep masks and maxima
                        }
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1) {
            // ----------------------------------------------------------------- loads
            TaskWalk w(ps, blockIdx.x, G);
            uint32_t turn[2] = {0u, 0u};
            Meta nx;
            for (Meta m = w.next(ps); m.valid; m = nx) {
                nx = w.next(ps);
                for (int s = 0; s < nsl; ++s) {
                    const uint32_t u = s & 1 ? turn[1]++ : turn[0]++;
                    const int st = (s & 1) * NST + u % NST;
                    prep_wait(ok, &bars[PB_ST_EMPTY + st], ((u / NST) & 1) ^ 1, p.err);
                    __syncwarp();
                    if (tc::elect_one()) {
                        unsigned char *to = sm + PREP_OFF_ST + st * STB;
                        uint64_t *full = &bars[PB_ST_FULL + st];
                        *reinterpret_cast<int4 *>(sm + PREP_OFF_META + 16 * st) = make_int4(m.n, m.row0, m.h, 0);
                        mbar_arrive_expect_tx(full, 2 * ST_Q + (p.gate == 0 ? 8192 : 0));
                        tma_load_3d(to, &maps.k, 32 * s, m.h / group, m.row0, full);
                        tma_load_3d(to + ST_Q, &maps.q, 32 * s, m.h / group, m.row0, full);
                        if (p.gate == 0) tma_load_3d(to + ST_G, &maps.g, 32 * s, m.h, m.row0, full);
                        // the ring holds too little of FP32 to hide HBM: the next chunk's slice to L2 (64 x 512
                        // tokens, 32 heads, K = 128: 508 us, not 587).  Of 16 bits it holds twice as many
                        // slices, and the copies only cost (16 x 512 x 64 heads: 213 us, not 203)
                        if (NST == 1 && nx.valid) {
                            tc::prefetch_3d(&maps.k, 32 * s, nx.h / group, nx.row0);
                            tc::prefetch_3d(&maps.q, 32 * s, nx.h / group, nx.row0);
                            if (p.gate == 0) tc::prefetch_3d(&maps.g, 32 * s, nx.h, nx.row0);
                        }
                    }
                    __syncwarp();
                }
            }
            // no copy may be in flight when the CTA ends
            for (int tg = 0; tg < 2; ++tg)
                for (uint32_t i = turn[tg] > NST ? turn[tg] - NST : 0; i < turn[tg]; ++i)
                    prep_wait(ok, &bars[PB_ST_FULL + tg * NST + i % NST], (i / NST) & 1, p.err);
        } else if (blockIdx.x == 0 && p.cu != nullptr) {
            list_units(ps, tid - 64);
        }
    } else if (warp >= 8 && warp < 24) {
        tc::fewer_registers<64>();
        // -------------------------------------------------------------- transform
        constexpr float L2E = 1.4426950408889634f;
        const int tw = warp & 7, tg = (warp >> 3) - 1;     // slices tg, tg + 2
        // second pass: this thread's row of K (quarters 0, 1) or Q (2, 3), sixteen channels of it
        const int quarter = warp & 3, row = 32 * (quarter & 1) + lane, half = tw >> 2;
        const bool isQ = quarter >= 2;
        const uint32_t ta = tmem + PREP_TM_A + (uint32_t(32 * quarter) << 16) + 16 * half;
        float *tot = reinterpret_cast<float *>(sm + PREP_OFF_TOT) + tg * 256;
        uint32_t *half_steep = reinterpret_cast<uint32_t *>(sm + PREP_OFF_HALF) + tg * 2;
        // first pass: four rows of two channels
        const int cp = lane & 15, rh = lane >> 4, row_e = 8 * tw + 4 * rh;
        const bool low = tw < 4;
        const float dir = low ? -L2E : L2E;
        auto group_sync = [&] {
            if (tg == 0) named_sync<1, 256>();
            else named_sync<6, 256>();
        };
        // chunk-heads of this CTA; which they are comes with the stages (a walk takes twelve registers)
        int32_t chunks = p.n_tasks / p.H;
        if (p.cu != nullptr) {
            int32_t sum = 0;
            for (int i = lane; i < p.nseq; i += 32) sum += nchunks<BT>(ps.cu[i], ps.cu[i + 1]);
            chunks = min(chunks, __reduce_add_sync(0xffffffffu, sum));
        }
        const uint32_t own = tg < nsl ? uint32_t(max(0, (chunks * p.H - int32_t(blockIdx.x) + G - 1) / G)) : 0u;
        uint32_t turn = 0;
        for (uint32_t c = 0; c < own; ++c) {
            float big = 0.f;                               // largest |k| or |q| seen
            for (int s = tg; s < nsl; s += 2, ++turn) {
                const int ob = tg, st = tg * NST + turn % NST;
                unsigned char *stage = sm + PREP_OFF_ST + st * STB;
                prep_wait(ok, &bars[PB_ST_FULL + st], (turn / NST) & 1, p.err);
                const int4 *meta = reinterpret_cast<const int4 *>(sm + PREP_OFF_META + 16 * st);
                const int n = ok ? meta->x : 0;
                // ---- E in g's place: rows 8 tw + 4 rh .. + 3 of channels 2 cp, 2 cp + 1; the 16-byte chunk j of row r
                // lies at j ^ (r & 7).  Decays in powers of two, of the lower rows negated: E runs outward from
                // between rows 31 and 32
                float *ge = reinterpret_cast<float *>(stage + ST_G + tw * 1024 + rh * 512 + 8 * (cp & 1));
                auto at = [&](int i) { return reinterpret_cast<float2 *>(ge + 32 * i + 4 * ((cp >> 1) ^ (4 * rh) ^ i)); };
                float2 gv[4], sum = make_float2(0.f, 0.f);
                if (p.gate == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) gv[i] = *at(i);
                } else {                                   // one decay to a row, from global memory
                    const float *gp = p.g + (int64_t(meta->y) + row_e) * p.H + meta->z;
#pragma unroll
                    for (int i = 0; i < 4; ++i) gv[i].x = gv[i].y = row_e + i < n ? gp[i * p.H] : 0.f;
                }
                if (n < row_e + 4) {                     // rows past the end hold the next request's
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (row_e + i >= n) gv[i] = make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    gv[i] = __fmul2_rn(gv[i], make_float2(dir, dir));
                    sum = __fadd2_rn(sum, gv[i]);
                }
                const float2 next = make_float2(__shfl_xor_sync(0xffffffffu, sum.x, 16),
                                                __shfl_xor_sync(0xffffffffu, sum.y, 16));
                const float2 eight = __fadd2_rn(sum, next);
                float2 *tb = reinterpret_cast<float2 *>(tot);      // free since the second synchronisation of the last slice
                if (rh == 0) tb[tw * 16 + cp] = eight;
                group_sync();
                float2 off = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < 3; ++w)
                    if (w < (low ? 3 - tw : tw - 4)) off = __fadd2_rn(off, tb[(low ? 3 - w : 4 + w) * 16 + cp]);
                if (tw == 0 || tw == 7) {                  // the half's decay: steep channels
                    const float2 t = __fadd2_rn(off, eight);
                    const float lim = PREP_SAFE * L2E;
                    const uint32_t ex = __ballot_sync(0xffffffffu, !(low ? t.x <= lim : t.x >= -lim)) & 0xffffu,
                                   ey = __ballot_sync(0xffffffffu, !(low ? t.y <= lim : t.y >= -lim)) & 0xffffu;
                    if (lane == 0) {                       // (true for NaN too)
                        uint32_t mask = 0u;
                        if ((ex | ey) != 0u)
                            for (int i = 0; i < 16; ++i) mask |= (((ex >> i) & 1u) | ((ey >> i) & 1u) << 1) << (2 * i);
                        half_steep[low ? 0 : 1] = mask;
                    }
                }
                if (low != (rh == 1)) off = __fadd2_rn(off, next);
                if (low) {
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        *at(i) = off;
                        off = __fadd2_rn(off, gv[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        off = __fadd2_rn(off, gv[i]);
                        *at(i) = off;
                    }
                }
                group_sync();
                const uint32_t steep = half_steep[0] | half_steep[1];
                if (tw == 0 && lane == 0) steep_m[(c & 7) * 4 + s] = steep;
                const bool rare = n < 64 || steep != 0u;
                // ---- operands: this thread's row
                prep_wait(ok, &bars[PB_OPS_EMPTY + ob], (turn & 1) ^ 1, p.err);
                tc::fence_after_sync();
                const unsigned char *er = stage + ST_G + row * 128, *xr = stage + (isQ ? ST_Q : 0);
                unsigned char *br = sm + PREP_OFF_OPS + ob * PREP_OPS_BYTES + row * 128;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {              // eight channels, chunks 4 half + 2 b and the next
                    float x[8], E[8];
                    load_row<T>(xr, row, 16 * half + 8 * b, x);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 t = *reinterpret_cast<const float4 *>(er + 16 * ((4 * half + 2 * b + j) ^ (row & 7)));
                        E[4 * j] = t.x; E[4 * j + 1] = t.y; E[4 * j + 2] = t.z; E[4 * j + 3] = t.w;
                    }
                    if (rare) {                            // rows past the end; a steep channel enters the product as zeros
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] = row < n ? x[i] : 0.f;
                            big = max3(big, x[i], x[i]);
                            if ((steep >> (16 * half + 8 * b + i)) & 1u) x[i] = E[i] = 0.f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; i += 2) big = max3(big, x[i], x[i + 1]);
                    uint32_t h[8], l[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        prep_split<prep_fine<T>()>(__fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(ex2(E[i]), ex2(E[i + 1]))), h[i],
                                        h[i + 1], l[i], l[i + 1]);
                    tc::st8(ta + ob * 64 + 8 * b, h);
                    tc::st8(ta + ob * 64 + 32 + 8 * b, l);
                    if (!isQ) {
#pragma unroll
                        for (int i = 0; i < 8; i += 2)
                            prep_split<prep_fine<T>()>(__fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(ex2(-E[i]), ex2(-E[i + 1]))),
                                            h[i], h[i + 1], l[i], l[i + 1]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            unsigned char *at = br + 16 * ((4 * half + 2 * b + j) ^ (row & 7));
                            *reinterpret_cast<uint4 *>(at) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
                            *reinterpret_cast<uint4 *>(at + 8192) = make_uint4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
                        }
                    }
                }
                if (s + 2 >= nsl) {
                    big = warp_max(big);
                    if (lane == 0) kq_m[(c & 7) * 16 + 8 * tg + tw] = big;
                }
                tc::wait_st();
                tc::fence_before_sync();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[PB_OPS_FULL + ob]);
                    mbar_arrive(&bars[PB_ST_EMPTY + st]);
                }
            }
        }
    } else if (warp < 8) {
        tc::more_registers<104>();
        // --------------------------------------------------------------- epilogue
        const bool isP = warp >= 6;
        const int i = 32 * (warp & 1) + lane;              // chunk row
        float2 *sc = reinterpret_cast<float2 *>(sm + PREP_OFF_SC) + (isP ? 64 : 0);
        TaskWalk walk(ps, blockIdx.x, G);
        int32_t qi;
        Meta m = walk.next(ps, &qi);
        for (uint32_t c = 0; m.valid; ++c, m = walk.next(ps, &qi)) {
            const int db = c & 1;
            float *Ab = reinterpret_cast<float *>(sm + prep_off_at<T>()) + db * 2560;
            float f = p.scale;
            if (!isP)
                f = i < m.n ? widen1(static_cast<const T *>(p.beta)[(int64_t(m.row0) + i) * p.H + m.h]) : 0.f;
            if (!isP) prep_wait(ok, &bars[PB_AT_EMPTY + db], ((c >> 1) & 1) ^ 1, p.err);
            prep_wait(ok, &bars[PB_D_FULL + db], (c >> 1) & 1, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const uint32_t td = tmem + PREP_TM_D + db * 64 + (uint32_t(32 * (warp - 4)) << 16);
            const int last = isP ? i : i - 1;              // largest column of this row
            const int nb = 2 * (warp & 1) + 2;             // blocks of 16 columns with any of this warp's rows
            const uint32_t sb = (c & 7) * 4;
            uint32_t any = 0u;
            for (int s = 0; s < nsl; ++s) any |= steep_m[sb + s];
            if (any != 0u) {
                // steep channels: k_j q_i (or k_i) prod_{j < t <= i} e^{g_t}, from the diagonal left, added to
                // the accumulator
                const int64_t row = int64_t(m.row0) + i;
                const int64_t kb = (row * p.Hk + m.h / group) * p.K;
                const bool live = i < m.n;
                auto sync = [&] {
                    if (isP) named_sync<2, 64>();
                    else named_sync<3, 64>();
                };
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    float x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0.f;
#pragma unroll 1
                    for (int s = 0; s < nsl; ++s) {
                        uint32_t mask = steep_m[sb + s];
                        while (mask != 0u) {
                            const int d = 32 * s + __ffs(mask) - 1;
                            mask &= mask - 1u;
                            sync();                        // the previous channel is consumed
                            const float kd = live ? widen1(static_cast<const T *>(p.k)[kb + d]) : 0.f;
                            const float own = isP ? (live ? widen1(static_cast<const T *>(p.q)[kb + d]) : 0.f) : kd;
                            const float gd = live ? p.g[p.gate == 0 ? (row * p.H + m.h) * p.K + d : row * p.H + m.h] : 0.f;
                            sc[i] = make_float2(expf(gd), kd);
                            sync();
                            float run = own;
                            if (!isP) run *= sc[i].x;      // A starts one token before the row's own
                            for (int j = last; j >= 16 * b + 16; --j) run *= sc[j].x;
#pragma unroll
                            for (int e = 15; e >= 0; --e) {
                                const float2 t = sc[16 * b + e];
                                if (16 * b + e <= last) {
                                    x[e] = fmaf(run, t.y, x[e]);
                                    run *= t.x;
                                }
                            }
                        }
                    }
                    if (b < nb) {
                        float v[16];
                        uint32_t w[2][8];
                        tc::ld16(td + 16 * b, v);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e >> 3][e & 7] = __float_as_uint(v[e] + x[e]);
                        tc::st8(td + 16 * b, w[0]);
                        tc::st8(td + 16 * b + 8, w[1]);
                        tc::wait_st();
                    }
                }
            }
            // columns 8 b .. of this row, masked by selects: what they drop may hold anything
            auto columns = [&](int b, float (&x)[8]) {
                tc::ld8(td + 8 * b, x);
                if (prep_fine<T>()) {
                    float y[8];
                    tc::ld8(td + PREP_TM_FINE + 8 * b, y);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] += y[e];
                } else {
                    tc::wait_ld();
                }
                const int end = i < m.n ? last - 8 * b : -1;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = e <= end ? x[e] * f : 0.f;
            };
            auto done = [&] {                              // the accumulator is read
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[PB_D_EMPTY + db]);
            };
            if (!isP) {
#pragma unroll 1
                for (int b = 0; b < 2 * nb; ++b) {
                    float x[8];
                    columns(b, x);
                    if (16 * (b >> 1) <= i) {
                        float4 *to = reinterpret_cast<float4 *>(at_elem(Ab, i, 8 * b));
                        to[0] = make_float4(x[0], x[1], x[2], x[3]);
                        to[1] = make_float4(x[4], x[5], x[6], x[7]);
                    }
                }
                done();
                if (lane == 0) mbar_arrive(&bars[PB_AT_FULL + db]);
            } else {
                float mx = 0.f, inv;
#pragma unroll 1
                for (int b = 0; b < 2 * nb; ++b) {
                    float x[8];
                    columns(b, x);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) mx = max3(mx, x[e], x[e + 1]);
                }
                const float s = pow2_scale(warp_max(mx), KQ_LO, KQ_HI, inv);
                unsigned char *img = p.ws + int64_t(qi) * IMG_BYTES, *pi = sm + prep_off_p<T>();
                if (warp == 6 && lane == 0) tc::bulk_wait_read();      // the previous image has left
                named_sync<2, 64>();
#pragma unroll 1
                for (int b = 0; b < 8; ++b) {
                    float x[8];
                    if (b < 2 * nb) {
                        columns(b, x);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = 0.f;
                    }
                    image_put(pi, pi + 8192, i, b, x, s);
                }
                done();
                fence_proxy_async();
                named_sync<2, 64>();
                float *hdr = reinterpret_cast<float *>(img + IMG_HDR);
                if (lane == 0) hdr[HDR_PINV + (warp & 1)] = inv;
                if (warp == 6) {
                    if (lane == 0) {
                        tc::bulk_store(img + IMG_PHI, smem_u32(pi), 16384);
                        tc::bulk_commit();
                    }
                    // warps 0, 1, 4, 5 of a group of eight saw k, the others q; the second group is idle at K = 32
                    const float t = lane < 8 * (nsl > 1 ? 2 : 1) ? kq_m[(c & 7) * 16 + lane] : 0.f;
                    const float km = warp_max((lane & 3) < 2 ? t : 0.f), qm = warp_max((lane & 3) < 2 ? 0.f : t);
                    if (lane == 0) {
                        hdr[HDR_KMAX] = km;
                        hdr[HDR_QMAX] = qm;
                    }
                }
            }
        }
        if (warp == 6 && lane == 0) tc::bulk_wait();
    } else {
        tc::more_registers<112>();
        // ------------------------------------------------------------ solve pairs
        const int pr = (warp - 24) >> 1, pt = tid - 24 * 32 - 64 * pr, bar = 4 + pr;
        float *Ab = reinterpret_cast<float *>(sm + prep_off_at<T>()) + pr * 2560;
        float *X = reinterpret_cast<float *>(sm + prep_off_x<T>()) + pr * PREP_X_FLOATS;
        float *xs = reinterpret_cast<float *>(sm + prep_off_xs<T>()) + pr * 64 * PREP_XP;
        float *sbeta = reinterpret_cast<float *>(sm + PREP_OFF_BETA) + pr * 64;
        unsigned char *mi = sm + prep_off_m<T>() + pr * 16384;
        // what the solve leaves out
#pragma unroll 1
        for (int j = 0; j < 64; ++j) xs[pt * PREP_XP + j] = 0.f;
        TaskWalk walk(ps, int32_t(blockIdx.x) + pr * G, 2 * G);
        int32_t qi;
        Meta m = walk.next(ps, &qi);
        for (uint32_t c = 0; m.valid; ++c, m = walk.next(ps, &qi)) {
            const float b = pt < m.n ? widen1(static_cast<const T *>(p.beta)[(int64_t(m.row0) + pt) * p.H + m.h]) : 0.f;
            prep_wait(ok, &bars[PB_AT_FULL + pr], c & 1, p.err);
            if (pt == 0) tc::bulk_wait_read();             // the previous image has left
            bar64(bar);                                    // and the betas are consumed
            sbeta[pt] = b;
            prep_solve(Ab, X, xs, b, sbeta, pt, bar);
            if ((pt & 31) == 0) mbar_arrive(&bars[PB_AT_EMPTY + pr]);
            if (pt >= m.n) {                               // rows past the end: zeros whatever is in the others
#pragma unroll 1
                for (int j = 0; j < 64; ++j) xs[pt * PREP_XP + j] = 0.f;
            }
            auto columns = [&](int j, float (&x)[8]) {     // columns 8 j .. of row pt of M
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(xs + pt * PREP_XP + 8 * j + e);
                    x[e] = t.x; x[e + 1] = t.y; x[e + 2] = t.z; x[e + 3] = t.w;
                }
            };
            const int nj = 4 * (pt >> 5) + 4;              // blocks of 8 columns with any of this warp's rows
            float mx = 0.f, sum = 0.f, inv;
#pragma unroll 1
            for (int j = 0; j < nj; ++j) {
                float x[8];
                columns(j, x);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mx = max3(mx, x[e], x[e + 1]);
                    sum += fabsf(x[e]) + fabsf(x[e + 1]);
                }
            }
            const float s = pow2_scale(warp_max(mx), KQ_LO, KQ_HI, inv);
            sum = warp_max(sum);
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
                float x[8];
                if (j < nj) {
                    columns(j, x);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = 0.f;
                }
                image_put(mi, mi + 8192, pt, j, x, s);
            }
            fence_proxy_async();
            bar64(bar);
            unsigned char *img = p.ws + int64_t(qi) * IMG_BYTES;
            if ((pt & 31) == 0) {
                float *hdr = reinterpret_cast<float *>(img + IMG_HDR);
                hdr[HDR_MINV + (pt >> 5)] = inv;
                hdr[HDR_MSUM + (pt >> 5)] = sum;
            }
            if (pt == 0) {
                tc::bulk_store(img + IMG_MHI, smem_u32(mi), 16384);
                tc::bulk_commit();
            }
        }
        if (pt == 0) tc::bulk_wait();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 4) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

}  // namespace kda
