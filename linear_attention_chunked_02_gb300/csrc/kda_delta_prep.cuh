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
// One persistent CTA of seven warpgroups per SM; every role walks the same chunk-heads:
//   * warp 0: MMA issue; warp 1: TMA loads of q, k and g in slices of 32 channels into a
//     ring (plain loads stall here: what the CTA leaves of the L1 holds too little in
//     flight);
//   * warps 8-15 and 16-23 (transform): every second slice each into TF32 operands; lane = channel, warp = eight rows, so that the sums along the rows run in registers and
//     one exchange of eight totals to a channel;
//   * warps 4, 5 (A) and 6, 7 (P): the accumulator's rows out of tensor memory; A
//     with beta and the mask into the solve's tile, P straight into its image;
//   * warps 24-27: two pairs, each the 64-token solve of every second chunk-head,
//     and M's image.
// The warpgroups' registers are moved to where the row of 64 values needs them.
#pragma once

#include "kda_delta_rec.cuh"
#include "kda_kgb.cuh"

namespace kda {

// Image of one chunk-head in the workspace.  M and P are FP16 pairs hi + lo (22
// bits) scaled by a power of two for each half of 32 rows, 64 rows of 128
// bytes with the 128-byte swizzle: the B operands of the scan's products.
constexpr int IMG_MHI = 0, IMG_MLO = 8192, IMG_PHI = 16384, IMG_PLO = 24576;
template <bool PLO>
constexpr int img_hdr() { return PLO ? 32768 : 24576; }   // 16-bit outputs in bf16 need no low part of P
constexpr int IMG_HDR_BYTES = 128;
template <bool PLO>
constexpr int img_bytes() { return img_hdr<PLO>() + IMG_HDR_BYTES; }
// header (floats): 1 / scale of M rows 0-31, 32-63; largest row sum of |M| in the halves;
// 1 / scale of P in the halves; largest |k|, |q|
constexpr int HDR_MINV = 0, HDR_MSUM = 2, HDR_PINV = 4, HDR_KMAX = 6, HDR_QMAX = 7;

constexpr int PREP_THREADS = 28 * 32;
constexpr int PREP_TW = 8;                         // transform warps of a group
constexpr float PREP_SAFE = 48.0f;
constexpr int PREP_NOPS = 2;
constexpr int PREP_OPS_BYTES = 48 * 1024;          // A hi, A lo (128 rows), B hi, B lo (64 rows), 128-byte rows
// staging ring: a slice of 64 rows x 32 channels of k, q (at most 8 KiB each) and g
template <typename T>
constexpr int prep_stage_bytes() { return 2 * 64 * 32 * int(sizeof(T)) + 8192; }
template <typename T>
constexpr int prep_stages() { return sizeof(T) == 2 ? 3 : 2; }
constexpr int PB_OPS_FULL = 0, PB_OPS_EMPTY = PREP_NOPS, PB_D_FULL = 2 * PREP_NOPS, PB_D_EMPTY = PB_D_FULL + 2,
              PB_AT_FULL = PB_D_EMPTY + 2, PB_AT_EMPTY = PB_AT_FULL + 2, PB_ST_FULL = PB_AT_EMPTY + 2,
              PB_ST_EMPTY = PB_ST_FULL + 3, PREP_NBARS = PB_ST_EMPTY + 3;
constexpr int PREP_OFF_TMEM = PREP_NBARS * 8;
constexpr int PREP_OFF_STEEP = 256;                // [8 chunk-heads][4 slices]
constexpr int PREP_OFF_KQ = PREP_OFF_STEEP + 8 * 4 * 4;        // [8 chunk-heads][16 warps] largest |k|, |q|
constexpr int PREP_OFF_TOT = 1536;                 // [2 groups][2][8 warps][32 channels] sums of g
constexpr int PREP_OFF_SC = PREP_OFF_TOT + 4 * 8 * 32 * 4;     // slow path: e^g, k of a channel, for A and for P
constexpr int PREP_OFF_BETA = PREP_OFF_SC + 2 * 64 * 8;        // [pairs][64]
constexpr int PREP_OFF_CU = PREP_OFF_BETA + 2 * 64 * 4;
constexpr int PREP_OFF_OPS = 8 * 1024;
constexpr int PREP_OFF_AT = PREP_OFF_OPS + PREP_NOPS * PREP_OPS_BYTES;
constexpr int PREP_OFF_X = PREP_OFF_AT + 2 * 10 * 256 * 4;
constexpr int PREP_XP = 68;                        // pitch of the solved tile (floats)
constexpr int PREP_OFF_XS = PREP_OFF_X + 2 * KGB_X_FLOATS * 4;
constexpr int PREP_OFF_ST = PREP_OFF_XS + 2 * 64 * PREP_XP * 4;
template <typename T>
constexpr int prep_bytes() { return PREP_OFF_ST + prep_stages<T>() * prep_stage_bytes<T>() + 1024; }
static_assert(PREP_OFF_TMEM + 4 <= PREP_OFF_STEEP && PREP_OFF_KQ + 8 * 16 * 8 <= PREP_OFF_TOT, "header fits");
static_assert(PREP_OFF_CU + CU_CAP * 4 <= PREP_OFF_OPS, "cu_seqlens fits");
static_assert(PREP_OFF_ST % 128 == 0 && prep_bytes<float>() <= 227 * 1024 && prep_bytes<__half>() <= 227 * 1024,
              "fits the shared memory of one CTA");

// Tensor maps of q, k [rows, Hk, K] and g [rows, H, K] as {channels, heads, rows}: boxes of 32
// channels x 64 rows here, of all channels (and of v's values) in the scan.
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

// The hi part alone.
__device__ __forceinline__ uint32_t round_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Largest of m and |a|, |b|.
__device__ __forceinline__ float max3(float m, float a, float b) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_max(float v) {   // v >= 0
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// Row i of an image tile from 64 floats (already scaled): hi and, if `lo` is not null, lo.
__device__ __forceinline__ void image_row(unsigned char *hi, unsigned char *lo, int i, const float (&x)[64], float s) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint4 h, l;
        split_f16(x[8 * c] * s, x[8 * c + 1] * s, h.x, l.x);
        split_f16(x[8 * c + 2] * s, x[8 * c + 3] * s, h.y, l.y);
        split_f16(x[8 * c + 4] * s, x[8 * c + 5] * s, h.z, l.z);
        split_f16(x[8 * c + 6] * s, x[8 * c + 7] * s, h.w, l.w);
        const int at = i * 128 + 16 * (c ^ (i & 7));
        *reinterpret_cast<uint4 *>(hi + at) = h;
        if (lo != nullptr) *reinterpret_cast<uint4 *>(lo + at) = l;
    }
}

// A wait that gives up once, after WAIT_LIMIT_NS: the thread then records it and waits no
// more, but keeps arriving, so that no other thread is stranded.  The tries suspend
// the warp (polling takes issue slots from those at work), and the timer is read only
// every 64 of them: reading it takes longer than most of these waits.
__device__ __forceinline__ void prep_wait(bool &ok, uint64_t *bar, uint32_t parity, unsigned *err) {
    if (!ok || mbar_try_wait(bar, parity)) return;
    unsigned long long t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_suspend(bar, parity, 100000u)) return;
        if ((it & 63u) == 0u) {
            const unsigned long long t = globaltimer();
            if (t0 == 0) t0 = t;
            if (t - t0 > WAIT_LIMIT_NS) break;
        }
    }
    ok = false;
    atomicOr(err, ERR_WAIT_TIMEOUT);
}

template <typename T, bool PLO>
__global__ void __launch_bounds__(PREP_THREADS, 1) kda_delta_prep_kernel(const __grid_constant__ DeltaMaps maps, const DeltaParams p) {
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + PREP_OFF_TMEM);
    uint32_t *steep_m = reinterpret_cast<uint32_t *>(sm + PREP_OFF_STEEP);
    float2 *kq_m = reinterpret_cast<float2 *>(sm + PREP_OFF_KQ);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int NST = prep_stages<T>(), STB = prep_stage_bytes<T>(), ST_Q = 64 * 32 * int(sizeof(T)), ST_G = 2 * ST_Q;
    const int nsl = p.K / 32;
    const int32_t G = gridDim.x;
    const int group = p.H / p.Hk;
    pdl_launch_dependents();

    if (tid == 0) {
        for (int b = 0; b < NST; ++b) {
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
        tc::tmem_alloc(smem_u32(tmem_slot), 128);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    // registers: 896 threads of 72 at launch; 24 + 112 + 4 * 64 + 112 <= 7 * 72
    if (warp < 4) {
        tc::fewer_registers<24>();
        if (warp == 0) {
            // ------------------------------------------------------------- MMA issue
            TaskWalk w(ps, blockIdx.x, G);
            uint32_t u = 0;
            for (uint32_t c = 0; w.next(ps).valid; ++c) {
                const int db = c & 1;
                prep_wait(ok, &bars[PB_D_EMPTY + db], ((c >> 1) & 1) ^ 1, p.err);
                for (int s = 0; s < nsl; ++s, ++u) {
                    const int ob = u % PREP_NOPS;
                    prep_wait(ok, &bars[PB_OPS_FULL + ob], (u / PREP_NOPS) & 1, p.err);
                    __syncwarp();
                    tc::fence_after_sync();
                    const uint32_t ah = smem_u32(sm + PREP_OFF_OPS + ob * PREP_OPS_BYTES);
                    const uint32_t d = tmem + db * 64;
                    if (tc::elect_one()) {
                        // K = 8 channels: 32 bytes along the rows
                        uint64_t dah = tc::sw128_desc(ah), dal = tc::sw128_desc(ah + 16384),
                                 dbh = tc::sw128_desc(ah + 32768), dbl = tc::sw128_desc(ah + 40960);
#pragma unroll 1
                        for (int kk = 0; kk < 4; ++kk) {
                            tc::mma_tf32(d, dah, dbh, KGB_IDESC, s > 0 || kk > 0);
                            tc::mma_tf32(d, dah, dbl, KGB_IDESC, true);
                            tc::mma_tf32(d, dal, dbh, KGB_IDESC, true);
                            dah += 2;
                            dal += 2;
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
            uint32_t u = 0;
            for (Meta m = w.next(ps); m.valid; m = w.next(ps))
                for (int s = 0; s < nsl; ++s, ++u) {
                    const int st = u % NST;
                    prep_wait(ok, &bars[PB_ST_EMPTY + st], ((u / NST) & 1) ^ 1, p.err);
                    __syncwarp();
                    if (tc::elect_one()) {
                        unsigned char *to = sm + PREP_OFF_ST + st * STB;
                        uint64_t *full = &bars[PB_ST_FULL + st];
                        mbar_arrive_expect_tx(full, 2 * ST_Q + (p.gate == 0 ? 8192 : 0));
                        tma_load_3d(to, &maps.k, 32 * s, m.h / group, m.row0, full);
                        tma_load_3d(to + ST_Q, &maps.q, 32 * s, m.h / group, m.row0, full);
                        if (p.gate == 0) tma_load_3d(to + ST_G, &maps.g, 32 * s, m.h, m.row0, full);
                    }
                    __syncwarp();
                }
            // no copy may be in flight when the CTA ends
            for (uint32_t i = u > NST ? u - NST : 0; i < u; ++i)
                prep_wait(ok, &bars[PB_ST_FULL + i % NST], (i / NST) & 1, p.err);
        }
    } else if (warp >= 8 && warp < 24) {
        tc::fewer_registers<64>();
        // -------------------------------------------------------------- transform
        constexpr float L2E = 1.4426950408889634f;
        const int tw = warp & 7, tg = (warp >> 3) - 1;     // rows 8 tw .. + 7 of slices tg, tg + 2
        float *tot = reinterpret_cast<float *>(sm + PREP_OFF_TOT) + tg * 512;
        TaskWalk walk(ps, blockIdx.x, G);
        Meta m = walk.next(ps);
        uint32_t turn = 0;
        for (uint32_t c = 0; m.valid; ++c, m = walk.next(ps)) {
            float kmax = 0.f, qmax = 0.f;
            for (int s = tg; s < nsl; s += 2, ++turn) {
                const uint32_t u = c * nsl + s;
                const int ob = u % PREP_NOPS, st = u % NST;
                unsigned char *stage = sm + PREP_OFF_ST + st * STB;
                T *kt = reinterpret_cast<T *>(stage) + tw * 256 + lane;
                T *qt = reinterpret_cast<T *>(stage + ST_Q) + tw * 256 + lane;
                float *gt = reinterpret_cast<float *>(stage + ST_G) + tw * 256 + lane;
                prep_wait(ok, &bars[PB_ST_FULL + st], (u / NST) & 1, p.err);
                if (p.gate != 0) {                         // one decay to a row, from global memory
                    const float *gp = p.g + (int64_t(m.row0) + 8 * tw) * p.H + m.h;
#pragma unroll
                    for (int i = 0; i < 8; ++i) gt[32 * i] = 8 * tw + i < m.n ? gp[i * p.H] : 0.f;
                }
                for (int i = m.n > 8 * tw ? m.n - 8 * tw : 0; i < 8; ++i) {    // rows past the end hold the next request's
                    kt[32 * i] = T(0.f);
                    qt[32 * i] = T(0.f);
                    gt[32 * i] = 0.f;
                }
                float kv[8], qv[8], gv[8], sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    kv[i] = widen1(kt[32 * i]);
                    qv[i] = widen1(qt[32 * i]);
                    gv[i] = gt[32 * i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    gv[i] *= L2E;
                    sum += gv[i];
                    if (i & 1) {
                        kmax = max3(kmax, kv[i - 1], kv[i]);
                        qmax = max3(qmax, qv[i - 1], qv[i]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[PB_ST_EMPTY + st]);
                float *tb = tot + (turn & 1) * 256;
                tb[tw * 32 + lane] = sum;
                if (tg == 0) named_sync<1, 256>();
                else named_sync<6, 256>();
                // decay from the middle of the chunk (between rows 31 and 32) outward
                float lo = 0.f, hi = 0.f, off = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float t = tb[w * 32 + lane];
                    if (w < 4) lo += t;
                    else hi += t;
                    if (tw < 4 ? (w > tw && w < 4) : (w >= 4 && w < tw)) off += t;
                }
                const bool keep = lo >= -PREP_SAFE * L2E && hi >= -PREP_SAFE * L2E;     // false for NaN too
                float E[8];
                if (tw < 4) {
#pragma unroll
                    for (int i = 7; i >= 0; --i) {
                        E[i] = -off;
                        off += gv[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        off += gv[i];
                        E[i] = off;
                    }
                }
                const uint32_t steep = __ballot_sync(0xffffffffu, !keep);
                if (steep != 0u && !keep) {                // a steep channel enters the product as zeros
#pragma unroll
                    for (int i = 0; i < 8; ++i) kv[i] = qv[i] = E[i] = 0.f;
                }
                prep_wait(ok, &bars[PB_OPS_EMPTY + ob], ((u / PREP_NOPS) & 1) ^ 1, p.err);
                unsigned char *ops = sm + PREP_OFF_OPS + ob * PREP_OPS_BYTES + tw * 1024 + 4 * (lane & 3);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {           // two rows at a time, in paired instructions
                    const float2 k2 = make_float2(kv[i], kv[i + 1]);
                    const float2 up = make_float2(ex2(E[i]), ex2(E[i + 1])), dn = make_float2(ex2(-E[i]), ex2(-E[i + 1]));
                    uint32_t h[3][2], l[3][2];
                    split2(__fmul2_rn(k2, up), h[0][0], h[0][1], l[0][0], l[0][1]);
                    split2(__fmul2_rn(make_float2(qv[i], qv[i + 1]), up), h[1][0], h[1][1], l[1][0], l[1][1]);
                    split2(__fmul2_rn(k2, dn), h[2][0], h[2][1], l[2][0], l[2][1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // row 8 tw + i + e of the tile, its 16-byte chunk lane / 4 at position (lane / 4) ^ (i + e)
                        unsigned char *at = ops + (i + e) * 128 + 16 * ((lane >> 2) ^ (i + e));
                        *reinterpret_cast<uint32_t *>(at) = h[0][e];
                        *reinterpret_cast<uint32_t *>(at + 8192) = h[1][e];
                        *reinterpret_cast<uint32_t *>(at + 16384) = l[0][e];
                        *reinterpret_cast<uint32_t *>(at + 24576) = l[1][e];
                        *reinterpret_cast<uint32_t *>(at + 32768) = h[2][e];
                        *reinterpret_cast<uint32_t *>(at + 40960) = l[2][e];
                    }
                }
                if (tw == 0 && lane == 0) steep_m[(c & 7) * 4 + s] = steep;
                if (s + 2 >= nsl) {
                    kmax = warp_max(kmax);
                    qmax = warp_max(qmax);
                    if (lane == 0) kq_m[(c & 7) * 16 + 8 * tg + tw] = make_float2(kmax, qmax);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[PB_OPS_FULL + ob]);
            }
        }
    } else if (warp < 8) {
        tc::more_registers<112>();
        // --------------------------------------------------------------- epilogue
        const bool isP = warp >= 6;
        const int i = 32 * (warp & 1) + lane;              // chunk row
        float2 *sc = reinterpret_cast<float2 *>(sm + PREP_OFF_SC) + (isP ? 64 : 0);
        TaskWalk walk(ps, blockIdx.x, G);
        int32_t qi;
        Meta m = walk.next(ps, &qi);
        for (uint32_t c = 0; m.valid; ++c, m = walk.next(ps, &qi)) {
            const int db = c & 1;
            float *Ab = reinterpret_cast<float *>(sm + PREP_OFF_AT) + db * 2560;
            float f = p.scale;
            if (!isP)
                f = i < m.n ? widen1(static_cast<const T *>(p.beta)[(int64_t(m.row0) + i) * p.H + m.h]) : 0.f;
            if (!isP) prep_wait(ok, &bars[PB_AT_EMPTY + db], ((c >> 1) & 1) ^ 1, p.err);
            prep_wait(ok, &bars[PB_D_FULL + db], (c >> 1) & 1, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const uint32_t td = tmem + db * 64 + (uint32_t(32 * (warp - 4)) << 16);
            float x[64];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float v[16];
                tc::ld16(td + 16 * b, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[16 * b + e] = v[e];
            }
            tc::wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[PB_D_EMPTY + db]);
            const int last = isP ? i : i - 1;              // largest column of this row
            // select: rows past the end and masked columns may hold anything
#pragma unroll
            for (int j = 0; j < 64; ++j) x[j] = j <= last && i < m.n ? x[j] : 0.f;
            const uint32_t sb = (c & 7) * 4;
            uint32_t any = 0u;
            for (int s = 0; s < nsl; ++s) any |= steep_m[sb + s];
            if (any != 0u) {
                // steep channels: k_j q_i (or k_i) prod_{j < t <= i} e^{g_t}, from the diagonal left
                const int64_t row = int64_t(m.row0) + i;
                const int64_t kb = (row * p.Hk + m.h / group) * p.K;
                for (int s = 0; s < nsl; ++s) {
                    uint32_t mask = steep_m[sb + s];
                    while (mask != 0u) {
                        const int d = 32 * s + __ffs(mask) - 1;
                        mask &= mask - 1u;
                        if (isP) named_sync<2, 64>();
                        else named_sync<3, 64>();
                        const bool live = i < m.n;
                        const float kd = live ? widen1(static_cast<const T *>(p.k)[kb + d]) : 0.f;
                        const float own = isP ? (live ? widen1(static_cast<const T *>(p.q)[kb + d]) : 0.f) : kd;
                        const float gd = live ? p.g[p.gate == 0 ? (row * p.H + m.h) * p.K + d : row * p.H + m.h] : 0.f;
                        sc[i] = make_float2(expf(gd), kd);
                        if (isP) named_sync<2, 64>();
                        else named_sync<3, 64>();
                        if (live) {
                            float run = own;
                            if (!isP) run *= sc[i].x;      // A starts one token before the row's own
#pragma unroll
                            for (int j = 63; j >= 0; --j) {
                                const float2 t = sc[j];
                                if (j <= last) {
                                    x[j] = fmaf(run, t.y, x[j]);
                                    run *= t.x;
                                }
                            }
                        }
                    }
                }
                if (isP) named_sync<2, 64>();
                else named_sync<3, 64>();
            }
#pragma unroll
            for (int j = 0; j < 64; ++j) x[j] *= f;
            if (!isP) {
#pragma unroll
                for (int j0 = 0; j0 < 4; ++j0)
                    if (16 * j0 <= i) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(at_elem(Ab, i, 16 * j0 + e)) =
                                make_float4(x[16 * j0 + e], x[16 * j0 + e + 1], x[16 * j0 + e + 2], x[16 * j0 + e + 3]);
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[PB_AT_FULL + db]);
            } else {
                float mx = 0.f;
#pragma unroll
                for (int j = 0; j < 64; ++j) mx = fmaxf(mx, fabsf(x[j]));
                float inv;
                const float s = pow2_scale(warp_max(mx), KQ_LO, KQ_HI, inv);
                unsigned char *img = p.ws + int64_t(qi) * img_bytes<PLO>();
                image_row(img + IMG_PHI, PLO ? img + IMG_PLO : nullptr, i, x, s);
                float *hdr = reinterpret_cast<float *>(img + img_hdr<PLO>());
                if (lane == 0) hdr[HDR_PINV + (warp & 1)] = inv;
                if (warp == 6) {                           // 8 transform warps to a group, the second idle at K = 32
                    const float2 t = lane < 8 * (nsl > 1 ? 2 : 1) ? kq_m[(c & 7) * 16 + lane] : make_float2(0.f, 0.f);
                    const float km = warp_max(t.x), qm = warp_max(t.y);
                    if (lane == 0) {
                        hdr[HDR_KMAX] = km;
                        hdr[HDR_QMAX] = qm;
                    }
                }
            }
        }
    } else {
        tc::more_registers<112>();
        // ------------------------------------------------------------ solve pairs
        const int pr = (warp - 24) >> 1, pt = tid - 24 * 32 - 64 * pr, bar = 4 + pr;
        float *Ab = reinterpret_cast<float *>(sm + PREP_OFF_AT) + pr * 2560;
        float *X = reinterpret_cast<float *>(sm + PREP_OFF_X) + pr * KGB_X_FLOATS;
        float *xs = reinterpret_cast<float *>(sm + PREP_OFF_XS) + pr * 64 * PREP_XP;
        float *sbeta = reinterpret_cast<float *>(sm + PREP_OFF_BETA) + pr * 64;
        TaskWalk walk(ps, int32_t(blockIdx.x) + pr * G, 2 * G);
        int32_t qi;
        Meta m = walk.next(ps, &qi);
        for (uint32_t c = 0; m.valid; ++c, m = walk.next(ps, &qi)) {
            const float b = pt < m.n ? widen1(static_cast<const T *>(p.beta)[(int64_t(m.row0) + pt) * p.H + m.h]) : 0.f;
            prep_wait(ok, &bars[PB_AT_FULL + pr], c & 1, p.err);
            bar64(bar);                                    // the previous tile and betas are consumed
            sbeta[pt] = b;
            kgb_solve<float>(Ab, X, X + 4 * XTS, xs, PREP_XP, m.n, pt, bar);
            bar64(bar);
            if ((pt & 31) == 0) mbar_arrive(&bars[PB_AT_EMPTY + pr]);
            float x[64], mx = 0.f, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 64; j += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(xs + pt * PREP_XP + j);
                const float4 bt = *reinterpret_cast<const float4 *>(sbeta + j);
                const bool live = pt < m.n;
                x[j] = live ? t.x * bt.x : 0.f;
                x[j + 1] = live ? t.y * bt.y : 0.f;
                x[j + 2] = live ? t.z * bt.z : 0.f;
                x[j + 3] = live ? t.w * bt.w : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mx = fmaxf(mx, fabsf(x[j + e]));
                    sum += fabsf(x[j + e]);
                }
            }
            float inv;
            const float s = pow2_scale(warp_max(mx), KQ_LO, KQ_HI, inv);
            sum = warp_max(sum);
            unsigned char *img = p.ws + int64_t(qi) * img_bytes<PLO>();
            image_row(img + IMG_MHI, img + IMG_MLO, pt, x, s);
            if ((pt & 31) == 0) {
                float *hdr = reinterpret_cast<float *>(img + img_hdr<PLO>());
                hdr[HDR_MINV + (pt >> 5)] = inv;
                hdr[HDR_MSUM + (pt >> 5)] = sum;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 4) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 128);
    }
}

}  // namespace kda
