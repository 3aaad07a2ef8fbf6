// kda_delta_scan.cuh -- the chunked gated delta rule's walk over the chunks of one
// sequence-head, on tcgen05 with the state's operands in tensor memory.
//
// With the chunk's M and P (kda_delta_prep.cuh), G the cumulative log decay inside the
// chunk and S0 the state before it,
//
//   R  = V - (K e^G) S0,      U = M R,
//   O  = (scale Q e^G) S0 + P U,
//   S1 = diag(e^{G_C}) S0 + (K e^{G_C - G})^T U.
//
// Everything is computed transposed, one value column to a TMEM lane: the moving operands
// S^T, R^T and U^T [128 lanes x channels or tokens] are the A side in tensor memory,
// written there by the threads that made them; the chunk's own K e^G, scale Q e^G,
// K e^{G_C - G}, M and P are the B side in shared memory.  So no operand of the chain
// from state to state passes through shared memory, all 128 lanes work in every
// step, and lanes (value columns) never mix: a lane has scales of its own.
//
// FP32 accuracy from FP16: every operand is hi + lo (22 bits) and a product hi hi + hi lo +
// lo hi; what only reaches a bf16 output (Q, P) takes hi hi alone, 2^-11 against
// the output's 2^-9.  FP16 has range for that only under scales.  They are powers of two from
// rigorous bounds: the images carry the largest |k|, |q| and M's row sums; a lane
// measures |S| after each chunk and knows |v|; then |R| <= |v| + K |k| |S|,
// |U| <= |M|_1 |R|, |S1| <= |S| + 64 |k| |U|.  The bounds overshoot by up to 2^13
// and leave 2^-25 2^-15 2^13 of the largest value as the error of a product.  That is
// relative to the state and values that go in; where a chunk's decay clears the state and its
// values are next to nothing beside it, what comes out can be smaller than that:
// the four lane quarters each look out for such a chunk and take it token by token in
// FP32 (scan_tokens).
//
// One CTA of five warpgroups per sequence-head (registers moved to the chain):
//   * warps 0-7 (chain): two warps to each lane quarter, half the columns each; S in
//     registers;
//   * warps 8-15 (operands): K e^G, scale Q e^G, K e^{G_C-G} of the next chunk, from global memory
//     prefetched into registers; a thread has two channels of 16 rows;
//   * warp 16, one lane: MMA issue.  M and P arrive by bulk copy, double-buffered.
#pragma once

#include "kda_delta_prep.cuh"

namespace kda {

constexpr int SCAN_THREADS = 20 * 32;
constexpr int SB_S = 0, SB_KQ_FULL = 1, SB_KQ_EMPTY = 2, SB_D1 = 3, SB_O_EMPTY = 4, SB_IMG_FULL = 5, SB_IMG_EMPTY = 7,
              SB_R = 9, SB_D2 = 10, SB_KH_FULL = 11, SB_KH_EMPTY = 12, SB_U = 13, SB_D3 = 14, SB_O_FULL = 15,
              SCAN_NBARS = 16;
constexpr int SCAN_OFF_TMEM = SCAN_NBARS * 8;
constexpr int SCAN_OFF_RED = 192;                  // a word to a warp: chunks before the sequence
constexpr int SCAN_OFF_GAM = 512;                  // [2][128] e^{G_C}
constexpr int SCAN_OFF_MAX = SCAN_OFF_GAM + 2 * 128 * 4;       // [2 halves][128 lanes] largest |S|
constexpr int SCAN_OFF_VMAX = SCAN_OFF_MAX + 2 * 128 * 4;      // [2 halves][128 lanes] largest |v|
constexpr int SCAN_OFF_TOT = SCAN_OFF_VMAX + 2 * 128 * 4;      // [2][4 row groups][128] sums of g
constexpr int SCAN_OFF_SUM = 7680;                 // [2 halves][3][128], sums of a chunk taken token by token
constexpr int SCAN_OFF_KQ = 11 * 1024;             // K hi, K lo, Q hi, Q lo: [2 channel halves][64 rows][128 B] each
constexpr int SCAN_OFF_KH = SCAN_OFF_KQ + 4 * 16384;           // K e^{G_C-G} transposed, hi and lo: [128 channels][128 B]
constexpr int SCAN_OFF_IMG = SCAN_OFF_KH + 2 * 16384;
template <bool PLO>
constexpr int scan_img_pitch() { return (img_bytes<PLO>() + 1023) / 1024 * 1024; }
template <bool PLO>
constexpr int scan_bytes() { return SCAN_OFF_IMG + 2 * scan_img_pitch<PLO>() + 1024; }
static_assert(SCAN_OFF_TOT + 2 * 4 * 128 * 4 <= SCAN_OFF_SUM && SCAN_OFF_SUM + 2 * 3 * 128 * 4 <= SCAN_OFF_KQ,
              "small buffers fit");
// A chunk is taken token by token where its values are below 2^-16 of what the state can add to R
// and no channel keeps more than 2^-12 of the state: what comes out is then
// possibly below 2^-20 of what goes in.
constexpr float SCAN_WEAK_V = 65536.f, SCAN_WEAK_G = 1.f / 4096.f;
static_assert(scan_bytes<true>() <= 227 * 1024, "fits the shared memory of one CTA");

// TMEM columns.  U's accumulator takes the place of (K e^G) S's, which R has consumed.
constexpr uint32_t TM_SHI = 0, TM_SLO = 64, TM_RHI = 128, TM_RLO = 160, TM_D1 = 192, TM_O1 = 256, TM_O2 = 320,
                   TM_D3 = 384;
constexpr uint32_t SCAN_ID64 = tc::idesc_f16<128, 64>(), SCAN_ID128 = tc::idesc_f16<128, 128>();

// 16 values, scaled, to the hi and lo operand columns at ch, cl (8 columns each).
__device__ __forceinline__ void put_operand(uint32_t ch, uint32_t cl, const float (&x)[16], float s) {
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split_f16(x[2 * i] * s, x[2 * i + 1] * s, h[i], l[i]);
    tc::st8(ch, h);
    tc::st8(cl, l);
}

// D (+)= A B over KS steps of 16: A at TMEM columns ah, al; B at shared addresses bh, bl
// (128-byte rows of 64 values; the second 64 values of a row at + bstep).  HI: hi hi only.
template <int KS, bool HI>
__device__ __forceinline__ void mma_split(uint32_t d, uint32_t ah, uint32_t al, uint32_t bh, uint32_t bl,
                                          uint32_t bstep, uint32_t idesc) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const uint32_t b = (ks >> 2) * bstep + (ks & 3) * 32;
        tc::mma_f16_ts(d, ah + 8 * ks, tc::sw128_desc(bh + b), idesc, ks > 0);
        if (!HI) {
            tc::mma_f16_ts(d, ah + 8 * ks, tc::sw128_desc(bl + b), idesc, true);
            tc::mma_f16_ts(d, al + 8 * ks, tc::sw128_desc(bh + b), idesc, true);
        }
    }
}

// Two consecutive channels of q or k as they lie in memory, and widened.
template <typename T> struct Two;
template <> struct Two<float> { using raw = float2; static __device__ float2 wide(raw r) { return r; } };
template <> struct Two<__nv_bfloat16> {
    using raw = uint32_t;
    static __device__ float2 wide(raw r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
};
template <> struct Two<__half> {
    using raw = uint32_t;
    static __device__ float2 wide(raw r) { return __half22float2(*reinterpret_cast<const __half2 *>(&r)); }
};

// A chunk token by token, for the two warps of one lane quarter: thread (half, v) has
// S[64 half + i][v].  `row` is the chunk's first row, `n` its tokens; `sum` [2][3][128]
// of shared memory takes the halves' partial sums.
template <typename T>
__device__ __forceinline__ void scan_tokens(const DeltaParams &p, float (&S)[64], int64_t row, int n, int h, int half,
                                            int v, int quarter, float *sum) {
    const int hk = h / (p.H / p.Hk);
    for (int t = 0; t < n; ++t) {
        const int64_t r = row + t;
        const T *kp = static_cast<const T *>(p.k) + (r * p.Hk + hk) * p.K + 64 * half;
        const T *qp = static_cast<const T *>(p.q) + (r * p.Hk + hk) * p.K + 64 * half;
        const float *gp = p.g + (p.gate == 0 ? (r * p.H + h) * p.K + 64 * half : r * p.H + h);
        float a = 0.f, b = 0.f, qk = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (64 * half + i < p.K) {
                const float kd = widen1(kp[i]), qd = widen1(qp[i]);
                S[i] *= expf(gp[p.gate == 0 ? i : 0]);
                a = fmaf(kd, S[i], a);
                b = fmaf(qd, S[i], b);
                qk = fmaf(qd, kd, qk);
            }
        float *mine = sum + half * 384 + v;
        mine[0] = a;
        mine[128] = b;
        mine[256] = qk;
        asm volatile("bar.sync %0, 64;" ::"r"(8 + quarter) : "memory");
        a = sum[v] + sum[384 + v];
        b = sum[128 + v] + sum[512 + v];
        qk = sum[256 + v] + sum[640 + v];
        const bool in = v < p.V;
        const int64_t at = (r * p.H + h) * p.V + v;
        const float val = in ? widen1(static_cast<const T *>(p.v)[at]) : 0.f;
        const float u = widen1(static_cast<const T *>(p.beta)[r * p.H + h]) * (val - a);
        if (in && half == 0) put1(static_cast<T *>(p.o) + at, p.scale * fmaf(qk, u, b));
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (64 * half + i < p.K) S[i] = fmaf(widen1(kp[i]), u, S[i]);
        asm volatile("bar.sync %0, 64;" ::"r"(8 + quarter) : "memory");
    }
}

template <typename T, bool PLO>
__global__ void __launch_bounds__(SCAN_THREADS, 1) kda_delta_scan_kernel(const DeltaParams p) {
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + SCAN_OFF_TMEM);
    int32_t *red = reinterpret_cast<int32_t *>(sm + SCAN_OFF_RED);
    float *gam = reinterpret_cast<float *>(sm + SCAN_OFF_GAM);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = int(blockIdx.x) / p.H, h = int(blockIdx.x) - n * p.H;
    pdl_launch_dependents();

    if (tid == 0) {
        const int count[SCAN_NBARS] = {8, 8, 1, 1, 8, 1, 1, 1, 1, 8, 1, 8, 1, 8, 1, 1};
#pragma unroll
        for (int b = 0; b < SCAN_NBARS; ++b) mbar_init(&bars[b], count[b]);
        fence_mbar_init();
    }
    pdl_wait();
    if (warp == 0) {
        tc::tmem_alloc(smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    // the sequence's rows, and the number of chunks before its first
    int64_t ra, rb;
    sequence_rows(p, n, ra, rb);
    int32_t before = 0;
    if (p.cu != nullptr) {
        for (int i = tid; i < n; i += SCAN_THREADS) before += nchunks<BT>(__ldg(p.cu + i), __ldg(p.cu + i + 1));
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) red[warp] = before;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (p.cu != nullptr) {
        before = 0;
        for (int i = 0; i < SCAN_THREADS / 32; ++i) before += red[i];
    } else {
        before = n * p.cpr;
    }
    const int rows = int(rb - ra);
    int nc = (rows + BT - 1) / BT;
    // malformed cu_seqlens must not lead past the workspace
    if (before < 0 || (int64_t(before) + nc) * p.H > p.n_tasks) nc = 0;
    const unsigned char *img0 = p.ws + (int64_t(before) * p.H + h) * img_bytes<PLO>();
    const int64_t img_step = int64_t(p.H) * img_bytes<PLO>();
    bool ok = true;

    // registers: 640 threads of 96 at launch; 2 * 128 + 2 * 96 + 24 <= 5 * 96
    if (warp < 8) {
        tc::more_registers<128>();
        // ------------------------------------------------------------------ chain
        const int quarter = warp & 3, half = warp >> 2, v = 32 * quarter + lane;
        const uint32_t tq = tmem + (uint32_t(32 * quarter) << 16);
        float *smax = reinterpret_cast<float *>(sm + SCAN_OFF_MAX), *svmax = reinterpret_cast<float *>(sm + SCAN_OFF_VMAX);
        const int32_t e = state_entry(p, n);
        const bool mine = v < p.V;
        float S[64];                                       // S[64 half + i][v]
        {
            const float *sp = p.state_in + ((int64_t(e < 0 ? 0 : e) * p.H + h) * p.K + 64 * half) * p.V + v;
#pragma unroll
            for (int i = 0; i < 64; ++i)
                S[i] = p.state_in != nullptr && e >= 0 && mine && 64 * half + i < p.K ? sp[int64_t(i) * p.V] : 0.f;
        }
        const int vs = p.H * p.V;
        const T *vp = static_cast<const T *>(p.v) + (ra * p.H + h) * p.V + v;
        T *op = static_cast<T *>(p.o) + (ra * p.H + h) * p.V + v;
        float bS = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) bS = fmaxf(bS, fabsf(S[i]));
        float invS;
        if (nc > 0) {
            smax[half * 128 + v] = bS;
            asm volatile("bar.sync %0, 64;" ::"r"(8 + quarter) : "memory");
            bS = fmaxf(smax[v], smax[128 + v]);
            const float s = pow2_scale(bS, VS_LO, VS_HI, invS);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = S[16 * b + i];
                put_operand(tq + TM_SHI + 32 * half + 8 * b, tq + TM_SLO + 32 * half + 8 * b, x, s);
            }
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_S]);
        }
        for (int c = 0; c < nc; ++c) {
            const uint32_t ph = c & 1;
            const int left = rows - 64 * c, t0 = 32 * half;        // this thread's tokens t0 .. t0 + 31
            const int64_t at = int64_t(64 * c + t0) * vs;
            T vr[32];
            float bv = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) vr[i] = mine && t0 + i < left ? vp[at + i * vs] : T(0.f);
#pragma unroll
            for (int i = 0; i < 32; ++i) bv = fmaxf(bv, fabsf(widen1(vr[i])));
            svmax[half * 128 + v] = bv;
            prep_wait(ok, &bars[SB_IMG_FULL + ph], (c >> 1) & 1, p.err);
            const float *hdr = reinterpret_cast<const float *>(sm + SCAN_OFF_IMG + ph * scan_img_pitch<PLO>() + img_hdr<PLO>());
            const float minv = hdr[HDR_MINV + half], msum = fmaxf(hdr[HDR_MSUM], hdr[HDR_MSUM + 1]);
            const float pinv = hdr[HDR_PINV + half], kmax = hdr[HDR_KMAX], qmax = hdr[HDR_QMAX];
            asm volatile("bar.sync %0, 64;" ::"r"(8 + quarter) : "memory");
            bv = fmaxf(svmax[v], svmax[128 + v]);
            float invk, invq, invR, invU, invS1;
            pow2_scale(kmax, KQ_LO, KQ_HI, invk);
            pow2_scale(qmax * fabsf(p.scale), KQ_LO, KQ_HI, invq);
            const float bR = bv + float(p.K) * kmax * bS;
            const float sR = pow2_scale(bR, VS_LO, VS_HI, invR);
            const float bU = msum * bR;
            const float sU = pow2_scale(bU, VS_LO, VS_HI, invU);
            float sS = pow2_scale(bS + 64.f * kmax * bU, VS_LO, VS_HI, invS1);
            bool weak = __any_sync(0xffffffffu, bR > SCAN_WEAK_V * bv);
            if (weak) {                                            // the same in both warps of the quarter
                prep_wait(ok, &bars[SB_KH_FULL], ph, p.err);
                float gmax = 0.f;
                for (int i = 0; i < p.K; ++i) gmax = fmaxf(gmax, gam[ph * 128 + i]);
                weak = __all_sync(0xffffffffu, gmax < SCAN_WEAK_G);
                if (weak) {
                    scan_tokens<T>(p, S, ra + 64 * c, left < 64 ? left : 64, h, half, v, quarter,
                                   reinterpret_cast<float *>(sm + SCAN_OFF_SUM));
                    float mx = 0.f;                                // the new state's own bound
#pragma unroll
                    for (int i = 0; i < 64; ++i) mx = fmaxf(mx, fabsf(S[i]));
                    smax[half * 128 + v] = mx;
                    asm volatile("bar.sync %0, 64;" ::"r"(8 + quarter) : "memory");
                    sS = pow2_scale(fmaxf(smax[v], smax[128 + v]), VS_LO, VS_HI, invS1);
                }
            }
            // R = V - (K e^G) S
            prep_wait(ok, &bars[SB_D1], ph, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const float f1 = invS * invk;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[16];
                tc::ld16(tq + TM_D1 + t0 + 16 * b, x);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = fmaf(-f1, x[i], widen1(vr[16 * b + i]));
                put_operand(tq + TM_RHI + 16 * half + 8 * b, tq + TM_RLO + 16 * half + 8 * b, x, sR);
            }
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_R]);
            // U = M R
            prep_wait(ok, &bars[SB_D2], ph, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const float f2 = invR * minv * sU;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[16];
                tc::ld16(tq + TM_D1 + t0 + 16 * b, x);
                tc::wait_ld();
                put_operand(tq + TM_RHI + 16 * half + 8 * b, tq + TM_RLO + 16 * half + 8 * b, x, f2);
            }
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_U]);
            // S1 = diag(e^{G_C}) S + (K e^{G_C-G})^T U
            prep_wait(ok, &bars[SB_KH_FULL], ph, p.err);
            prep_wait(ok, &bars[SB_D3], ph, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const float f3 = invU * invk;
            float mx = 0.f;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float x[16];
                tc::ld16(tq + TM_D3 + 64 * half + 16 * b, x);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 gm = *reinterpret_cast<const float4 *>(gam + ph * 128 + 64 * half + 16 * b + i);
                    x[i] = fmaf(gm.x, S[16 * b + i], f3 * x[i]);
                    x[i + 1] = fmaf(gm.y, S[16 * b + i + 1], f3 * x[i + 1]);
                    x[i + 2] = fmaf(gm.z, S[16 * b + i + 2], f3 * x[i + 2]);
                    x[i + 3] = fmaf(gm.w, S[16 * b + i + 3], f3 * x[i + 3]);
                }
                if (weak) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = S[16 * b + i];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    S[16 * b + i] = x[i];
                    mx = fmaxf(mx, fabsf(x[i]));
                }
                put_operand(tq + TM_SHI + 32 * half + 8 * b, tq + TM_SLO + 32 * half + 8 * b, x, sS);
            }
            smax[half * 128 + v] = mx;
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_S]);
            // O = (scale Q e^G) S0 + P U
            prep_wait(ok, &bars[SB_O_FULL], ph, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const float f4 = invS * invq, f5 = invU * pinv;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[16], y[16];
                tc::ld16(tq + TM_O1 + t0 + 16 * b, x);
                tc::ld16(tq + TM_O2 + t0 + 16 * b, y);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (mine && !weak && t0 + 16 * b + i < left) put1(op + at + (16 * b + i) * vs, fmaf(f4, x[i], f5 * y[i]));
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_O_EMPTY]);
            asm volatile("bar.sync %0, 64;" ::"r"(8 + quarter) : "memory");
            bS = fmaxf(smax[v], smax[128 + v]);
            invS = invS1;
        }
        if (p.state_out != nullptr && e >= 0 && mine) {
            float *sp = p.state_out + ((int64_t(e) * p.H + h) * p.K + 64 * half) * p.V + v;
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (64 * half + i < p.K) sp[int64_t(i) * p.V] = S[i];
        }
    } else if (warp < 16) {
        tc::fewer_registers<96>();
        // --------------------------------------------------------------- operands
        constexpr float L2E = 1.4426950408889634f;
        using W2 = Two<T>;
        const int pw = warp - 8, ch = pw & 1, rg = pw >> 1;         // channel half, row group of 16
        const int d = 64 * ch + 2 * lane;                           // channels d, d + 1
        const bool chan = d < p.K;
        const int hk = h / (p.H / p.Hk);
        const int ks = p.Hk * p.K, gs = p.gate == 0 ? p.H * p.K : p.H;
        const T *qp = static_cast<const T *>(p.q) + ((ra + 16 * rg) * p.Hk + hk) * p.K + d;
        const T *kp = static_cast<const T *>(p.k) + ((ra + 16 * rg) * p.Hk + hk) * p.K + d;
        const float *gp = p.gate == 0 ? p.g + ((ra + 16 * rg) * p.H + h) * p.K + d : p.g + (ra + 16 * rg) * p.H + h;
        float *tot = reinterpret_cast<float *>(sm + SCAN_OFF_TOT);
        typename W2::raw rk[16], rq[16];
        float2 rgd[16];
        float2 kqmax = make_float2(0.f, 0.f);
        auto fetch = [&](int c) {
            const int left = rows - 64 * c - 16 * rg;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool in = chan && i < left;
                const int64_t r = int64_t(64) * c + i;
                rgd[i] = make_float2(0.f, 0.f);
                if (in) {
                    if (p.gate == 0) rgd[i] = *reinterpret_cast<const float2 *>(gp + r * gs);
                    else rgd[i].x = rgd[i].y = gp[r * gs];
                }
                rk[i] = in ? *reinterpret_cast<const typename W2::raw *>(kp + r * ks) : typename W2::raw{};
                rq[i] = in ? *reinterpret_cast<const typename W2::raw *>(qp + r * ks) : typename W2::raw{};
            }
            kqmax = *reinterpret_cast<const float2 *>(img0 + c * img_step + img_hdr<PLO>() + 4 * HDR_KMAX);
        };
        if (nc > 0) fetch(0);
        for (int c = 0; c < nc; ++c) {
            const uint32_t ph = c & 1;
            if (pw == 0 && lane == 0) {                             // M and P of this chunk
                prep_wait(ok, &bars[SB_IMG_EMPTY + ph], ((c >> 1) & 1) ^ 1, p.err);
                mbar_arrive_expect_tx(&bars[SB_IMG_FULL + ph], img_bytes<PLO>());
                bulk_load(sm + SCAN_OFF_IMG + ph * scan_img_pitch<PLO>(), img0 + c * img_step, img_bytes<PLO>(),
                          &bars[SB_IMG_FULL + ph]);
            }
            __syncwarp();
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sum.x += rgd[i].x;
                sum.y += rgd[i].y;
            }
            float *tb = tot + ph * 512;
            *reinterpret_cast<float2 *>(tb + rg * 128 + d) = sum;
            named_sync<1, 256>();
            float2 pre = make_float2(0.f, 0.f), post = pre, all = pre;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float2 t = *reinterpret_cast<const float2 *>(tb + w * 128 + d);
                if (w < rg) { pre.x += t.x; pre.y += t.y; }
                if (w > rg) { post.x += t.x; post.y += t.y; }
                all.x += t.x;
                all.y += t.y;
            }
            float unused;
            const float sk = pow2_scale(kqmax.x, KQ_LO, KQ_HI, unused);
            const float sq = p.scale * pow2_scale(kqmax.y * fabsf(p.scale), KQ_LO, KQ_HI, unused);
            // K e^G and scale Q e^G: row r of a tile is 128 bytes, its 16-byte chunk lane / 4 at (lane / 4) ^ (r & 7)
            prep_wait(ok, &bars[SB_KQ_EMPTY], ph ^ 1, p.err);
            unsigned char *kq = sm + SCAN_OFF_KQ + ch * 8192 + rg * 2048 + 4 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                pre.x += rgd[i].x;
                pre.y += rgd[i].y;
                const float2 kv = W2::wide(rk[i]), qv = W2::wide(rq[i]);
                const float e0 = ex2(pre.x * L2E), e1 = ex2(pre.y * L2E);
                uint32_t kh, kl, qh, ql;
                split_f16(kv.x * e0 * sk, kv.y * e1 * sk, kh, kl);
                split_f16(qv.x * e0 * sq, qv.y * e1 * sq, qh, ql);
                unsigned char *at = kq + i * 128 + 16 * ((lane >> 2) ^ (i & 7));
                *reinterpret_cast<uint32_t *>(at) = kh;
                *reinterpret_cast<uint32_t *>(at + 16384) = kl;
                *reinterpret_cast<uint32_t *>(at + 32768) = qh;
                if (PLO) *reinterpret_cast<uint32_t *>(at + 49152) = ql;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_KQ_FULL]);
            // K e^{G_C-G} transposed: channel d's row holds the 64 tokens, eight to a 16-byte chunk
            prep_wait(ok, &bars[SB_KH_EMPTY], ph ^ 1, p.err);
            if (rg == 0) *reinterpret_cast<float2 *>(gam + ph * 128 + d) = make_float2(ex2(all.x * L2E), ex2(all.y * L2E));
#pragma unroll
            for (int o = 1; o >= 0; --o) {                          // tokens 8 o .. 8 o + 7 of the group, from the end
                float x[8], y[8];
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    const float2 kv = W2::wide(rk[8 * o + i]);
                    x[i] = kv.x * ex2(post.x * L2E) * sk;
                    y[i] = kv.y * ex2(post.y * L2E) * sk;
                    post.x += rgd[8 * o + i].x;
                    post.y += rgd[8 * o + i].y;
                }
                uint4 xh, xl, yh, yl;
                split_f16(x[0], x[1], xh.x, xl.x); split_f16(x[2], x[3], xh.y, xl.y);
                split_f16(x[4], x[5], xh.z, xl.z); split_f16(x[6], x[7], xh.w, xl.w);
                split_f16(y[0], y[1], yh.x, yl.x); split_f16(y[2], y[3], yh.y, yl.y);
                split_f16(y[4], y[5], yh.z, yl.z); split_f16(y[6], y[7], yh.w, yl.w);
                const int cc = 2 * rg + o;                          // chunk of the row
                unsigned char *a0 = sm + SCAN_OFF_KH + d * 128 + 16 * (cc ^ (d & 7));
                unsigned char *a1 = sm + SCAN_OFF_KH + (d + 1) * 128 + 16 * (cc ^ ((d + 1) & 7));
                *reinterpret_cast<uint4 *>(a0) = xh;
                *reinterpret_cast<uint4 *>(a0 + 16384) = xl;
                *reinterpret_cast<uint4 *>(a1) = yh;
                *reinterpret_cast<uint4 *>(a1 + 16384) = yl;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_KH_FULL]);
            if (c + 1 < nc) fetch(c + 1);
        }
        // no copy may be in flight when the CTA ends
        if (pw == 0 && lane == 0)
            for (int c = nc > 2 ? nc - 2 : 0; c < nc; ++c) prep_wait(ok, &bars[SB_IMG_FULL + (c & 1)], (c >> 1) & 1, p.err);
    } else {
        tc::fewer_registers<24>();
        // ------------------------------------------------------------- MMA issue
        if (warp == 16 && lane == 0) {
        const uint32_t kq = smem_u32(sm + SCAN_OFF_KQ), kh = smem_u32(sm + SCAN_OFF_KH);
        auto commit = [&](int b) { tc::commit(smem_u32(&bars[b])); };
        for (int c = 0; c < nc; ++c) {
            const uint32_t ph = c & 1;
            const uint32_t img = smem_u32(sm + SCAN_OFF_IMG + ph * scan_img_pitch<PLO>());
            prep_wait(ok, &bars[SB_KQ_FULL], ph, p.err);
            prep_wait(ok, &bars[SB_S], ph, p.err);
            tc::fence_after_sync();
            mma_split<8, false>(tmem + TM_D1, tmem + TM_SHI, tmem + TM_SLO, kq, kq + 16384, 8192, SCAN_ID64);
            commit(SB_D1);
            prep_wait(ok, &bars[SB_O_EMPTY], ph ^ 1, p.err);
            tc::fence_after_sync();
            mma_split<8, !PLO>(tmem + TM_O1, tmem + TM_SHI, tmem + TM_SLO, kq + 32768, kq + 49152, 8192, SCAN_ID64);
            commit(SB_KQ_EMPTY);
            prep_wait(ok, &bars[SB_IMG_FULL + ph], (c >> 1) & 1, p.err);
            prep_wait(ok, &bars[SB_R], ph, p.err);
            tc::fence_after_sync();
            mma_split<4, false>(tmem + TM_D1, tmem + TM_RHI, tmem + TM_RLO, img + IMG_MHI, img + IMG_MLO, 0, SCAN_ID64);
            commit(SB_D2);
            prep_wait(ok, &bars[SB_KH_FULL], ph, p.err);
            prep_wait(ok, &bars[SB_U], ph, p.err);
            tc::fence_after_sync();
            mma_split<4, false>(tmem + TM_D3, tmem + TM_RHI, tmem + TM_RLO, kh, kh + 16384, 0, SCAN_ID128);
            commit(SB_D3);
            commit(SB_KH_EMPTY);
            mma_split<4, !PLO>(tmem + TM_O2, tmem + TM_RHI, tmem + TM_RLO, img + IMG_PHI, img + IMG_PLO, 0, SCAN_ID64);
            commit(SB_O_FULL);
            commit(SB_IMG_EMPTY + ph);
        }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

}  // namespace kda
