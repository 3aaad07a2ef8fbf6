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
// lo hi, for all types: Q and P of BF16 calls with their high parts alone saved 2 to 4 %
// (16 x 512 x 64 heads: 462 us, 476 with both) and took their outputs 1.1e-3 of the norm away from
// the rounded 64-bit result, which they now meet to 1e-4.  FP16 has range for that only under scales.  They are powers of
// two from rigorous bounds: the images carry the largest |k|, |q| and M's row sums; a lane
// measures |S| after each chunk and knows |v|; then |R| <= |v| + K |k| |S|,
// |U| <= |M|_1 |R|, |S1| <= |S| + 64 |k| |U|.  The bounds overshoot by up to 2^13
// and leave 2^-25 2^-15 2^13 of the largest value as the error of a product.  That is
// relative to the state and values that go in; where a chunk's decay clears the state and its
// values are next to nothing beside it, what comes out can be smaller than that:
// the four lane quarters each look out for such a chunk and take it token by token in
// FP32 (scan_tokens).  A segment's map has the same limit: kda_delta_join_kernel looks out for that.
//
// Few heads and long sequences leave most of the GPU idle in that walk, so sequences can be split
// into segments.  A segment maps the state by S -> M S + N, M [K, K], N [K, V]: a first run of
// this kernel (TRANS) takes N from the walk without outputs, from zero states (the sequence's
// own in its first segment), and M from the walk of the identity with v = 0;
// kda_delta_join_kernel chains them into every segment's initial state; then all
// segments are walked at once.  That last run reads no state that it may write: what the first segments
// start from was copied by the first run, since a state pool is usually updated in place.
//
// One persistent CTA of eight warpgroups per SM, whose roles go through its walks (sequence-heads, or
// their segments) as one stream of chunks: the loads and operands of the next walk
// are under way while the chain ends one.  Registers are moved to the chain.
//   * warps 0-15 (chain): four warps to each lane quarter, a quarter of the columns each; S in
//     registers.  What bounds the walk is their path from state to state, so all
//     else is on other warps;
//   * warps 16-23 (operands): K e^G, scale Q e^G, K e^{G_C-G} of the next chunk; a thread has two or
//     four channels of eight rows, so that sums along the rows run in registers and eight tokens
//     of a channel make one 16-byte store;
//   * warps 24-27 (output): O, a lane quarter each;
//   * warp 28: MMA issue; warps 29, 30 and 31: the loads (TMA) of q, k and g, of v, and of the
//     images.  Plain loads stall here (what the CTA leaves of the L1 holds too
//     little in flight), so g is staged in shared memory, and q and k where they find room: of 16
//     bits, or of 32 bits and up to 64 channels (2 x 1000 tokens, 16 heads, K = 64: 5 % less time).
//     32-bit ones of more channels are read directly (64 x 512 tokens, 32 heads of
//     K = V = 128, the whole operator: 1250 us, 1397 with g read directly too).
// 16 x 512 tokens x 64 heads of BF16, K = V = 128: 266 us and 1126 MB, 4.2 TB/s; 4.9 us a chunk and
// CTA.  185 million warp instructions take 62 % of the issue slots, and the chain and the operand
// warps each need about the whole of a chunk's 9500 cycles.  With segments (1 x 16384 x 32 heads):
// N and M 360 us (3.1 us a chunk), the join 49, the walk 289.
#pragma once

#include "kda_delta_prep.cuh"

namespace kda {

constexpr int SCAN_THREADS = 32 * 32, SCAN_REGISTERS = 64;     // per thread at launch
constexpr int SCAN_PARTS = 4;                      // chain threads to a lane
constexpr int SB_S = 0, SB_KQ_FULL = 1, SB_KQ_EMPTY = 2, SB_D1 = 3, SB_O_EMPTY = 4, SB_IMG_FULL = 5, SB_IMG_EMPTY = 6,
              SB_R = 7, SB_D2 = 8, SB_KH_FULL = 9, SB_KH_EMPTY = 10, SB_U = 11, SB_D3 = 12, SB_O_FULL = 13,
              SB_V_FULL = 14, SB_V_EMPTY = 15, SB_ST_FULL = 16, SB_ST_EMPTY = 17, SB_IMG_READ = 18,
              SB_GAM = 19, SCAN_NBARS = 21;
constexpr int SCAN_OFF_TMEM = SCAN_NBARS * 8;
constexpr int SCAN_OFF_GAM = 256;                  // [2][128] e^{G_C}
constexpr int SCAN_OFF_MAX = SCAN_OFF_GAM + 2 * 128 * 4;       // [4 parts][128 lanes] largest |S|
constexpr int SCAN_OFF_VMAX = SCAN_OFF_MAX + 4 * 128 * 4;      // [4 parts][128 lanes] largest |v|
constexpr int SCAN_OFF_OUT = SCAN_OFF_VMAX + 4 * 128 * 4;          // [2][128 lanes] inverse scales of S and U for O
constexpr int SCAN_OFF_TOT = SCAN_OFF_OUT + 2 * 128 * 8;       // [8 row groups][128] sums of g
constexpr int SCAN_OFF_SUM = SCAN_OFF_TOT + 8 * 128 * 4;       // [4 parts][128], sums of a chunk taken token by token
constexpr int SCAN_OFF_GH = SCAN_OFF_SUM + 4 * 128 * 4;     // [64] decays of the rows, where a head has one
constexpr int SCAN_OFF_KQ = 14 * 1024;             // K hi, K lo, Q hi, Q lo: [2 channel halves][64 rows][128 B] each
constexpr int SCAN_OFF_KH = SCAN_OFF_KQ + 4 * 16384;   // K e^{G_C-G} transposed, hi and lo: [128 channels][128 B]
constexpr int SCAN_OFF_IMG = SCAN_OFF_KH + 2 * 16384;  // the chunk's image (two find no room)
constexpr int SCAN_OFF_V = SCAN_OFF_IMG + (IMG_BYTES + 1023) / 1024 * 1024;    // [64 tokens][V]
template <typename T>
constexpr int scan_off_st() { return SCAN_OFF_V + 64 * 128 * int(sizeof(T)); }         // k, q, g: [64 rows][K] each
template <typename T>
constexpr bool scan_staged(int K) { return sizeof(T) == 2 || K <= 64; }    // q and k too, not g alone
template <typename T>
constexpr int scan_off_g(int K) { return !scan_staged<T>(K) ? 0 : 32768; } // g, in the staging buffer
template <typename T>
constexpr int scan_stage(int K) { return scan_off_g<T>(K) + 64 * (K <= 64 ? 64 : 128) * 4; }
template <typename T>
constexpr int scan_bytes(int K) { return scan_off_st<T>() + scan_stage<T>(K) + 1024; }
static_assert(SCAN_OFF_TMEM + 4 <= SCAN_OFF_GAM, "header fits");
static_assert(SCAN_OFF_GH + 64 * 4 <= SCAN_OFF_KQ, "small buffers fit");
static_assert(scan_bytes<float>(64) <= 227 * 1024 && scan_bytes<float>(128) <= 227 * 1024 &&
                  scan_bytes<__half>(128) <= 227 * 1024, "fits the shared memory of one CTA");
// A chunk is taken token by token where its values are below 2^-16 of what the state can add to R
// and no channel keeps more than 2^-12 of the state: what comes out is then
// possibly below 2^-20 of what goes in.
constexpr float SCAN_WEAK_V = 65536.f, SCAN_WEAK_G = 1.f / 4096.f;

// TMEM columns.  U's accumulator takes the place of (K e^G) S's, which R has consumed.
constexpr uint32_t TM_SHI = 0, TM_SLO = 64, TM_RHI = 128, TM_RLO = 160, TM_D1 = 192, TM_O1 = 256, TM_O2 = 320,
                   TM_D3 = 384;
constexpr uint32_t SCAN_ID64 = tc::idesc_f16<128, 64>(), SCAN_ID128 = tc::idesc_f16<128, 128>();

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// 16 values, scaled, to the hi and lo operand columns at ch, cl (8 columns each).
__device__ __forceinline__ void put_operand(uint32_t ch, uint32_t cl, const float (&x)[16], float s) {
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 y = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), both(s));
        split_f16(y.x, y.y, h[i], l[i]);
    }
    tc::st8(ch, h);
    tc::st8(cl, l);
}

// D (+)= A B over `steps` steps of 16: A at TMEM columns ah, al; B at shared addresses bh, bl
// (128-byte rows of 64 values; the second 64 values of a row at + bstep).
// Not unrolled: the issuing warp has few registers.
__device__ __forceinline__ void mma_split(int steps, uint32_t d, uint32_t ah, uint32_t al, uint32_t bh, uint32_t bl,
                                          uint32_t bstep, uint32_t idesc) {
    uint64_t dh = tc::sw128_desc(bh), dl = tc::sw128_desc(bl);
#pragma unroll 1
    for (int ks = 0; ks < steps; ++ks) {
        tc::mma_f16_ts(d, ah, dh, idesc, ks > 0);
        tc::mma_f16_ts(d, ah, dl, idesc, true);
        tc::mma_f16_ts(d, al, dh, idesc, true);
        ah += 8;
        al += 8;
        const uint32_t step = (ks == 3 ? bstep - 96 : 32) >> 4;    // the address field counts 16 bytes
        dh += step;
        dl += step;
    }
}

// Two 16-bit values in a register.
template <typename T> struct Pair {
    uint32_t r;
    __device__ Pair() : r(0u) {}
    __device__ Pair(T a, T b) : r(uint32_t(reinterpret_cast<const uint16_t &>(a)) | uint32_t(reinterpret_cast<const uint16_t &>(b)) << 16) {}
    __device__ Pair abs() const { Pair x; x.r = r & 0x7fff7fffu; return x; }
    __device__ Pair max(Pair o) const;                     // of values without NaN; a NaN counts as nothing
    __device__ float2 wide() const;
};
template <> __device__ __forceinline__ Pair<__nv_bfloat16> Pair<__nv_bfloat16>::max(Pair o) const {
    Pair x;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(x.r) : "r"(r), "r"(o.r));
    return x;
}
template <> __device__ __forceinline__ Pair<__half> Pair<__half>::max(Pair o) const {
    Pair x;
    asm("max.f16x2 %0, %1, %2;" : "=r"(x.r) : "r"(r), "r"(o.r));
    return x;
}
template <> __device__ __forceinline__ float2 Pair<__nv_bfloat16>::wide() const {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 Pair<__half>::wide() const {
    return __half22float2(reinterpret_cast<const __half2 &>(r));
}
template <> struct Pair<float> {};

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

// A chunk token by token, for the four warps of one lane quarter: thread (part, v) has
// S[32 part + i][v].  `row` is the chunk's first row, `n` its tokens; `sum` [4][128]
// of shared memory takes the parts' sums.  OUT: with the outputs.
template <typename T, bool OUT>
__device__ __forceinline__ void scan_tokens(const DeltaParams &p, float (&S)[32], int64_t row, int n, int h, int part,
                                            int v, int quarter, float *sum) {
    const int hk = h / (p.H / p.Hk), d0 = 32 * part;
    auto sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(8 + quarter) : "memory"); };
    auto total = [&](float x) {
        sum[part * 128 + v] = x;
        sync();
        x = (sum[v] + sum[128 + v]) + (sum[256 + v] + sum[384 + v]);
        sync();
        return x;
    };
    for (int t = 0; t < n; ++t) {
        const int64_t r = row + t;
        const T *kp = static_cast<const T *>(p.k) + (r * p.Hk + hk) * p.K + d0;
        const T *qp = static_cast<const T *>(p.q) + (r * p.Hk + hk) * p.K + d0;
        const float *gp = p.g + (p.gate == 0 ? (r * p.H + h) * p.K + d0 : r * p.H + h);
        float a = 0.f, b = 0.f, qk = 0.f;
        if (d0 < p.K) {                                    // K is a multiple of 32
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float kd = widen1(kp[i]);
                S[i] *= expf(gp[p.gate == 0 ? i : 0]);
                a = fmaf(kd, S[i], a);
                if (OUT) {
                    const float qd = widen1(qp[i]);
                    b = fmaf(qd, S[i], b);
                    qk = fmaf(qd, kd, qk);
                }
            }
        }
        a = total(a);
        if (OUT) {
            b = total(b);
            qk = total(qk);
        }
        const bool in = v < p.V;
        const int64_t at = (r * p.H + h) * p.V + v;
        const float val = in ? widen1(static_cast<const T *>(p.v)[at]) : 0.f;
        const float u = widen1(static_cast<const T *>(p.beta)[r * p.H + h]) * (val - a);
        if (OUT && in && part == 0) put1(static_cast<T *>(p.o) + at, p.scale * fmaf(qk, u, b));
        if (d0 < p.K) {
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = fmaf(widen1(kp[i]), u, S[i]);
        }
    }
}

// KW 128: K and V are 128, which makes every row pitch an immediate; 64: K is at most 64; 0: other
// widths.  Staged rows are KP channels and 128 values long for all, zeros past K and V from the copy.  (One kernel for the last two, which reads FP32 both staged and not, took 592 us for 64 x 512
// tokens, 32 heads of K = 64, V = 128; its own takes 434.)
template <typename T, int KW, bool TRANS>
__global__ void __launch_bounds__(SCAN_THREADS, 1) kda_delta_scan_kernel(const __grid_constant__ DeltaMaps maps, const DeltaParams p) {
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + SCAN_OFF_TMEM);
    float *gam = reinterpret_cast<float *>(sm + SCAN_OFF_GAM);
    constexpr bool W128 = KW == 128, STAGED = scan_staged<T>(KW == 64 ? 64 : 128);
    constexpr bool FOUR = W128 || (KW == 0 && STAGED);     // operands: four channels to a lane
    constexpr int KP = KW == 64 ? 64 : 128;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int K = W128 ? 128 : p.K, V = W128 ? 128 : p.V;
    pdl_launch_dependents();

    if (tid == 0) {
        const int count[SCAN_NBARS] = {16, 8, 1, 1, 4, 1, 1, 16, 1, 8, 1, 16, 1, 1, 1, 16, 1, 8, 4, 1, 1};
#pragma unroll
        for (int b = 0; b < SCAN_NBARS; ++b) mbar_init(&bars[b], count[b]);
        fence_mbar_init();
    }
    pdl_wait();
    if (warp == 0) {
        tc::tmem_alloc(smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // walk w: unit w / H.  TRANS: N, then M of every unit in turn; dense, only what the join needs: N of a
    // sequence's first segment, N and M of the others but the last (a CTA goes through walks gridDim.x
    // apart, and those with nothing to do would leave some CTAs twice the work of others)
    const int32_t parts = p.cu == nullptr && p.seg > 0 ? (p.cpr + p.seg - 1) / p.seg : 1;     // dense: segments
    const int32_t maps1 = max(1, 2 * parts - 3);           // dense, TRANS: walks to a sequence-head
    const int32_t walks = !TRANS ? p.n_units * p.H : p.cu != nullptr ? 2 * p.n_units * p.H
                                                                     : parts > 1 ? p.nseq * maps1 * p.H : 0;
    auto unit_at = [&](int32_t w, int &run) {              // run 1: M
        run = 0;
        if (!TRANS) return w / p.H;
        if (p.cu != nullptr) {
            run = w & 1;
            return (w >> 1) / p.H;
        }
        const int32_t g = w / p.H, n = g / maps1, r = g - n * maps1;
        if (r == 0) return n * parts;
        run = (r - 1) & 1;
        return n * parts + 1 + ((r - 1) >> 1);
    };
    auto entry = [&](int32_t w) {
        if (w >= walks) return make_int4(0, 0, 0, 0);
        int run;
        const int32_t u = unit_at(w, run);
        if (p.cu != nullptr) return p.units[u];            // a plain load: the call's first kernel wrote it
        const int32_t n = u / parts;
        return make_int4(n, u - n * parts, n * p.cpr, parts);
    };
    struct Walk1 {
        int32_t w, unit, h, run, rows, nc, row;    // run 1: M; first row
        int4 e;
        int32_t before;                    // chunks before the first
        bool idle, last;
    };
    auto walk_at = [&](int32_t w, const int4 &e) {
        Walk1 x;
        x.w = w;
        x.e = e;
        x.unit = unit_at(w, x.run);
        x.h = TRANS && p.cu != nullptr ? (w >> 1) - x.unit * p.H : w - w / p.H * p.H;
        int64_t a = 0, b = 0;
        if (e.w > 0) sequence_rows(p, e.x, a, b);
        x.last = e.y == e.w - 1;
        a += int64_t(64) * e.y * p.seg;
        if (p.seg > 0 && b - a > int64_t(64) * p.seg) b = a + int64_t(64) * p.seg;
        x.rows = b > a ? int(b - a) : 0;
        x.row = int(a);
        x.nc = (x.rows + BT - 1) / BT;
        x.before = e.z + e.y * p.seg;
        // malformed cu_seqlens must not lead past the workspace; the last segment's map is not
        // needed, nor what the first makes of another state than its own
        if (x.before < 0 || (int64_t(x.before) + x.nc) * p.H > p.n_tasks) x.nc = 0;
        // (nor past the maps: with them, all units of a sequence are listed)
        x.idle = w >= walks || e.w <= 0 || (p.seg > 0 && int64_t(x.unit) - e.y + e.w > p.n_units) ||
                 (TRANS && (x.last || (x.run == 1 && e.y == 0)));
        if (x.idle) x.nc = 0;
        return x;
    };
    auto image_at = [&](const Walk1 &x) { return p.ws + (int64_t(x.before) * p.H + x.h) * IMG_BYTES; };
    const int32_t w0 = blockIdx.x, wstep = gridDim.x;
    const int64_t img_step = int64_t(p.H) * IMG_BYTES;
    constexpr int nh = KW == 64 ? 1 : 2;                         // halves of 64 channels
    bool ok = true;

    static_assert(4 * 80 + 2 * 64 + 40 + 24 <= SCAN_THREADS / 128 * SCAN_REGISTERS, "the groups' shares");
    if (warp < 16) {
        tc::more_registers<80>();
        // ------------------------------------------------------------------ chain
        const int quarter = warp & 3, part = warp >> 2, v = 32 * quarter + lane;
        const uint32_t tq = tmem + (uint32_t(32 * quarter) << 16);
        float *smax = reinterpret_cast<float *>(sm + SCAN_OFF_MAX) + v, *svmax = reinterpret_cast<float *>(sm + SCAN_OFF_VMAX) + v;
        float2 *sout = reinterpret_cast<float2 *>(sm + SCAN_OFF_OUT);
        // the four threads of a lane
        auto lane_max = [&](float &x, float &y) {          // of the state and of the values
            smax[part * 128] = x;
            svmax[part * 128] = y;
            asm volatile("bar.sync %0, 128;" ::"r"(8 + quarter) : "memory");
            x = fmaxf(max3(smax[0], smax[128], smax[256]), smax[384]);
            y = fmaxf(max3(svmax[0], svmax[128], svmax[256]), svmax[384]);
        };
        auto release = [&](int b) {                        // operand columns written, accumulators read
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[b]);
        };
        auto accumulator = [&](int b, uint32_t ph) {
            prep_wait(ok, &bars[b], ph, p.err);
            __syncwarp();
            tc::fence_after_sync();
        };
        float S[32];                                       // S[32 part + i][v]
        const bool held = 32 * part < K;                   // K is a multiple of 32
        const int t0 = 16 * part;                          // this thread's tokens of a chunk: t0 .. t0 + 15
        T *sv = reinterpret_cast<T *>(sm + SCAN_OFF_V) + t0 * 128 + v;
        const uint32_t sop = tq + TM_SHI + 16 * part, rop = tq + TM_RHI + 8 * part;      // operand columns, hi parts
        auto put_state = [&](float s) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = S[16 * b + i];
                put_operand(sop + 8 * b, sop + TM_SLO - TM_SHI + 8 * b, x, s);
            }
        };
        auto state_max = [&] {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 32; i += 2) m = max3(m, S[i], S[i + 1]);
            return m;
        };
        const int64_t sz = int64_t(K) * V, tz = sz + int64_t(K) * K;
        uint32_t cc = 0, vc = 0;                           // chunks so far, and those with values
        int4 next = entry(w0);
        for (int32_t w = w0; w < walks; w += wstep) {
        const Walk1 x = walk_at(w, next);
        next = entry(w + wstep);
        const int run = x.run, W = run == 1 ? K : V;       // columns of the state that is walked
        const bool mine = v < W && held;
        // the state that it starts from, and where it ends
        float *to = nullptr, *keep = nullptr;
        {
            const float *from = nullptr;
            if (!x.idle) {
                const int32_t e = state_entry(p, x.e.x);
                float *map = p.trans + (int64_t(x.unit) * p.H + x.h) * tz;
                if (x.e.y > 0) {
                    if (!TRANS) from = map - int64_t(p.H) * tz;        // chained into the segment before
                } else if (p.state_in != nullptr && e >= 0) {
                    from = p.state_in + (int64_t(e) * p.H + x.h) * sz;
                    // The last segment's walk may store over that entry (state_out may be state_in) before the
                    // last run gets to this one: walks go to CTAs in turn, and nothing orders two of them.  So
                    // the first run copies the state to the last segment's place, whose own map nobody makes or
                    // reads, and the last run starts from the copy.
                    if (x.e.w > 1) {
                        float *copy = map + int64_t(x.e.w - 1) * p.H * tz;
                        if (TRANS) keep = copy;
                        else from = copy;
                    }
                }
                if (TRANS) to = map + (run == 1 ? sz : 0);
                else if (x.last && p.state_out != nullptr && e >= 0) to = p.state_out + (int64_t(e) * p.H + x.h) * sz;
            }
            const float *sp = from + int64_t(32 * part) * W + v;
            const bool read = from != nullptr && mine;
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = read ? sp[int64_t(i) * W] : 0.f;
            if (TRANS && keep != nullptr && mine) {
                float *kp = keep + int64_t(32 * part) * W + v;
#pragma unroll
                for (int i = 0; i < 32; ++i) kp[int64_t(i) * W] = S[i];
            }
            if (run == 1) {
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] = 32 * part + i == v && held ? 1.f : 0.f;
            }
        }
        // a chunk's values: this thread's part of the largest, and 16-bit ones themselves.  The next chunk's
        // come while the products of this one run
        Pair<T> vr[sizeof(T) == 2 ? 8 : 1];                // two tokens to a word
        auto values = [&](int left) {
            float bv = 0.f;
            if (run == 1) return bv;                       // values of zero
            prep_wait(ok, &bars[SB_V_FULL], vc++ & 1, p.err);
            // rows past the end hold the next request's; columns past V stay in their lanes
#pragma unroll 1
            for (int i = left > t0 ? left - t0 : 0; i < 16; ++i)
                sv[i * 128] = T(0.f);
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) vr[i] = Pair<T>(sv[2 * i * 128], sv[(2 * i + 1) * 128]);
                Pair<T> m = vr[0].abs();
#pragma unroll
                for (int i = 1; i < 8; ++i) m = m.max(vr[i].abs());
                const float2 f = m.wide();
                bv = fmaxf(f.x, f.y);
            } else {
#pragma unroll
                for (int i = 0; i < 16; i += 2) bv = max3(bv, widen1(sv[i * 128]), widen1(sv[(i + 1) * 128]));
            }
            return bv;
        };
        float bS = 0.f, bv = 0.f, invS = 1.f;
        if (x.nc > 0) {
            bS = state_max();
            bv = values(x.rows);
            lane_max(bS, bv);
            put_state(pow2_scale(bS, VS_LO, VS_HI, invS));
            release(SB_S);
        }
        for (int c = 0; c < x.nc; ++c, ++cc) {
            const uint32_t ph = cc & 1;
            const int left = x.rows - 64 * c;
            prep_wait(ok, &bars[SB_IMG_FULL], ph, p.err);
            const float *hdr = reinterpret_cast<const float *>(sm + SCAN_OFF_IMG + IMG_HDR);
            const float minv = hdr[HDR_MINV + (part >> 1)], msum = fmaxf(hdr[HDR_MSUM], hdr[HDR_MSUM + 1]);
            const float kmax = hdr[HDR_KMAX];
            float invk, invR, invU, invS1;
            pow2_scale(kmax, KQ_LO, KQ_HI, invk);
            const float bR = bv + float(K) * kmax * bS;
            const float sR = pow2_scale(bR, VS_LO, VS_HI, invR);
            const float bU = msum * bR;
            const float sU = pow2_scale(bU, VS_LO, VS_HI, invU);
            float sS = pow2_scale(bS + 64.f * kmax * bU, VS_LO, VS_HI, invS1);
            // (M has no values: where its loss would count, the join takes the segment token by token)
            bool weak = run == 0 && __any_sync(0xffffffffu, bR > SCAN_WEAK_V * bv);
            if (weak) {                                    // the same in the four warps of the quarter
                prep_wait(ok, &bars[SB_GAM + ph], (cc >> 1) & 1, p.err);
                float gmax = 0.f;
#pragma unroll 1
                for (int i = 0; i < K; ++i) gmax = fmaxf(gmax, gam[ph * 128 + i]);
                weak = __all_sync(0xffffffffu, gmax < SCAN_WEAK_G);
                if (weak) {
                    scan_tokens<T, !TRANS>(p, S, x.row + 64 * c, left < 64 ? left : 64, x.h, part, v, quarter,
                                   reinterpret_cast<float *>(sm + SCAN_OFF_SUM));
                    float m = state_max(), unused = 0.f;
                    lane_max(m, unused);
                    sS = pow2_scale(m, VS_LO, VS_HI, invS1);           // the new state's own bound
                }
            }
            if (!TRANS && part == 0) sout[ph * 128 + v] = weak ? both(-1.f) : make_float2(invS, invU);
            // R = V - (K e^G) S, scaled
            accumulator(SB_D1, ph);
            {
                const float2 f = both(-invS * invk * sR), s2 = both(sR);
                float x[16];
                uint32_t hi[8], lo[8];
                tc::ld16(tq + TM_D1 + t0, x);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2 w;
                    if constexpr (sizeof(T) == 2) w = vr[i].wide();
                    else w = run == 1 ? both(0.f) : make_float2(widen1(sv[2 * i * 128]), widen1(sv[(2 * i + 1) * 128]));
                    w = __ffma2_rn(f, make_float2(x[2 * i], x[2 * i + 1]), __fmul2_rn(w, s2));
                    split_f16(w.x, w.y, hi[i], lo[i]);
                }
                tc::st8(rop, hi);
                tc::st8(rop + TM_RLO - TM_RHI, lo);
            }
            if (left < 64) fence_proxy_async();            // zeros written into v's tile, before the next copy there
            release(SB_R);
            if (run == 0 && lane == 0) mbar_arrive(&bars[SB_V_EMPTY]);
            // U = M R
            accumulator(SB_D2, ph);
            {
                float x[16];
                tc::ld16(tq + TM_D1 + t0, x);
                tc::wait_ld();
                put_operand(rop, rop + TM_RLO - TM_RHI, x, invR * minv * sU);
            }
            release(SB_U);
            const bool more = c + 1 < x.nc;                // the next walk puts its own state
            float bvn = more ? values(left - 64) : 0.f;
            // S1 = diag(e^{G_C}) S + (K e^{G_C-G})^T U
            prep_wait(ok, &bars[SB_GAM + ph], (cc >> 1) & 1, p.err);
            accumulator(SB_D3, ph);
            float mx = 0.f;
            if (weak) {                                    // S is there
                if (more) put_state(sS);
                mx = state_max();
            } else if (held) {                             // channels past K stay zero
                const float2 f = both(invU * invk);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float x[16];
                    tc::ld16(tq + TM_D3 + 32 * part + 16 * b, x);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 gm = *reinterpret_cast<const float2 *>(gam + ph * 128 + 32 * part + 16 * b + i);
                        const float2 w = __ffma2_rn(gm, make_float2(S[16 * b + i], S[16 * b + i + 1]),
                                                    __fmul2_rn(f, make_float2(x[i], x[i + 1])));
                        mx = max3(mx, w.x, w.y);
                        S[16 * b + i] = x[i] = w.x;
                        S[16 * b + i + 1] = x[i + 1] = w.y;
                    }
                    if (more) put_operand(sop + 8 * b, sop + TM_SLO - TM_SHI + 8 * b, x, sS);
                }
            }
            if (more) {
                release(SB_S);
                lane_max(mx, bvn);
                bS = mx;
                bv = bvn;
                invS = invS1;
            }
        }
        if (to != nullptr && mine) {
            float *sp = to + int64_t(32 * part) * W + v;
#pragma unroll
            for (int i = 0; i < 32; ++i) sp[int64_t(i) * W] = S[i];
        }
        }
    } else if (warp < 24) {
        // (64 registers, as at launch)
        // --------------------------------------------------------------- operands
        constexpr float L2E = 1.4426950408889634f;
        using W2 = Two<T>;
        using raw = typename W2::raw;
        const int rg = warp - 16;                          // rows 8 rg .. + 7
        float *tot = reinterpret_cast<float *>(sm + SCAN_OFF_TOT);
        // this thread's first row in the staging buffer or in memory; its channels are 64 x + 2 lane and
        // the next one.  Channels past K are zeros where staged, else another's values under a scale of zero.
        const int ks = STAGED ? KP : p.Hk * K;
        unsigned char *st = sm + scan_off_st<T>();
        float *sg = reinterpret_cast<float *>(sm + SCAN_OFF_GH);
        uint32_t cc = 0;
        int4 next = entry(w0);
        for (int32_t w = w0; w < walks; w += wstep) {
        const Walk1 wk = walk_at(w, next);
        next = entry(w + wstep);
        const int h = wk.h, hk = h / (p.H / p.Hk);
        const unsigned char *img0 = image_at(wk);
        for (int c = 0; c < wk.nc; ++c, ++cc) {
            const uint32_t ph = cc & 1;
            const int left = wk.rows - 64 * c - 8 * rg;    // live rows from this thread's first on
            const int64_t row = wk.row + 64 * c + 8 * rg;
            const T *kp, *qp;
            const float *gp = reinterpret_cast<float *>(st + scan_off_g<T>(KP)) + 8 * rg * KP;
            if (STAGED) {
                kp = reinterpret_cast<T *>(st) + 8 * rg * KP;
                qp = reinterpret_cast<T *>(st + 16384) + 8 * rg * KP;
            } else {
                kp = static_cast<const T *>(p.k) + (row * p.Hk + hk) * K;
                qp = static_cast<const T *>(p.q) + (row * p.Hk + hk) * K;
            }
            if (p.gate != 0) {                             // one decay to a row
                if (lane < 8) sg[8 * rg + lane] = lane < left ? p.g[(row + lane) * p.H + h] : 0.f;
                __syncwarp();
                gp = sg + 8 * rg;
            }
            const float2 kqmax = *reinterpret_cast<const float2 *>(img0 + c * img_step + IMG_HDR + 4 * HDR_KMAX);
            if (STAGED || p.gate == 0) {
                prep_wait(ok, &bars[SB_ST_FULL], ph, p.err);
#pragma unroll 1
                for (int i = left > 0 ? left : 0; i < 8; ++i)      // rows past the end hold the next request's
#pragma unroll 1
                    for (int x = lane; x < K; x += 32) {
                        if (STAGED) {
                            const_cast<T *>(kp)[i * ks + x] = T(0.f);
                            const_cast<T *>(qp)[i * ks + x] = T(0.f);
                        }
                        if (p.gate == 0) const_cast<float *>(gp)[i * KP + x] = 0.f;
                    }
                __syncwarp();
            }
            auto chan = [&](int x) { const int d = 64 * x + 2 * lane; return STAGED || W128 || d < K ? d : 2 * lane % K; };
            auto two = [&](const T *at, int i, int d) {
                const bool in = STAGED || i < left;
                return in ? *reinterpret_cast<const raw *>(at + i * ks + d) : raw{};
            };
            auto decay = [&](int i, int d) {
                if (p.gate != 0) return both(gp[i]);
                return *reinterpret_cast<const float2 *>(gp + i * KP + d);
            };
            // above 64 channels a lane has four in a row for the first two passes: half the loads and stores
            // of two (the scan of 16 x 512 tokens, 64 heads: 263 us, not 267)
            struct alignas(2 * sizeof(raw)) raw4 { raw r[2]; };
            auto four = [&](const T *at, int i) {
                const bool in = STAGED || i < left;
                return in ? *reinterpret_cast<const raw4 *>(at + i * ks + 4 * lane) : raw4{};
            };
            auto decay4 = [&](int i) {
                if (p.gate != 0) return make_float4(gp[i], gp[i], gp[i], gp[i]);
                return *reinterpret_cast<const float4 *>(gp + i * KP + 4 * lane);
            };
            if (FOUR) {
                float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 t = decay4(i);
                    s0 = __ffma2_rn(make_float2(t.x, t.y), both(L2E), s0);      // in powers of two
                    s1 = __ffma2_rn(make_float2(t.z, t.w), both(L2E), s1);
                }
                *reinterpret_cast<float4 *>(tot + rg * 128 + 4 * lane) = make_float4(s0.x, s0.y, s1.x, s1.y);
            }
#pragma unroll 1
            for (int x = 0; !FOUR && x < nh; ++x) {
                float2 sum = both(0.f);
                const int d = chan(x);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = __ffma2_rn(decay(i, d), both(L2E), sum);   // in powers of two
                *reinterpret_cast<float2 *>(tot + rg * 128 + 64 * x + 2 * lane) = sum;
            }
            float inv, unused, gmax = 0.f;
            const float sk1 = pow2_scale(kqmax.x, KQ_LO, KQ_HI, inv);
            const float2 cq = both(p.scale * pow2_scale(kqmax.y * fabsf(p.scale), KQ_LO, KQ_HI, unused) * inv);
            named_sync<1, 256>();
            // K e^G and scale Q e^G: row r of a tile is 128 bytes, its 16-byte chunk lane / 4 at (lane / 4) ^ (r & 7)
            prep_wait(ok, &bars[SB_KQ_EMPTY], ph ^ 1, p.err);
            if (FOUR) {
                float2 G[2] = {both(0.f), both(0.f)};
                for (int w = 0; w < rg; ++w) {
                    const float4 t = *reinterpret_cast<const float4 *>(tot + w * 128 + 4 * lane);
                    G[0] = __fadd2_rn(G[0], make_float2(t.x, t.y));
                    G[1] = __fadd2_rn(G[1], make_float2(t.z, t.w));
                }
                unsigned char *kq = sm + SCAN_OFF_KQ + (lane >> 4) * 8192 + rg * 1024 + 8 * (lane & 1);
#pragma unroll 1
                for (int b = 0; b < 8; b += 4) {
                    raw4 rk[4], rq[4];                     // all loads before the first store
                    float4 g[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        rk[i] = four(kp, b + i);
                        if (!TRANS) rq[i] = four(qp, b + i);
                        g[i] = decay4(b + i);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t kh[2], kl[2], qh[2], ql[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            G[j] = __ffma2_rn(j == 0 ? make_float2(g[i].x, g[i].y) : make_float2(g[i].z, g[i].w), both(L2E), G[j]);
                            const float2 e = __fmul2_rn(make_float2(ex2(G[j].x), ex2(G[j].y)), both(sk1));
                            const float2 kv = __fmul2_rn(W2::wide(rk[i].r[j]), e);
                            split_f16(kv.x, kv.y, kh[j], kl[j]);
                            if (!TRANS) {
                                const float2 qv = __fmul2_rn(W2::wide(rq[i].r[j]), __fmul2_rn(e, cq));
                                split_f16(qv.x, qv.y, qh[j], ql[j]);
                            }
                        }
                        unsigned char *at = kq + (b + i) * 128 + 16 * (((lane & 15) >> 1) ^ (b + i));
                        *reinterpret_cast<uint2 *>(at) = make_uint2(kh[0], kh[1]);
                        *reinterpret_cast<uint2 *>(at + 16384) = make_uint2(kl[0], kl[1]);
                        if (!TRANS) *reinterpret_cast<uint2 *>(at + 32768) = make_uint2(qh[0], qh[1]);
                        if (!TRANS) *reinterpret_cast<uint2 *>(at + 49152) = make_uint2(ql[0], ql[1]);
                    }
                }
                if (rg == 7) {                             // here G is the whole chunk's sum
                    const float4 e = make_float4(ex2(G[0].x), ex2(G[0].y), ex2(G[1].x), ex2(G[1].y));
                    *reinterpret_cast<float4 *>(gam + ph * 128 + 4 * lane) = e;
                    if (4 * lane < K) gmax = fmaxf(fmaxf(e.x, e.y), fmaxf(e.z, e.w));
                }
            }
#pragma unroll 1
            for (int x = 0; !FOUR && x < nh; ++x) {
                const float *tb = tot + 64 * x + 2 * lane;
                float2 G = both(0.f);
                for (int w = 0; w < rg; ++w) G = __fadd2_rn(G, *reinterpret_cast<const float2 *>(tb + w * 128));
                unsigned char *kq = sm + SCAN_OFF_KQ + x * 8192 + rg * 1024 + 4 * (lane & 3);
                const int d = chan(x);
                const float2 sk = both(STAGED || W128 || 64 * x + 2 * lane < K ? sk1 : 0.f);
#pragma unroll 1
                for (int b = 0; b < 8; b += 4) {
                    raw rk[4], rq[4];                      // all loads before the first store
                    float2 g[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        rk[i] = two(kp, b + i, d);
                        if (!TRANS) rq[i] = two(qp, b + i, d);
                        g[i] = decay(b + i, d);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        G = __ffma2_rn(g[i], both(L2E), G);
                        const float2 e = __fmul2_rn(make_float2(ex2(G.x), ex2(G.y)), sk);
                        const float2 kv = __fmul2_rn(W2::wide(rk[i]), e);
                        uint32_t kh, kl, qh = 0u, ql = 0u;
                        split_f16(kv.x, kv.y, kh, kl);
                        if (!TRANS) {
                            const float2 qv = __fmul2_rn(W2::wide(rq[i]), __fmul2_rn(e, cq));
                            split_f16(qv.x, qv.y, qh, ql);
                        }
                        unsigned char *at = kq + (b + i) * 128 + 16 * ((lane >> 2) ^ (b + i));
                        *reinterpret_cast<uint32_t *>(at) = kh;
                        *reinterpret_cast<uint32_t *>(at + 16384) = kl;
                        if (!TRANS) *reinterpret_cast<uint32_t *>(at + 32768) = qh;
                        if (!TRANS) *reinterpret_cast<uint32_t *>(at + 49152) = ql;
                    }
                }
                if (rg == 7) {                             // here G is the whole chunk's sum
                    const float2 e = make_float2(ex2(G.x), ex2(G.y));
                    *reinterpret_cast<float2 *>(gam + ph * 128 + 64 * x + 2 * lane) = e;
                    if (64 * x + 2 * lane < K) gmax = fmaxf(gmax, fmaxf(e.x, e.y));
                }
            }
            if (TRANS && rg == 7 && wk.run == 1) {         // for the join
                gmax = warp_max(gmax);
                if (lane == 0)
                    *reinterpret_cast<float *>(const_cast<unsigned char *>(img0) + c * img_step + IMG_HDR + 4 * HDR_GMAX) = gmax;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[SB_KQ_FULL]);
                // e^{G_C} for the chain, on barriers for even and odd chunks: the next chunk's may come
                // before a slow warp of the chain has seen this one's, but not the one's after
                if (rg == 7) mbar_arrive(&bars[SB_GAM + ph]);
            }
            // K e^{G_C-G} transposed: channel d's row holds the 64 tokens, eight to a 16-byte chunk
            prep_wait(ok, &bars[SB_KH_EMPTY], ph ^ 1, p.err);
#pragma unroll 1
            for (int x = 0; x < nh; ++x) {
                const float *tb = tot + 64 * x + 2 * lane;
                float2 after = both(0.f), y[8], g[8];
                const int dc = chan(x);
                const float2 sk = both(STAGED || W128 || 64 * x + 2 * lane < K ? sk1 : 0.f);
                for (int w = 7; w > rg; --w) after = __fadd2_rn(after, *reinterpret_cast<const float2 *>(tb + w * 128));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = W2::wide(two(kp, i, dc));
                    g[i] = decay(i, dc);
                }
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    y[i] = __fmul2_rn(y[i], __fmul2_rn(make_float2(ex2(after.x), ex2(after.y)), sk));
                    after = __ffma2_rn(g[i], both(L2E), after);
                }
                // the staged chunk is read.  The loads must be done, not on their way, before a copy may follow:
                // hence after what uses them, and with the fence.  (Without both, one run in fifteen with
                // three walks to a CTA took some row's decays from the next chunk.)
                if (x == nh - 1) {
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[SB_ST_EMPTY]);
                }
                uint4 ah, al, bh, bl;
                split_f16(y[0].x, y[1].x, ah.x, al.x); split_f16(y[2].x, y[3].x, ah.y, al.y);
                split_f16(y[4].x, y[5].x, ah.z, al.z); split_f16(y[6].x, y[7].x, ah.w, al.w);
                split_f16(y[0].y, y[1].y, bh.x, bl.x); split_f16(y[2].y, y[3].y, bh.y, bl.y);
                split_f16(y[4].y, y[5].y, bh.z, bl.z); split_f16(y[6].y, y[7].y, bh.w, bl.w);
                const int d = 64 * x + 2 * lane;
                unsigned char *a0 = sm + SCAN_OFF_KH + d * 128 + 16 * (rg ^ (d & 7));
                unsigned char *a1 = sm + SCAN_OFF_KH + (d + 1) * 128 + 16 * (rg ^ ((d + 1) & 7));
                *reinterpret_cast<uint4 *>(a0) = ah;
                *reinterpret_cast<uint4 *>(a0 + 16384) = al;
                *reinterpret_cast<uint4 *>(a1) = bh;
                *reinterpret_cast<uint4 *>(a1 + 16384) = bl;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_KH_FULL]);
            named_sync<1, 256>();                          // the sums are consumed
        }
        }
    } else if (warp < 28) {
        tc::fewer_registers<40>();
        // ----------------------------------------------------------------- output
        const int quarter = warp & 3, v = 32 * quarter + lane;
        const uint32_t tq = tmem + (uint32_t(32 * quarter) << 16);
        const bool mine = v < V;
        const float2 *sout = reinterpret_cast<const float2 *>(sm + SCAN_OFF_OUT);
        // token 8 b + i of a chunk: a base that is the same for the warp, and this lane's offset of row i
        const uint32_t step = uint32_t(p.H) * V * sizeof(T);
        uint32_t off[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) off[i] = v * sizeof(T) + i * step;
        uint32_t cc = 0;
        int4 next = entry(w0);
        for (int32_t w = w0; !TRANS && w < walks; w += wstep) {
        const Walk1 wk = walk_at(w, next);
        next = entry(w + wstep);
        unsigned char *const ob = static_cast<unsigned char *>(p.o) + (int64_t(wk.row) * p.H + wk.h) * V * int64_t(sizeof(T));
        for (int c = 0; c < wk.nc; ++c, ++cc) {
            const uint32_t ph = cc & 1;
            // O = (scale Q e^G) S0 + P U
            prep_wait(ok, &bars[SB_U], ph, p.err);         // the chain's scales
            const float2 inv = sout[ph * 128 + v];
            const float *hdr = reinterpret_cast<const float *>(sm + SCAN_OFF_IMG + IMG_HDR);
            prep_wait(ok, &bars[SB_IMG_FULL], ph, p.err);
            const float p0 = hdr[HDR_PINV], p1 = hdr[HDR_PINV + 1], qmax = hdr[HDR_QMAX];
            float invq;
            pow2_scale(qmax * fabsf(p.scale), KQ_LO, KQ_HI, invq);
            fence_proxy_async();                           // read before the next image's copy
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_IMG_READ]);
            prep_wait(ok, &bars[SB_O_FULL], ph, p.err);
            __syncwarp();
            tc::fence_after_sync();
            const bool weak = inv.x < 0.f;
            const int left = mine && !weak ? wk.rows - 64 * c : 0;
            const bool whole = __all_sync(0xffffffffu, left >= 64);
            const float2 f = both(inv.x * invq);
#pragma unroll 1
            for (int b = 0; b < 8; ++b) {
                const float2 f2 = both(inv.y * (b < 4 ? p0 : p1));
                float x[8], y[8];
                tc::ld8(tq + TM_O1 + 8 * b, x);
                tc::ld8(tq + TM_O2 + 8 * b, y);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 w = __ffma2_rn(f, make_float2(x[i], x[i + 1]), __fmul2_rn(f2, make_float2(y[i], y[i + 1])));
                    x[i] = w.x;
                    x[i + 1] = w.y;
                }
                unsigned char *o = ob + int64_t(64 * c + 8 * b) * step;
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) put1(reinterpret_cast<T *>(o + off[i]), x[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (8 * b + i < left) put1(reinterpret_cast<T *>(o + off[i]), x[i]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SB_O_EMPTY]);
        }
        }
    } else {
        tc::fewer_registers<24>();
        if (warp == 28) {
            // --------------------------------------------------------- MMA issue
            const uint32_t kq = smem_u32(sm + SCAN_OFF_KQ), kh = smem_u32(sm + SCAN_OFF_KH);
            const int steps = 4 * nh;                      // of 16 channels
            const uint32_t id3 = nh == 2 ? SCAN_ID128 : SCAN_ID64;
            auto commit = [&](int b) { tc::commit(smem_u32(&bars[b])); };
            auto wait = [&](int b, uint32_t parity) { prep_wait(ok, &bars[b], parity, p.err); };
            uint32_t c = 0, end = 0;                       // chunks so far, and at the end of this walk
            int4 next = entry(w0);
            for (int32_t w = w0; w < walks; w += wstep) {
            end += walk_at(w, next).nc;
            next = entry(w + wstep);
            for (; c < end; ++c) {
                const uint32_t ph = c & 1;
                const uint32_t img = smem_u32(sm + SCAN_OFF_IMG);
                wait(SB_KQ_FULL, ph);
                wait(SB_S, ph);
                __syncwarp();
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    mma_split(steps, tmem + TM_D1, tmem + TM_SHI, tmem + TM_SLO, kq, kq + 16384, 8192, SCAN_ID64);
                    commit(SB_D1);
                    if (TRANS) commit(SB_KQ_EMPTY);
                }
                if (!TRANS) wait(SB_O_EMPTY, ph ^ 1);
                __syncwarp();
                tc::fence_after_sync();
                if (!TRANS && tc::elect_one()) {
                    mma_split(steps, tmem + TM_O1, tmem + TM_SHI, tmem + TM_SLO, kq + 32768, kq + 49152, 8192,
                                    SCAN_ID64);
                    commit(SB_KQ_EMPTY);
                }
                wait(SB_IMG_FULL, ph);
                wait(SB_R, ph);
                __syncwarp();
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    mma_split(4, tmem + TM_D1, tmem + TM_RHI, tmem + TM_RLO, img + IMG_MHI, img + IMG_MLO, 0,
                                     SCAN_ID64);
                    commit(SB_D2);
                }
                wait(SB_KH_FULL, ph);
                wait(SB_U, ph);
                __syncwarp();
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    mma_split(4, tmem + TM_D3, tmem + TM_RHI, tmem + TM_RLO, kh, kh + 16384, 0, id3);
                    commit(SB_D3);
                    commit(SB_KH_EMPTY);
                    if (!TRANS) {
                        mma_split(4, tmem + TM_O2, tmem + TM_RHI, tmem + TM_RLO, img + IMG_PHI, img + IMG_PLO, 0,
                                        SCAN_ID64);
                        commit(SB_O_FULL);
                    }
                    commit(SB_IMG_EMPTY);
                }
                __syncwarp();
            }
            }
        } else if (warp == 29) {
            // ------------------------------------------------- loads of q, k and g
            if (STAGED || p.gate == 0) {
                unsigned char *st = sm + scan_off_st<T>();
                const uint32_t bytes = (STAGED ? (TRANS ? 1 : 2) * 64 * KP * sizeof(T) : 0) + (p.gate == 0 ? 64 * KP * 4 : 0);
                uint32_t cc = 0;
                Walk1 wk = walk_at(w0, entry(w0));
                for (int32_t w = w0; w < walks; w += wstep) {
                    const Walk1 nx = walk_at(w + wstep, entry(w + wstep));
                    const int hk = wk.h / (p.H / p.Hk);
                    for (int c = 0; c < wk.nc; ++c, ++cc) {
                        prep_wait(ok, &bars[SB_ST_EMPTY], (cc & 1) ^ 1, p.err);
                        __syncwarp();
                        if (tc::elect_one()) {
                            const int r = wk.row + 64 * c;
                            mbar_arrive_expect_tx(&bars[SB_ST_FULL], bytes);
                            if (STAGED) tma_load_3d(st, &maps.k, 0, hk, r, &bars[SB_ST_FULL]);
                            if (STAGED && !TRANS) tma_load_3d(st + 16384, &maps.q, 0, hk, r, &bars[SB_ST_FULL]);
                            if (p.gate == 0) tma_load_3d(st + scan_off_g<T>(KP), &maps.g, 0, wk.h, r, &bars[SB_ST_FULL]);
                            // the next chunk's on their way to L2 meanwhile
                            const bool more = c + 1 < wk.nc;
                            if (more || nx.nc > 0) {
                                const int pr = more ? r + 64 : nx.row, ph = more ? wk.h : nx.h, pk = ph / (p.H / p.Hk);
                                tc::prefetch_3d(&maps.k, 0, pk, pr);
                                if (!TRANS) tc::prefetch_3d(&maps.q, 0, pk, pr);
                                if (p.gate == 0) tc::prefetch_3d(&maps.g, 0, ph, pr);
                            }
                        }
                        __syncwarp();
                    }
                    wk = nx;
                }
                if (cc > 0) prep_wait(ok, &bars[SB_ST_FULL], (cc - 1) & 1, p.err);
            }
        } else if (warp == 30) {
            // --------------------------------------------------------- loads of v
            uint32_t cc = 0;                               // chunks that have values
            int4 next = entry(w0);
            for (int32_t w = w0; w < walks; w += wstep) {
                const Walk1 wk = walk_at(w, next);
                next = entry(w + wstep);
                for (int c = 0; wk.run == 0 && c < wk.nc; ++c, ++cc) {
                    prep_wait(ok, &bars[SB_V_EMPTY], (cc & 1) ^ 1, p.err);
                    __syncwarp();
                    if (tc::elect_one()) {
                        mbar_arrive_expect_tx(&bars[SB_V_FULL], 64 * 128 * sizeof(T));
                        tma_load_3d(sm + SCAN_OFF_V, &maps.v, 0, wk.h, wk.row + 64 * c, &bars[SB_V_FULL]);
                        if (c + 1 < wk.nc) tc::prefetch_3d(&maps.v, 0, wk.h, wk.row + 64 * c + 64);
                    }
                    __syncwarp();
                }
            }
            if (cc > 0) prep_wait(ok, &bars[SB_V_FULL], (cc - 1) & 1, p.err);
        } else {
            // ------------------------------------------------- loads of M and P
            uint32_t cc = 0;
            int4 next = entry(w0);
            for (int32_t w = w0; w < walks; w += wstep) {
                const Walk1 wk = walk_at(w, next);
                next = entry(w + wstep);
                const unsigned char *src = image_at(wk);
                for (int c = 0; c < wk.nc; ++c, ++cc, src += img_step) {
                    prep_wait(ok, &bars[SB_IMG_EMPTY], (cc & 1) ^ 1, p.err);
                    if (!TRANS) prep_wait(ok, &bars[SB_IMG_READ], (cc & 1) ^ 1, p.err);
                    __syncwarp();
                    if (tc::elect_one()) {
                        unsigned char *img = sm + SCAN_OFF_IMG;
                        uint64_t *full = &bars[SB_IMG_FULL];
                        if (TRANS) {                       // M and the header
                            mbar_arrive_expect_tx(full, IMG_PHI + IMG_HDR_BYTES);
                            bulk_load(img, src, IMG_PHI, full);
                            bulk_load(img + IMG_HDR, src + IMG_HDR, IMG_HDR_BYTES, full);
                        } else {
                            mbar_arrive_expect_tx(full, IMG_BYTES);
                            bulk_load(img, src, IMG_BYTES, full);
                        }
                        if (c + 1 < wk.nc) tc::prefetch_bulk(src + img_step, TRANS ? IMG_PHI : IMG_BYTES);
                    }
                    __syncwarp();
                }
            }
            if (cc > 0) prep_wait(ok, &bars[SB_IMG_FULL], (cc - 1) & 1, p.err);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// The segments' maps chained: the state that segment i + 1 of a sequence starts from replaces N of
// segment i.  A block has 16 columns of one sequence-head, a thread four of them in two rows.  FP32;
// the sequence's first segment gave its state itself.  M comes through shared memory 64 columns
// at a time, the next ones' copy under way during a product: at that size two blocks share an SM,
// and the 256 blocks of 32 heads are one wave (8 segments: 45 us, 57 with all of M staged; 49 with the
// check that follows).
//
// M's columns are as good as 2^-34 or so of what went into each chunk, so where a chunk clears the state
// M can have lost what little is left of it.  That counts where the state that comes in is so large
// that the rest of it, M S, is not lost beside N.  A block which finds M S below JOIN_FALL of S in a column, but not
// below 2^-20 of the sum, looks for such a chunk in the segment, and if there is one walks the
// segment token by token (join_tokens): about a microsecond a token.
constexpr int JOIN_THREADS = 256, JOIN_COLS = 16, JOIN_PITCH = 68;
constexpr int JOIN_BYTES = 2 * 128 * JOIN_PITCH * 4;
constexpr float JOIN_FALL = 1.f / 256.f, JOIN_COUNTS = 1.f / 1048576.f;

struct JoinShared {
    float S[128][JOIN_COLS];
    float k[2][128], d[2][128];                             // join_tokens: a token's key and decays
    float part[2][8][JOIN_COLS];                            // the warps' sums or maxima
    int32_t red[8];
};

// Whether one of the `n` chunks from `chunk` on keeps less than SCAN_WEAK_G of every channel of head h, from what
// M's walk left in their images (reading the decays themselves took 50 us at 1 x 2048 tokens x 32 heads).  The
// same for all threads.
__device__ __forceinline__ bool join_cleared(const DeltaParams &p, int64_t chunk, int n, int h) {
    bool any = false;
    for (int i = int(threadIdx.x); i < n && (chunk + i + 1) * p.H <= p.n_tasks; i += JOIN_THREADS)
        any |= *reinterpret_cast<const float *>(p.ws + ((chunk + i) * p.H + h) * IMG_BYTES + IMG_HDR + 4 * HDR_GMAX) < SCAN_WEAK_G;
    return __syncthreads_or(any) != 0;
}

// The state of rows r, r + 1 and columns c .. + 3 of the block's after rows a .. b, token by token in FP32.
template <typename T>
__device__ __forceinline__ void join_tokens(const DeltaParams &p, JoinShared &sh, float4 (&s)[2], int64_t a, int64_t b, int h,
                                            int r, int c, int column) {
    const int tid = threadIdx.x, hk = h / (p.H / p.Hk);
    const bool in = r < p.K;
    s[0] = in ? *reinterpret_cast<const float4 *>(&sh.S[r][c]) : make_float4(0.f, 0.f, 0.f, 0.f);
    s[1] = in ? *reinterpret_cast<const float4 *>(&sh.S[r + 1][c]) : make_float4(0.f, 0.f, 0.f, 0.f);
    float nk = 0.f, ng = 0.f;                               // channel tid's key and log decay of the token that comes next
    auto fetch = [&](int64_t t) {
        if (t < b && tid < p.K) {
            nk = widen1(static_cast<const T *>(p.k)[(t * p.Hk + hk) * p.K + tid]);
            ng = p.g[p.gate == 0 ? (t * p.H + h) * p.K + tid : t * p.H + h];
        }
    };
    auto put = [&](int at) {
        if (tid < 128) {
            sh.k[at][tid] = tid < p.K ? nk : 0.f;
            sh.d[at][tid] = tid < p.K ? expf(ng) : 0.f;
        }
    };
    fetch(a);
    put(0);
    fetch(a + 1);
    __syncthreads();
#pragma unroll 1
    for (int64_t t = a; t < b; ++t) {
        const int at = int(t - a) & 1;
        const T *vp = static_cast<const T *>(p.v) + (t * p.H + h) * p.V + column + c;
        const float beta = widen1(static_cast<const T *>(p.beta)[t * p.H + h]);
        const float v[4] = {widen1(vp[0]), widen1(vp[1]), widen1(vp[2]), widen1(vp[3])};
        const float k0 = sh.k[at][r], k1 = sh.k[at][r + 1], d0 = sh.d[at][r], d1 = sh.d[at][r + 1];
        s[0].x *= d0; s[0].y *= d0; s[0].z *= d0; s[0].w *= d0;
        s[1].x *= d1; s[1].y *= d1; s[1].z *= d1; s[1].w *= d1;
        float x[4] = {fmaf(k1, s[1].x, k0 * s[0].x), fmaf(k1, s[1].y, k0 * s[0].y), fmaf(k1, s[1].z, k0 * s[0].z),
                      fmaf(k1, s[1].w, k0 * s[0].w)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
        if ((tid & 31) < 4) *reinterpret_cast<float4 *>(&sh.part[at][tid >> 5][c]) = make_float4(x[0], x[1], x[2], x[3]);
        put(at ^ 1);                                        // (read last before the barrier of the token before)
        fetch(t + 2);
        __syncthreads();
        float u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) sum += sh.part[at][w][c + e];
            u[e] = beta * (v[e] - sum);
        }
        s[0] = make_float4(fmaf(k0, u[0], s[0].x), fmaf(k0, u[1], s[0].y), fmaf(k0, u[2], s[0].z), fmaf(k0, u[3], s[0].w));
        s[1] = make_float4(fmaf(k1, u[0], s[1].x), fmaf(k1, u[1], s[1].y), fmaf(k1, u[2], s[1].z), fmaf(k1, u[3], s[1].w));
    }
    __syncthreads();                                        // part is used again
}

template <typename T>
__global__ void __launch_bounds__(JOIN_THREADS) kda_delta_join_kernel(const DeltaParams p) {
    extern __shared__ __align__(16) float join_m[];
    __shared__ __align__(16) JoinShared sh;
    auto &S = sh.S;
    auto &red = sh.red;
    const int tid = threadIdx.x, r = 2 * (tid >> 2), c = 4 * (tid & 3);
    const int slices = p.V / JOIN_COLS, slice = int(blockIdx.x) % slices, nh = int(blockIdx.x) / slices;
    const int n = nh / p.H, h = nh - n * p.H;
    pdl_launch_dependents();
    pdl_wait();
    // the sequence's first unit, and its units
    int32_t u0 = 0, parts;
    if (p.cu == nullptr) {
        parts = max(1, (p.cpr + p.seg - 1) / p.seg);
        u0 = n * parts;
    } else {
        for (int i = tid; i < n; i += JOIN_THREADS)
            u0 += max(1, (nchunks<BT>(__ldg(p.cu + i), __ldg(p.cu + i + 1)) + p.seg - 1) / p.seg);
        u0 = __reduce_add_sync(0xffffffffu, u0);
        if ((tid & 31) == 0) red[tid >> 5] = u0;
        __syncthreads();
        u0 = 0;
        for (int w = 0; w < JOIN_THREADS / 32; ++w) u0 += red[w];
        parts = max(1, (nchunks<BT>(__ldg(p.cu + n), __ldg(p.cu + n + 1)) + p.seg - 1) / p.seg);
    }
    if (u0 < 0 || int64_t(u0) + parts > p.n_units) return;  // malformed cu_seqlens
    const int64_t sz = int64_t(p.K) * p.V, tz = sz + int64_t(p.K) * p.K;
    float *map0 = p.trans + (int64_t(u0) * p.H + h) * tz;
    const int halves = p.K > 64 ? 2 : 1;
    auto fetch = [&](int j) {                               // columns 64 (j % halves) .. of segment j / halves's M
        const int i = halves == 2 ? j >> 1 : j, k0 = halves == 2 ? 64 * (j & 1) : 0;
        if (i < parts - 1) {
            const int k4 = min(64, p.K - k0) / 4;           // 16-byte pieces of a row
            const float *m = map0 + int64_t(i) * p.H * tz + sz + k0;
            float *to = join_m + (j & 1) * 128 * JOIN_PITCH;
            for (int x4 = tid; x4 < p.K * k4; x4 += JOIN_THREADS) {
                const int row = x4 / k4, x = 4 * (x4 - row * k4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + row * JOIN_PITCH + x)),
                             "l"(m + int64_t(row) * p.K + x) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int64_t at = int64_t(r) * p.V + JOIN_COLS * slice + c;
    auto row = [&](int i, int j) { return reinterpret_cast<float4 *>(map0 + int64_t(i) * p.H * tz + at + int64_t(j) * p.V); };
    if (parts > 2 && r < p.K) {                             // the state after the first segment
        *reinterpret_cast<float4 *>(&S[r][c]) = *row(0, 0);
        *reinterpret_cast<float4 *>(&S[r + 1][c]) = *row(0, 1);
    }
    fetch(halves);
    // the largest values of column tid of 16 after the segment before (columns_max's)
    auto columns_max = [&](const float4 (&x)[2], int to) {
        float m[4] = {fmaxf(fabsf(x[0].x), fabsf(x[1].x)), fmaxf(fabsf(x[0].y), fabsf(x[1].y)),
                      fmaxf(fabsf(x[0].z), fabsf(x[1].z)), fmaxf(fabsf(x[0].w), fabsf(x[1].w))};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o));
        if ((tid & 31) < 4) *reinterpret_cast<float4 *>(&sh.part[to][tid >> 5][c]) = make_float4(m[0], m[1], m[2], m[3]);
    };
    auto column_max = [&](int from) {
        float m = 0.f;
#pragma unroll
        for (int w = 0; w < JOIN_THREADS / 32; ++w) m = fmaxf(m, sh.part[from][w][tid & (JOIN_COLS - 1)]);
        return m;
    };
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    float before = 0.f;
    if (parts > 2) {
        const float4 s[2] = {r < p.K ? *row(0, 0) : zero4, r < p.K ? *row(0, 1) : zero4};
        columns_max(s, 0);
        __syncthreads();
        before = column_max(0);
        __syncthreads();
    }
    for (int i = 1; i < parts - 1; ++i) {
        float4 a[2] = {zero4, zero4}, n4[2] = {zero4, zero4};
        if (r < p.K) {
            n4[0] = *row(i, 0);
            n4[1] = *row(i, 1);
        }
        for (int j = halves * i; j < halves * (i + 1); ++j) {
            fetch(j + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            if (r < p.K) {
                const int k0 = 64 * (j - halves * i), kn = min(64, p.K - k0);
                const float *m = join_m + (j & 1) * 128 * JOIN_PITCH + r * JOIN_PITCH;
#pragma unroll 2
                for (int k = 0; k < kn; k += 4) {
                    const float4 m0 = *reinterpret_cast<const float4 *>(m + k), m1 = *reinterpret_cast<const float4 *>(m + JOIN_PITCH + k);
                    const float mk[2][4] = {{m0.x, m0.y, m0.z, m0.w}, {m1.x, m1.y, m1.z, m1.w}};
#pragma unroll
                    for (int e4 = 0; e4 < 4; ++e4) {
                        const float4 s = *reinterpret_cast<const float4 *>(&S[k0 + k + e4][c]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            a[e].x = fmaf(mk[e][e4], s.x, a[e].x); a[e].y = fmaf(mk[e][e4], s.y, a[e].y);
                            a[e].z = fmaf(mk[e][e4], s.z, a[e].z); a[e].w = fmaf(mk[e][e4], s.w, a[e].w);
                        }
                    }
                }
            }
            __syncthreads();
        }
        columns_max(a, 0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {                       // what goes out: N + M S
            n4[e].x += a[e].x; n4[e].y += a[e].y; n4[e].z += a[e].z; n4[e].w += a[e].w;
        }
        columns_max(n4, 1);
        __syncthreads();
        const float rest = column_max(0), after = column_max(1);
        if (__syncthreads_or(rest < JOIN_FALL * before && rest > JOIN_COUNTS * after)) {
            int64_t r0, r1;
            sequence_rows(p, n, r0, r1);
            r0 += int64_t(BT) * p.seg * i;
            if (r1 > r0 + int64_t(BT) * p.seg) r1 = r0 + int64_t(BT) * p.seg;
            const int64_t chunk = p.cu == nullptr ? int64_t(n) * p.cpr : int64_t(p.units[u0].z);
            if (join_cleared(p, max(int64_t(0), chunk) + int64_t(p.seg) * i, p.seg, h))
                join_tokens<T>(p, sh, n4, r0, r1, h, r, c, JOIN_COLS * slice);
            columns_max(n4, 1);
            __syncthreads();
            before = column_max(1);
            __syncthreads();
        } else {
            before = after;
        }
        if (r < p.K) {
            *row(i, 0) = *reinterpret_cast<float4 *>(&S[r][c]) = n4[0];
            *row(i, 1) = *reinterpret_cast<float4 *>(&S[r + 1][c]) = n4[1];
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace kda
