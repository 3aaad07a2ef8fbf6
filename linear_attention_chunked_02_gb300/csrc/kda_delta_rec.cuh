// kda_delta_rec.cuh -- the gated delta rule token by token, for decoding steps
// (one token to a sequence) and short prompts.
//
// With D = diag(exp(g)), one token maps the state S [K, V] and gives its output by
//     u = beta (v - (D S)^T k),   S' = D S + k u^T,
//     o = scale S'^T q = scale ((D S)^T q + (q . k) u),
// so both sums over K, (D S)^T k and (D S)^T q, are taken in one pass over the
// state, and the state is read and written once.
//
// A block holds VC = 4 CQ columns of one sequence-head's state in registers:
// thread (rg, cq) has the four columns 4 cq .. + 3 of rows rg, rg + RG, ..., so a
// row of the block's columns is read and written as consecutive 16-byte vectors.
// The partial sums over a thread's rows meet in shared memory.  All of it is
// FP32 FMA.  A decoding step is bound by HBM (the state in and out, K V 8 bytes
// to a request-head, against 7 K V operations): 256 requests of 64 heads, K = V = 128, take
// 313 us back to back, 6.9 TB/s, what a copy reaches.  Four blocks of 32 KB to an SM, so that the loads of
// some run beside the stores of others (two of 64 KB: 355 us), and loads and stores that do not
// stay in the L2 (318 us without).
#pragma once

#include "kda_kernels.cuh"

namespace kda {

struct DeltaParams {
    const void *q, *k, *v;      // [rows, Hk, K], [rows, Hk, K], [rows, H, V]
    const float *g;             // [rows, H, K] or [rows, H]
    const void *beta;           // [rows, H]
    void *o;                    // [rows, H, V]
    const float *state_in;      // [entries, H, K, V] or nullptr
    float *state_out;           // likewise
    const int32_t *slots;       // [sequences] or nullptr
    int32_t num_slots;
    const int32_t *cu;          // packed: cu_seqlens; dense: nullptr
    int32_t nseq;               // sequences (dense: batch rows)
    int64_t T;                  // dense: rows per batch row; packed: total rows
    int32_t Hk, H, K, V;
    int32_t gate;               // kda_gate_t
    float scale;
    unsigned *err;              // device error word
    // the chunked form
    int32_t cpr;                // dense: chunks per batch row
    int32_t n_tasks;            // bound on chunk-heads
    unsigned char *ws;          // workspace: one image to a chunk-head
    int32_t seg;                // chunks to a segment of a sequence; 0: sequences are not split
    int32_t n_units;            // bound on segments (seg == 0: sequences)
    float *trans;               // [n_units][H]{N [K, V], M [K, K]}: what a segment does to the state; in N's place
                                // of a sequence's last segment, the state that the sequence starts from
    int4 *units;                // packed: [n_units] segments (kda_delta_prep.cuh writes them)
};

// State entry of sequence n, or -1 for none.
__device__ __forceinline__ int32_t state_entry(const DeltaParams &p, int32_t n) {
    if (p.slots == nullptr) return n;
    const int32_t s = __ldg(p.slots + n);
    return s >= 0 && s < p.num_slots ? s : -1;
}

// Rows [a, b) of sequence n on the flattened token axis; malformed cu_seqlens are
// clamped to [0, T].
__device__ __forceinline__ void sequence_rows(const DeltaParams &p, int32_t n, int64_t &a, int64_t &b) {
    if (p.cu == nullptr) {
        a = int64_t(n) * p.T;
        b = a + p.T;
        return;
    }
    a = __ldg(p.cu + n);
    b = __ldg(p.cu + n + 1);
    if (a < 0) a = 0;
    if (b > p.T) b = p.T;
    if (b < a) b = a;
}

__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ float widen1(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen1(__half v) { return __half2float(v); }

constexpr int REC_THREADS = 256;

// CQ column quads to a block: 8 (32 columns) or 16 (64 columns).
template <typename T, int CQ>
__global__ void __launch_bounds__(REC_THREADS, 4) kda_delta_rec_kernel(const DeltaParams p) {
    constexpr int VC = 4 * CQ, RG = REC_THREADS / CQ, RPT = 128 / RG;
    __shared__ float sk[128], sq[128], sd[128];
    __shared__ __align__(16) float pk[RG][VC], pq[RG][VC];
    __shared__ __align__(16) float su[VC];
    __shared__ float sqk[4];
    const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
    const int splits = p.V / VC;
    const int vs = int(blockIdx.x) % splits;
    const int nh = int(blockIdx.x) / splits, n = nh / p.H, h = nh - n * p.H;
    const int hk = h / (p.H / p.Hk);
    const int v0 = vs * VC;
    pdl_launch_dependents();
    pdl_wait();
    int64_t a, b;
    sequence_rows(p, n, a, b);
    const int32_t e = state_entry(p, n);
    const int64_t sbase = (int64_t(e < 0 ? 0 : e) * p.H + h) * p.K * p.V + v0 + 4 * cq;
    float4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        S[i] = p.state_in != nullptr && e >= 0 && r < p.K
                   ? __ldcs(reinterpret_cast<const float4 *>(p.state_in + sbase + int64_t(r) * p.V))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    const T *beta = static_cast<const T *>(p.beta);
    // channel tid's q, k, decay of the token that comes next; column tid's v
    float nq = 0.f, nk = 0.f, nd = 0.f, nv = 0.f, nb = 0.f;
    auto fetch = [&](int64_t t) {
        if (tid < p.K) {
            nq = widen1(q[(t * p.Hk + hk) * p.K + tid]);
            nk = widen1(k[(t * p.Hk + hk) * p.K + tid]);
            nd = p.g[p.gate == 0 ? (t * p.H + h) * p.K + tid : t * p.H + h];
        }
        if (tid < VC) {
            nv = widen1(v[(t * p.H + h) * p.V + v0 + tid]);
            nb = widen1(beta[t * p.H + h]);
        }
    };
    if (a < b) fetch(a);
    for (int64_t t = a; t < b; ++t) {
        if (tid < 128) {
            const bool in = tid < p.K;
            sk[tid] = in ? nk : 0.f;
            sq[tid] = in ? nq : 0.f;
            sd[tid] = in ? expf(nd) : 0.f;
            float x = in ? nk * nq : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if ((tid & 31) == 0) sqk[tid >> 5] = x;
        }
        const float vt = nv, bt = nb;
        __syncthreads();
        if (t + 1 < b) fetch(t + 1);
        float4 ak = make_float4(0.f, 0.f, 0.f, 0.f), aq = ak;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg + RG * i;
            const float d = sd[r], kr = sk[r], qr = sq[r];
            S[i].x *= d; S[i].y *= d; S[i].z *= d; S[i].w *= d;
            ak.x = fmaf(kr, S[i].x, ak.x); ak.y = fmaf(kr, S[i].y, ak.y);
            ak.z = fmaf(kr, S[i].z, ak.z); ak.w = fmaf(kr, S[i].w, ak.w);
            aq.x = fmaf(qr, S[i].x, aq.x); aq.y = fmaf(qr, S[i].y, aq.y);
            aq.z = fmaf(qr, S[i].z, aq.z); aq.w = fmaf(qr, S[i].w, aq.w);
        }
        *reinterpret_cast<float4 *>(&pk[rg][4 * cq]) = ak;
        *reinterpret_cast<float4 *>(&pq[rg][4 * cq]) = aq;
        __syncthreads();
        if (tid < VC) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int i = 0; i < RG; ++i) {
                x += pk[i][tid];
                y += pq[i][tid];
            }
            const float u = bt * (vt - x);
            const float qk = (sqk[0] + sqk[1]) + (sqk[2] + sqk[3]);
            su[tid] = u;
            put1(static_cast<T *>(p.o) + (t * p.H + h) * p.V + v0 + tid, p.scale * fmaf(qk, u, y));
        }
        __syncthreads();
        const float4 u = *reinterpret_cast<const float4 *>(&su[4 * cq]);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kr = sk[rg + RG * i];
            S[i].x = fmaf(kr, u.x, S[i].x); S[i].y = fmaf(kr, u.y, S[i].y);
            S[i].z = fmaf(kr, u.z, S[i].z); S[i].w = fmaf(kr, u.w, S[i].w);
        }
        if (t + 1 < b) __syncthreads();        // sk, sqk, su are rewritten for the next token
    }
    if (p.state_out != nullptr && e >= 0) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg + RG * i;
            if (r < p.K) __stcs(reinterpret_cast<float4 *>(p.state_out + sbase + int64_t(r) * p.V), S[i]);
        }
    }
}

}  // namespace kda
