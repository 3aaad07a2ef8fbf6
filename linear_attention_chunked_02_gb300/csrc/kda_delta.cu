// kda_delta.cu -- C ABI of the gated delta rule: argument checks and dispatch of
// kda_delta_prefill and kda_delta_step.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>

#include "kda_delta_rec.cuh"
#include "kda_delta_scan.cuh"
#include "kda_delta_launch.h"
#include "kda_internal.h"
#include "kda_launch.cuh"
#include "kda_layer.h"

namespace {

using namespace kda;

// Whether prompts of this shape go chunk by chunk rather than token by token: from an average length
// of 16 on.  Measured for 32 heads of K = V = 128 in BF16, us token by token and by chunks:
//   1 sequence of 16 / 24 / 32 tokens:     20 / 31 / 41     25 / 25 / 25
//   32 sequences of 8 / 16 / 24 tokens:    57 / 115 / 176   106 / 107 / 107
//   128 sequences of 8 / 16 / 24 tokens:   240 / 439 / 637  335 / 336 / 338
// The lengths themselves are on the device, so the average decides for all sequences, and the rule is only as good
// as they are alike: 255 sequences of one token beside one of 2048 go token by token, 3900 us, where the
// prompt alone takes 172 and a decoding step of the others 171; 63 beside one of 900, 1680 us against 108 and 50.
bool chunked_form(int64_t B, int64_t T, int32_t num_seqs) {
    const int64_t seqs = num_seqs > 0 ? num_seqs : B;
    return B > 0 && T > 0 && B * T >= 16 * seqs;
}

// Chunks to a segment for this shape, 0 where sequences are not split, and a bound on the segments.
// The model: a chunk of the walk takes 4.7 us, 2.9 without outputs; the first run has two walks to a
// segment but the first's one and the last's none; the join takes 6 us a segment and the two more
// launches 10.  Sized for the 152 SMs of a GB300, and for sequences of like lengths.  K = V = 128 in BF16, us
// for the whole operator with sequences whole, in 3, 4, 6 and 9 segments, and in as many as the model takes, when it
// was fitted (now 919, 1805, 165 and 745 in the last column, a chunk of the walk 4.9 us, 3.1 without outputs):
//   1 x 16384 tokens, 32 heads:  1192   855  916  889  913    861 (8)
//   1 x 65536, 16 heads:         4302  2853 2251 1659 1650   1650 (9)
//   1 x 2048, 32 heads:           176   155  171  193  201    155 (3)
//   1 x 8192, 64 heads:           707   872  841  866  959    699 (2)
int32_t segment_chunks(int64_t B, int64_t T, int32_t H, int32_t num_seqs, int64_t &units) {
    const int64_t seqs = num_seqs > 0 ? num_seqs : B, heads = seqs * H, sms = 152;
    const int64_t total = max_chunks(B, T, num_seqs, BT);
    const double c = double(total) / double(seqs);
    auto waves = [&](int64_t n) { return double((n + sms - 1) / sms); };
    double best = waves(heads) * c * 4.7;
    int32_t seg = 0;
    for (int P = 2; P <= 32 && heads < sms; ++P) {
        const int32_t s = int32_t(c / P + 0.999);
        if (s < 4) break;
        const double t = waves((2 * P - 3) * heads) * s * 2.9 + waves(P * heads) * s * 4.7 + 6.0 * P + 10.0;
        if (t < 0.95 * best) {
            best = t;
            seg = s;
        }
    }
    units = seg == 0 ? seqs : num_seqs > 0 ? total / seg + seqs : B * ((((T + BT - 1) / BT) + seg - 1) / seg);
    return seg;
}

size_t image_bytes(int64_t B, int64_t T, int32_t H, int32_t num_seqs) {
    return size_t(max_chunks(B, T, num_seqs, BT)) * size_t(H) * IMG_BYTES;
}

// The workspace of a call whose sequences are cut into segments of `seg` chunks (0: whole), `units` in all.
size_t workspace_bytes_for(int64_t B, int64_t T, int32_t H, int32_t num_seqs, int32_t K, int32_t V, int32_t seg,
                           int64_t units) {
    return image_bytes(B, T, H, num_seqs) + (num_seqs > 0 ? size_t(units) * sizeof(int4) : 0) +
           (seg > 0 ? size_t(units) * size_t(H) * size_t(K) * size_t(K + V) * sizeof(float) : 0);
}

bool width_ok(int32_t w) { return w == 32 || w == 64 || w == 96 || w == 128; }

template <typename T>
cudaError_t launch_rec(const DeltaParams &p, int sms, cudaStream_t s) {
    // 64 columns of a head to a block, or 32 where there are few heads.  A step of BF16, K = V = 128, in us, by
    // 64 and by 32: 3.2 and 3.3 at 32 heads, 6.6 and 5.5 at 128, 8.4 and 9.3 at 256, 14.6 and 16.0 at 512,
    // 44 and 53 at 2048, 313 and 426 at 16384
    const int64_t heads = int64_t(p.nseq) * p.H;
    if (p.V % 64 == 0 && heads >= sms)
        return launch_pdl(true, kda_delta_rec_kernel<T, 16>, unsigned(heads * (p.V / 64)), REC_THREADS, 0, s, p);
    return launch_pdl(true, kda_delta_rec_kernel<T, 8>, unsigned(heads * (p.V / 32)), REC_THREADS, 0, s, p);
}

kda_status_t run_rec(const DeltaParams &p, int32_t dtype, cudaStream_t s) {
    int device = 0;
    DeviceInfo info;
    if (cudaGetDevice(&device) != cudaSuccess || device_info(device, info) != cudaSuccess) return KDA_ERR_CUDA;
    cudaError_t e;
    switch (dtype) {
        case KDA_F32: e = launch_rec<float>(p, info.num_sms, s); break;
        case KDA_BF16: e = launch_rec<__nv_bfloat16>(p, info.num_sms, s); break;
        default: e = launch_rec<__half>(p, info.num_sms, s); break;
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// [rows, heads, width] as {width, heads, rows} with boxes of box x 1 x 64; swizzled: over the
// box's row of 64 or 128 bytes.
bool encode_rows(CUtensorMap *map, const void *base, int32_t dt, int64_t rows, int32_t heads, int32_t width, int box,
                 bool swizzle = false) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const CUtensorMapDataType ty = dt == KDA_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dt == KDA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t es = cuuint64_t(elt_size(dt));
    const cuuint64_t dims[3] = {cuuint64_t(width), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(width) * es, cuuint64_t(heads) * cuuint64_t(width) * es};
    const cuuint32_t boxes[3] = {cuuint32_t(box), 1, 64}, estr[3] = {1, 1, 1};
    return fn(map, ty, 3, const_cast<void *>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              !swizzle             ? CU_TENSOR_MAP_SWIZZLE_NONE
              : box * es == 64     ? CU_TENSOR_MAP_SWIZZLE_64B
                                   : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of both kernels; g has none where a head has one decay.
bool encode_delta(const DeltaParams &p, int32_t dt, int64_t rows, DeltaMaps &prep, DeltaMaps &scan) {
    std::memset(&prep, 0, sizeof(prep));
    std::memset(&scan, 0, sizeof(scan));
    const int box = p.K <= 64 ? 64 : 128;                  // the scan's rows, whatever K
    return encode_rows(&prep.q, p.q, dt, rows, p.Hk, p.K, 32, true) && encode_rows(&prep.k, p.k, dt, rows, p.Hk, p.K, 32, true) &&
           encode_rows(&scan.v, p.v, dt, rows, p.H, p.V, 128) && encode_rows(&scan.q, p.q, dt, rows, p.Hk, p.K, box) &&
           encode_rows(&scan.k, p.k, dt, rows, p.Hk, p.K, box) &&
           (p.gate != KDA_GATE_CHANNEL || (encode_rows(&prep.g, p.g, KDA_F32, rows, p.H, p.K, 32, true) &&
                                           encode_rows(&scan.g, p.g, KDA_F32, rows, p.H, p.K, box)));
}

kda_status_t run_chunked(DeltaParams p, int32_t dtype, int64_t rows, cudaStream_t s) {
    int device = 0;
    DeviceInfo info;
    if (cudaGetDevice(&device) != cudaSuccess || device_info(device, info) != cudaSuccess) return KDA_ERR_CUDA;
    p.err = info.err;
    DeltaMaps prep, scan;
    if (!encode_delta(p, dtype, rows, prep, scan)) return KDA_ERR_CUDA;
    cudaError_t e;
    switch (dtype) {
        case KDA_F32: e = launch_chunked_f32(p, prep, scan, device, info.num_sms, s); break;
        case KDA_BF16: e = launch_chunked_bf16(p, prep, scan, device, info.num_sms, s); break;
        default: e = launch_chunked_f16(p, prep, scan, device, info.num_sms, s); break;
    }
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Heads, widths, types and the gate form.
kda_status_t check_heads(int32_t Hk, int32_t H, int32_t K, int32_t V, int32_t dtype, int32_t gate) {
    if (!dtype_ok(dtype) || !width_ok(K) || !width_ok(V)) return KDA_ERR_UNSUPPORTED;
    if (Hk < 1 || H < 1 || H % Hk != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (gate != KDA_GATE_CHANNEL && gate != KDA_GATE_HEAD) return KDA_ERR_INVALID_ARGUMENT;
    if (int64_t(H) * 128 >= (int64_t(1) << 24)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Pointers of the token tensors: present and aligned.
kda_status_t check_tokens(const void *q, const void *k, const void *v, const float *g, const void *beta,
                          const void *o, int32_t dtype) {
    const size_t es = size_t(elt_size(dtype));
    if (q == nullptr || k == nullptr || v == nullptr || g == nullptr || beta == nullptr || o == nullptr)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(o) ||
        reinterpret_cast<uintptr_t>(beta) % es != 0)
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

// A buffer of a call; no pointer or no bytes: not used.
struct Span {
    const void *at;
    size_t bytes;
};
bool meet(const Span &a, const Span &b) {
    return a.at != nullptr && b.at != nullptr && a.bytes > 0 && b.bytes > 0 && overlaps(a.at, a.bytes, b.at, b.bytes);
}

// Whether something that a call writes (o, states, workspace) lies on something else of its buffers; the
// states may be updated in place.
bool buffers_meet(const DeltaParams &p, size_t rows, int32_t dtype, size_t entries, size_t workspace_bytes) {
    const size_t es = size_t(elt_size(dtype)), H = size_t(p.H);
    const size_t qb = rows * size_t(p.Hk) * size_t(p.K) * es, vb = rows * H * size_t(p.V) * es;
    const size_t gb = rows * H * (p.gate == KDA_GATE_CHANNEL ? size_t(p.K) : 1) * 4;
    const size_t sb = entries * H * size_t(p.K) * size_t(p.V) * 4, nseq = size_t(p.nseq);
    const Span in[] = {{p.q, qb}, {p.k, qb}, {p.v, vb}, {p.g, gb}, {p.beta, rows * H * es},
                       {p.slots, nseq * 4}, {p.cu, (nseq + 1) * 4}};
    const Span state_in{p.state_in, sb}, o{p.o, vb}, state_out{p.state_out, sb}, ws{p.ws, workspace_bytes};
    for (const Span &x : in)
        if (meet(o, x) || meet(state_out, x) || meet(ws, x)) return true;
    return meet(o, state_in) || meet(o, state_out) || meet(o, ws) || meet(ws, state_in) || meet(ws, state_out) ||
           (p.state_in != p.state_out && meet(state_in, state_out));
}

}  // namespace

extern "C" {

size_t kda_delta_prefill_workspace_size(int64_t B, int64_t T, int32_t H, int32_t num_seqs, int32_t K, int32_t V) {
    if (H < 1 || num_seqs < 0 || !width_ok(K) || !width_ok(V)) return 0;
    if (num_seqs > 0 && B != 1) return 0;
    if (!chunked_form(B, T, num_seqs)) return 0;
    int64_t units = 0;
    const int32_t seg = segment_chunks(B, T, H, num_seqs, units);
    return workspace_bytes_for(B, T, H, num_seqs, K, V, seg, units);
}

kda_status_t kda_delta_prefill(const void *q, const void *k, const void *v, const float *g, const void *beta, void *o,
                               const float *state_in, float *state_out, const int32_t *slots, int32_t num_slots,
                               const int32_t *cu_seqlens, int32_t num_seqs, int64_t B, int64_t T, int32_t Hk,
                               int32_t H, int32_t K, int32_t V, int32_t dtype, int32_t gate, float scale,
                               void *workspace, size_t workspace_bytes, void *stream) {
    kda_status_t st = check_heads(Hk, H, K, V, dtype, gate);
    if (st != KDA_OK) return st;
    if (B < 0 || T < 0 || num_seqs < 0) return KDA_ERR_INVALID_ARGUMENT;
    if ((cu_seqlens != nullptr) != (num_seqs > 0)) return KDA_ERR_INVALID_ARGUMENT;
    if (cu_seqlens != nullptr && B != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (slots != nullptr && num_slots < 0) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t seqs = cu_seqlens != nullptr ? num_seqs : B;
    const int64_t max_rows = (int64_t(1) << 31) - 1 - 2 * BT;
    if (T > 0 && B > max_rows / T) return KDA_ERR_UNSUPPORTED;
    if (max_chunks(B, T, num_seqs, BT) * H >= (int64_t(1) << 30) || seqs * H >= (int64_t(1) << 28))
        return KDA_ERR_UNSUPPORTED;
    if (seqs == 0) return KDA_OK;
    const size_t rows = size_t(B) * size_t(T);
    if (rows > 0) {
        st = check_tokens(q, k, v, g, beta, o, dtype);
        if (st != KDA_OK) return st;
    }
    if (!aligned16(state_in) || !aligned16(state_out)) return KDA_ERR_INVALID_ARGUMENT;
    int32_t seg = 0;
    int64_t units = 0;
    size_t need = 0;
    if (chunked_form(B, T, num_seqs)) {
        seg = segment_chunks(B, T, H, num_seqs, units);
        need = workspace_bytes_for(B, T, H, num_seqs, K, V, seg, units);
        if (workspace_bytes < need && seg > 0) {           // no room for the maps: sequences whole
            seg = 0;
            units = seqs;
            need = workspace_bytes_for(B, T, H, num_seqs, K, V, seg, units);
        }
        if (workspace == nullptr || workspace_bytes < need) return KDA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return KDA_ERR_INVALID_ARGUMENT;
    }
    DeltaParams p{q, k, v, g, beta, o, state_in, state_out, slots, num_slots, cu_seqlens, int32_t(seqs), T,
                  Hk, H, K, V, gate, scale, nullptr, 0, 0, nullptr, 0, 0, nullptr, nullptr};
    p.ws = need > 0 ? static_cast<unsigned char *>(workspace) : nullptr;
    if (buffers_meet(p, rows, dtype, size_t(slots != nullptr ? num_slots : seqs), need)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows == 0 && state_out == nullptr) return KDA_OK;
    if (!chunked_form(B, T, num_seqs)) return run_rec(p, dtype, static_cast<cudaStream_t>(stream));
    p.cpr = int32_t((T + BT - 1) / BT);
    p.n_tasks = int32_t(max_chunks(B, T, num_seqs, BT) * H);
    p.seg = seg;
    p.n_units = int32_t(units);
    unsigned char *after = p.ws + image_bytes(B, T, H, num_seqs);
    if (num_seqs > 0) {
        p.units = reinterpret_cast<int4 *>(after);
        after += size_t(units) * sizeof(int4);
    }
    p.trans = reinterpret_cast<float *>(after);
    return run_chunked(p, dtype, int64_t(rows), static_cast<cudaStream_t>(stream));
}

kda_status_t kda_delta_step(const void *q, const void *k, const void *v, const float *g, const void *beta, void *o,
                            float *state, const int32_t *slots, int32_t num_slots, int32_t N, int32_t Hk, int32_t H,
                            int32_t K, int32_t V, int32_t dtype, int32_t gate, float scale, void *stream) {
    kda_status_t st = check_heads(Hk, H, K, V, dtype, gate);
    if (st != KDA_OK) return st;
    if (N < 0 || num_slots < 0 || (slots == nullptr && num_slots < N)) return KDA_ERR_INVALID_ARGUMENT;
    if (int64_t(N) * H >= (int64_t(1) << 28)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    st = check_tokens(q, k, v, g, beta, o, dtype);
    if (st != KDA_OK) return st;
    if (state == nullptr || !aligned16(state)) return KDA_ERR_INVALID_ARGUMENT;
    const DeltaParams p{q, k, v, g, beta, o, state, state, slots, num_slots, nullptr, N, 1, Hk, H, K, V, gate, scale,
                        nullptr, 0, 0, nullptr, 0, 0, nullptr, nullptr};
    if (buffers_meet(p, size_t(N), dtype, size_t(num_slots), 0)) return KDA_ERR_INVALID_ARGUMENT;
    return run_rec(p, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
