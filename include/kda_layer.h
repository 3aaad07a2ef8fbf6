/*
 * kda_layer.h -- C ABI of the operators around the chunk solve: the gated delta
 * rule over prompts and for single tokens, and the norms of the layer that holds
 * it.  Part of the same library as kda_solve_tril.h, whose rules on ownership,
 * streams, stream capture and errors hold here too.
 *
 * The gated delta rule.  Every head keeps a state S [K, V] in FP32.  For each
 * token of a sequence, with its query q, key k (K values each), value v (V
 * values), log decays g and beta:
 *
 *     S <- diag(exp(g)) S
 *     u  = beta (v - S^T k)
 *     S <- S + k u^T
 *     o  = scale S^T q
 *
 * g is the token's own log decay (not a cumulative one), one for each channel
 * (KDA_GATE_CHANNEL) or one for a whole head (KDA_GATE_HEAD), and not positive.
 *
 * Tensors are contiguous and row-major:
 *   q, k    [.., Hk, K] of dtype; head h of the H heads uses key head h / (H / Hk)
 *   v, o    [.., H, V] of dtype
 *   g       [.., H, K] (channel) or [.., H] (head), float32
 *   beta    [.., H] of dtype
 *   states  [entries, H, K, V], float32
 * with K and V each 32, 64, 96 or 128.
 */
#ifndef KDA_LAYER_H
#define KDA_LAYER_H

#include "kda_solve_tril.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_GATE_CHANNEL = 0,         /* g [.., H, K] */
    KDA_GATE_HEAD = 1             /* g [.., H] */
} kda_gate_t;

typedef enum {
    KDA_ACT_SIGMOID = 0,
    KDA_ACT_SILU = 1
} kda_act_t;

/* Largest row width of kda_add_norm and kda_gated_norm. */
#define KDA_NORM_MAX_DIM 16384

/*
 * Workspace bytes kda_delta_prefill needs for this shape: 0 for an empty or
 * invalid one, and for sequences of fewer than 16 tokens on average, which run
 * token by token; else 32,896 for each chunk of 64 tokens and head (packed: for
 * the bound (T + 63 num_seqs) / 64 on the chunks, at most T); packed, 16 for each
 * sequence; and where sequences are split (few heads, many chunks) K (K + V) 4 for
 * each segment and head, the 16 bytes then for each segment.  It depends on nothing
 * but the arguments.  It can be less for a larger T, which may take fewer segments;
 * what it gives for a T is enough for every smaller one all the same.  Pure host
 * arithmetic.
 */
KDA_API size_t kda_delta_prefill_workspace_size(int64_t B, int64_t T, int32_t H, int32_t num_seqs, int32_t K,
                                                int32_t V);

/*
 * The gated delta rule over whole sequences.
 *
 *   q, k, v, g, beta, o   as above with leading dimensions [B, T] (dense: every
 *               batch row is a sequence) or [1, T] with cu_seqlens (packed).
 *               16-byte aligned (beta: to its element size).
 *   cu_seqlens, num_seqs, B, T   as for kda_solve_tril.  Sequences may be empty.
 *   state_in    states to start from, or NULL: all zero.
 *   state_out   states after the last token, or NULL: not wanted.  May be
 *               state_in itself.
 *   slots       device int32 [sequences], or NULL.  Sequence n uses entry
 *               slots[n] of state_in and state_out, which then have num_slots
 *               entries; a slot outside [0, num_slots) means that the sequence
 *               starts from zero and its state is not stored.  Two sequences must
 *               not share a slot.  NULL: sequence n uses entry n (num_slots is
 *               ignored).
 *   Hk, H       key heads and heads; H is a multiple of Hk.  H < 2^17 whatever K
 *               and V, B*T <= 2^31 - 129, sequences * H < 2^28 and chunks * H < 2^30
 *               with chunks of 64 tokens (bounded as for the workspace); larger
 *               sizes give KDA_ERR_UNSUPPORTED.
 *   gate        kda_gate_t.
 *   scale       factor on the output, usually K^-0.5.
 *   workspace   device, 16-byte aligned, kda_delta_prefill_workspace_size()
 *               bytes; its contents are scratch.  One that has no room for the
 *               segments but for the rest leaves sequences whole (as accurate, and
 *               slower); less, or none, gives KDA_ERR_WORKSPACE.
 *
 * o, state_out and the workspace must not overlap each other or anything that is
 * read (KDA_ERR_INVALID_ARGUMENT), but for state_out, which may be state_in.
 *
 * Sequences of no tokens copy their state (zeros without state_in).  With T == 0
 * or B == 0 there is nothing to read but the states.  Rows of T past the last
 * sequence of cu_seqlens are not written.
 *
 * Accuracy.  Products keep FP32's 22 to 24 bits of their operands, the states and
 * all sums are FP32, whatever the type: outputs and states are within about 1e-6 of
 * the 64-bit result's norm, before a 16-bit output's one rounding.  Any decay is
 * allowed: channels that fall by more than e^-48 over half a chunk of 64 tokens, and
 * chunks that clear the state, take slower ways of the same accuracy (16 x 512
 * tokens x 64 heads whose channels all lose two nats a token: 20.5 ms, at up to 1.5
 * nats 0.48).  Errors are relative to the largest state and value that go into a
 * chunk, column by column: where values fall by more than some 10^4 inside a chunk
 * that also clears what was before, the small ones keep fewer digits.  The result
 * does not depend on the values in other heads and sequences, nor on what the
 * workspace held; repeated calls give the same bits.  A NaN or an infinity can reach
 * the tokens before it in its chunk as well as all after it (one in v: in its column
 * alone).
 *
 * The call launches one to four kernels and allocates nothing; it may be captured
 * into a graph after one call of the same type and widths on the device, which sets
 * the kernels' shared memory sizes.
 */
KDA_API kda_status_t kda_delta_prefill(const void *q, const void *k, const void *v, const float *g, const void *beta,
                                       void *o, const float *state_in, float *state_out, const int32_t *slots,
                                       int32_t num_slots, const int32_t *cu_seqlens, int32_t num_seqs, int64_t B,
                                       int64_t T, int32_t Hk, int32_t H, int32_t K, int32_t V, int32_t dtype,
                                       int32_t gate, float scale, void *workspace, size_t workspace_bytes,
                                       void *stream);

/*
 * One token of each of N running requests; the states are updated in place.
 *
 *   q, k, v, g, beta, o   as above with the leading dimension [N].
 *   state       [num_slots, H, K, V].
 *   slots       device int32 [N], or NULL: request n uses entry n, and num_slots
 *               is at least N.  A slot outside [0, num_slots) (-1 for the padding
 *               rows of a captured batch) reads a state of zeros and stores
 *               nothing.  Two requests must not share a slot.
 *               o and state must not overlap each other or another tensor.
 *   N           N == 0 is a no-op.  N * H < 2^28 and H < 2^17, else
 *               KDA_ERR_UNSUPPORTED.
 */
KDA_API kda_status_t kda_delta_step(const void *q, const void *k, const void *v, const float *g, const void *beta,
                                    void *o, float *state, const int32_t *slots, int32_t num_slots, int32_t N,
                                    int32_t Hk, int32_t H, int32_t K, int32_t V, int32_t dtype, int32_t gate,
                                    float scale, void *stream);

/*
 * The norm before a block, with the residual sum that precedes it:
 *
 *     r = residual + alpha x;   residual_out = r;   y = r / sqrt(mean(r^2) + eps) * weight
 *
 *   x, residual, residual_out, y   [rows, dim] of dtype; weight [dim] of dtype.
 *               residual may be NULL (r = alpha x); residual_out may be NULL (not
 *               wanted) or residual itself.  y may be x.  No other overlap.
 *               Aligned to the element size.
 *   dim         1 .. KDA_NORM_MAX_DIM, else KDA_ERR_UNSUPPORTED.
 *   rows        rows == 0 is a no-op.
 * r and the norm are FP32; y comes from r before it is rounded to residual_out.
 */
KDA_API kda_status_t kda_add_norm(const void *x, const void *residual, const void *weight, void *y,
                                  void *residual_out, int64_t rows, int32_t dim, float alpha, float eps,
                                  int32_t dtype, void *stream);

/*
 * The norm after a block, times its gate:
 *
 *     y = x / sqrt(mean(x^2) + eps) * weight * act(gate)
 *
 *   x, gate, y  [rows, dim] of dtype (one row for each token and head); weight
 *               [dim] of dtype.  y may be x or gate.  Aligned to the element size.
 *   act         kda_act_t: sigmoid(z) or z sigmoid(z).
 *   dim, rows   as for kda_add_norm.
 */
KDA_API kda_status_t kda_gated_norm(const void *x, const void *gate, const void *weight, void *y, int64_t rows,
                                    int32_t dim, float eps, int32_t act, int32_t dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LAYER_H */
