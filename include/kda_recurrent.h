/*
 * kda_recurrent.h -- C ABI of the gated linear recurrence (whole sequences, their
 * gradients, single tokens) and of what its training keeps: 8-bit checkpoints of
 * activations, and the gradients of the gated norm.  Part of the same library as
 * kda_solve_tril.h and kda_layer.h, whose rules on ownership, streams, stream
 * capture and errors hold here too.
 *
 * The recurrence.  Every one of D channels keeps a state h in FP32.  For each
 * token of a sequence, with its input x and its gate value g,
 *
 *     a = exp(g)               (KDA_DECAY_LOG: g is a log decay, not positive)
 *     a = 1 / (1 + exp(-g))    (KDA_DECAY_SIGMOID)
 *     h <- a h + c x,          c = 1, or 1 - a with `complement`
 *     y  = h
 *
 * Sequences, packed or dense, are rows of one stream [rows, D]: row b T + t of the
 * dense layout is token t of batch row b.  Tensors are row-major with contiguous
 * rows; inputs may have a pitch (`ld..`, in elements, at least D) between rows,
 * outputs are contiguous.  Everything is aligned to its element size.  Rows that are whole 16-byte
 * pieces (addresses, pitches and D) take the quicker kernels.
 *
 *   x, y     [rows, D] of dtype
 *   g        [rows, D] of g_dtype: dtype or KDA_F32
 *   states   [entries, D], float32
 *   chunk_states  [ceil(rows / 64), D], float32: entry j is the state before row
 *            64 j of the stream, for a row that begins a sequence the state that the
 *            sequence starts from.
 *
 * Accuracy.  Decays, sums and states are FP32; outputs are rounded to their type once.  Decays are
 * within two units in the last place, and 1 - a too, but for sigmoids of 16-bit arguments and of
 * codes, where 1 - a (and a decay below 1/2) is within |g| 2^-24 + 2^-21 of itself, 0 below 2^-126, and a at least 2^-126:
 * the argument's own rounding is 2^-12 |g| at best.  Results do not depend on the
 * values of other sequences and channels, nor on timing: repeated calls give the same bits.  A
 * NaN or an infinity reaches the later tokens of its channel and sequence (in the gradients also
 * the earlier ones), nothing else.
 *
 * Capture.  A call can be captured into a graph after one of the same types, form (decay, complement) and alignment on
 * the device, which sets the kernel's limits.  The blocks of a cluster wait on one another's messages for a second at
 * most; a wait that runs out (it never should) is reported by kda_device_error().
 */
#ifndef KDA_RECURRENT_H
#define KDA_RECURRENT_H

#include "kda_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_DECAY_LOG = 0,
    KDA_DECAY_SIGMOID = 1
} kda_decay_t;

/* Rows to a chunk state. */
#define KDA_RECUR_CHUNK 64
/* Largest D. */
#define KDA_RECUR_MAX_DIM (1 << 20)
/* Elements of a row that share a checkpoint's exponent. */
#define KDA_CHECKPOINT_BLOCK 32

/*
 * The recurrence over whole sequences.
 *
 *   state_in    states to start from, or NULL: zeros.
 *   state_out   states after the last token, or NULL: not wanted.  May be state_in
 *               itself.
 *   slots, num_slots   as for kda_delta_prefill.
 *   chunk_states   written where not NULL, for kda_gated_scan_backward.  Entries whose
 *               row belongs to no sequence are not written.
 *   cu_seqlens, num_seqs, B, T   as for kda_solve_tril; sequences may be empty, their
 *               states are copied.  Rows of T outside [cu_seqlens[0],
 *               cu_seqlens[num_seqs]) are neither read nor written.
 *   D           1 .. KDA_RECUR_MAX_DIM.  B T < 2^31 - 2^16 and num_seqs < 2^30 (dense: B < 2^30),
 *               else KDA_ERR_UNSUPPORTED.
 * y, state_out and chunk_states must not overlap each other or anything that is read
 * (KDA_ERR_INVALID_ARGUMENT), but for state_out, which may be state_in.
 *
 * One launch, no workspace.
 */
KDA_API kda_status_t kda_gated_scan(const void *x, int64_t ldx, const void *g, int64_t ldg, void *y,
                                    const float *state_in, float *state_out, const int32_t *slots, int32_t num_slots,
                                    float *chunk_states, const int32_t *cu_seqlens, int32_t num_seqs, int64_t B,
                                    int64_t T, int32_t D, int32_t dtype, int32_t g_dtype, int32_t decay,
                                    int32_t complement, void *stream);

/*
 * Its gradients.  With dy and dstate_out those of y and of the final states,
 *
 *     d_t = dy_t + a_{t+1} d_{t+1}     (last token: dy + dstate_out)
 *     dx  = c d;   da = d (h_{t-1} - [complement] x);   dg = da a, or da a (1 - a) for the sigmoid
 *     dstate_in = a_0 d_0
 *
 *   dy, dx      [rows, D] of dtype, dy at pitch lddy.
 *   x, g        as given to kda_gated_scan; or, with x_exponents or g_exponents, the
 *               int8 codes of their checkpoints (kda_checkpoint_save of [rows, D]; the
 *               pitch is then D).
 *   chunk_states   as kda_gated_scan left them: h_{t-1} is computed again from them,
 *               and from state_in where a sequence begins.
 *   state_in    [sequences, D], the states that the sequences started from, or NULL:
 *               zeros.
 *   dstate_out  [sequences, D] or NULL: zeros.
 *   dg          [rows, D] of g_dtype.
 *   dstate_in   [sequences, D] or NULL: not wanted.
 *   the rest    as for kda_gated_scan.
 * dx, dg and dstate_in must not overlap each other or anything that is read.
 *
 * One launch, no workspace.
 */
KDA_API kda_status_t kda_gated_scan_backward(const void *dy, int64_t lddy, const void *x, const uint8_t *x_exponents,
                                             int64_t ldx, const void *g, const uint8_t *g_exponents, int64_t ldg,
                                             const float *chunk_states, const float *state_in,
                                             const float *dstate_out, void *dx, void *dg, float *dstate_in,
                                             const int32_t *cu_seqlens, int32_t num_seqs, int64_t B, int64_t T,
                                             int32_t D, int32_t dtype, int32_t g_dtype, int32_t decay,
                                             int32_t complement, void *stream);

/*
 * One token of each of N running requests; the states are updated in place.
 *
 *   x, g, y     as above with N rows.
 *   state       [num_slots, D]; NULL where num_slots is 0.
 *   slots       device int32 [N], or NULL: request n uses entry n, and num_slots is at
 *               least N.  A slot outside [0, num_slots) reads a state of zeros and stores
 *               nothing.  Two requests must not share a slot.
 *   N           N == 0 is a no-op.  N * ceil(D / 256) < 2^30, else KDA_ERR_UNSUPPORTED.
 * y and state must not overlap each other or another tensor.
 */
KDA_API kda_status_t kda_gated_step(const void *x, int64_t ldx, const void *g, int64_t ldg, void *y, float *state,
                                    const int32_t *slots, int32_t num_slots, int32_t N, int32_t D, int32_t dtype,
                                    int32_t g_dtype, int32_t decay, int32_t complement, void *stream);

/*
 * Activations kept in 8 bits for a backward pass.  A row's elements are taken in blocks
 * of 32 (the last one may be short); with e the least integer for which the block's largest magnitude
 * is at most 127 * 2^e, and at least -127,
 *
 *     code = x / 2^e rounded to the nearest integer (ties to even),   x ~ code * 2^e
 *
 * so that the error is at most 2^(e-1): 1 / 127 of the block's largest magnitude, or 2^-128 where e is -127.  (A code whose value
 * would pass the type's largest is rounded towards zero: 63 in place of 64 where x is within
 * 1 / 128 of it.)  The scale is a
 * power of two: codes are exact whatever arithmetic computes them, and the values that they stand
 * for are representable in x's type.  A block with a NaN or an infinity is kept as one that
 * reads back as NaN throughout.
 *
 *   x           [rows, dim] of dtype; for save at pitch ldx.
 *   codes       int8 [rows, dim].
 *   exponents   uint8 [rows, ceil(dim / 32)]: e + 127, or 255 for a block that was not finite.
 *   dim, rows   dim 1 .. KDA_RECUR_MAX_DIM; rows * ceil(dim / 32) < 2^36; rows == 0 is a no-op.
 * No overlaps.  kda_checkpoint_load gives the values in any dtype (rounded once, where it is narrower than the
 * one that was saved).
 */
KDA_API kda_status_t kda_checkpoint_save(const void *x, int64_t ldx, int8_t *codes, uint8_t *exponents, int64_t rows,
                                         int32_t dim, int32_t dtype, void *stream);
KDA_API kda_status_t kda_checkpoint_load(const int8_t *codes, const uint8_t *exponents, void *x, int64_t rows,
                                         int32_t dim, int32_t dtype, void *stream);

/*
 * The gradients of kda_gated_norm.  With n = x / sqrt(mean(x^2) + eps), s = act(gate) and u = dy weight s,
 *
 *     dx = (u - n mean(u n)) / sqrt(mean(x^2) + eps)
 *     dgate = dy n weight act'(gate)
 *     dweight = sum over rows of dy n s
 *
 *   dy, dx, dgate   [rows, dim] of dtype; weight [dim] of dtype; dweight [dim], float32.
 *   x, gate     [rows, dim] of dtype; or, with x_exponents or gate_exponents, the codes of
 *               their checkpoints.
 *   act         kda_act_t.
 *   dim, rows   as for kda_gated_norm.  With rows == 0, dweight is zeroed.
 *   workspace   device, 16-byte aligned, kda_gated_norm_backward_workspace_size() bytes; scratch.  Calls that may run at the
 *               same time, replays of graphs among them, need workspaces of their own.
 * dx, dgate, dweight and the workspace must not overlap each other or anything that is read
 * (KDA_ERR_INVALID_ARGUMENT).
 *
 * Sums are FP32, dweight's in an order that depends on shapes, types and alignment alone.  act and act' of 16-bit gates and of
 * codes have the recurrence's accuracy for such sigmoids, but are 0 for gates below -126 ln 2.  Two launches.
 */
KDA_API size_t kda_gated_norm_backward_workspace_size(int64_t rows, int32_t dim);
KDA_API kda_status_t kda_gated_norm_backward(const void *dy, const void *x, const uint8_t *x_exponents,
                                             const void *gate, const uint8_t *gate_exponents, const void *weight,
                                             void *dx, void *dgate, float *dweight, int64_t rows, int32_t dim,
                                             float eps, int32_t act, int32_t dtype, void *workspace,
                                             size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_RECURRENT_H */
