/*
 * dwconv_seq.h -- C ABI of the sequence operators that stand around a short
 * depthwise convolution in a linear-attention block on MI355X (gfx950):
 *
 *   dwconv_causal_*  causal depthwise 1-D convolution of packed sequences
 *   dwconv_delta_*   the gated delta rule (one matrix of state per head)
 *   dwconv_norm_*    norm after a block, gate, residual scale, residual and
 *                    the norm before the next block, in one pass
 *   dwconv_scan_*    the selective scan of a state space mixer (a few states
 *                    per channel)
 *   dwconv_group_*   norm over groups of channels of an image or a sequence,
 *                    with an activation
 *
 * Shared conventions (status codes, dtypes and errors as in dwconv.h):
 *
 * Tokens of several sequences lie one behind the other.  `offsets` holds
 * seqs + 1 int32 device values: sequence s is tokens offsets[s] ..
 * offsets[s+1]-1; they rise, start at 0 and end at or below `tokens`.  A
 * sequence may be empty.  tokens and seqs are at most 2^31 - 129.  What tokens
 * behind the last sequence hold does not matter, and their outputs are left as
 * they were.  offsets == NULL: one sequence of all tokens (seqs must be 1).  The
 * offsets are device data that the host does not see: the kernels clamp them to
 * [0, tokens], so wrong ones give wrong results but no access out of bounds.
 *
 * Token strides (ld...) count elements between two tokens; within a token the
 * channels (heads x channels) are dense.  A stride is at least the token's
 * channels, so queries, keys and values may be slices of one tensor.  Every
 * alignment that fits the element type is accepted; tensors whose rows are
 * not 16-byte aligned run narrower loads.
 *
 * The caller owns all device memory, workspaces included; nothing here
 * allocates device memory, synchronises or keeps a pointer.  A plan holds
 * host data only, is immutable and may be used from several threads and on
 * several streams.  A workspace serves one call at a time: calls that may run
 * at once (two streams, two captured graphs) need one each.  Its contents on
 * entry do not matter.  Work is enqueued on `stream`, which belongs to the
 * current device, as do all pointers.  Outputs must not overlap inputs unless
 * stated.  Every sum is formed in a fixed order without atomics: the same call
 * gives the same bits.
 *
 * A call whose grid would pass 2^32 lanes returns DWCONV_ERR_UNSUPPORTED before
 * anything is launched:
 *   convolution  2^24 workgroups of 256 lanes, a lane a vector of channels (16
 *                bytes, 8 for K > 4, one element where rows are not aligned) of up
 *                to 64 tokens, in a step of one row; gradients also 2^30 (K + 1) x C
 *   delta rule   2^23 (tokens / 64 + sequences) x key heads, or 2^21 sequences x
 *                value heads x ceil(Dv / 64); bf16 and fp16 also 2^24 sequences x
 *                key heads (rounded up to a multiple of 8) x value heads a key head
 *                x ceil(Dv / 32)
 *   its step     2^24 rows x value heads x ceil(Dv / 128), with Dv / 32 where rows
 *                are not aligned to four elements
 *   norms        2^32 lanes, 16 to 1024 a row
 *   scan         2^24 workgroups of 256 lanes, a workgroup 64 channels of a group (32,
 *                16, 8 for N > 16, 32, 64) of a sequence or of 64 or more tokens of
 *                it, in a step of one row; gradients also 2^24 for every 8 (4, 2, 1)
 *                tokens of a group of channels; the workspace's size is then given as
 *                SIZE_MAX.  Token strides are at most 2^26 elements there (but in a step)
 *   group norm   2^24 workgroups of 256 lanes, 2^23 of 512, 2^22 of 1024, each 8 channels
 *                or more of an image, or 8 KB or more;
 *                2^22 groups of all images where one image is more than a workgroup's
 *                registers hold (in gradients groups + C / 8)
 *
 * float (fp32) everywhere: biases, scales, norm weights, decays, rates, write
 * strengths, states of the rule and the scan and the gradients of all of these.  Sums and
 * statistics are fp32 or wider; a value of type `dtype` is rounded once, to
 * nearest even, when it is stored.
 */
#ifndef DWCONV_SEQ_H
#define DWCONV_SEQ_H

#include <stddef.h>
#include <stdint.h>

#include "dwconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dwconv_causal_plan *dwconv_causal_t;
typedef struct dwconv_delta_plan *dwconv_delta_t;
typedef struct dwconv_norm_plan *dwconv_norm_t;
typedef struct dwconv_scan_plan *dwconv_scan_t;
typedef struct dwconv_group_plan *dwconv_group_t;

/* Activation of the causal convolution's output and of a gate. */
typedef enum {
    DWCONV_SEQ_ACT_NONE = 0,     /* identity                                   */
    DWCONV_SEQ_ACT_SILU = 1,     /* z / (1 + exp(-z))                          */
    DWCONV_SEQ_ACT_SIGMOID = 2   /* 1 / (1 + exp(-z)); gates only              */
} dwconv_seq_act_t;

typedef enum {
    DWCONV_NORM_NONE = 0,        /* identity                                   */
    DWCONV_NORM_RMS = 1,         /* x / sqrt(mean x^2 + eps) * w               */
    DWCONV_NORM_LAYER = 2        /* (x - mean) / sqrt(var + eps) * w + b       */
} dwconv_norm_kind_t;

/* ------------------------------------------------------------------------
 * Causal depthwise convolution.
 *
 *   ext  = [state_in (K-1 rows); x (L rows)]         per sequence
 *   z[t] = bias + sum_{k<K} w[k] * ext[t + k]        w[K-1] meets the token itself
 *   y[t] = act(z[t])
 *   state_out = the last K-1 rows of ext
 *
 *   x, y       tokens x C (dtype), token strides ldx, ldy
 *   w          K x C (dtype), bias C float or NULL
 *   state_*    seqs x (K-1) x C (dtype), dense; NULL state_in: zeros; NULL
 *              state_out: not written; the two must not overlap
 * ------------------------------------------------------------------------ */

/* 2 <= K <= 8, C >= 1, dtype F32 / F16 / BF16, act NONE or SILU; anything
 * else is DWCONV_ERR_INVALID_ARG and *out = NULL. */
dwconv_status_t dwconv_causal_create(dwconv_causal_t *out, int C, int K, dwconv_dtype_t dtype,
                                     dwconv_seq_act_t act);
dwconv_status_t dwconv_causal_destroy(dwconv_causal_t h);

dwconv_status_t dwconv_causal_fwd(dwconv_causal_t h, const void *x, int64_t ldx, const void *w,
                                  const float *bias, const int32_t *offsets, int seqs, int tokens,
                                  const void *state_in, void *state_out, void *y, int64_t ldy,
                                  hipStream_t stream);

/* One token for each of `rows` sequences whose states lie in a cache of
 * n_slots x (K-1) x C: row i reads and shifts cache entry slots[i] (int32
 * device values; NULL: entry i, rows <= n_slots).  A row whose slot is outside
 * [0, n_slots) is skipped: its y is left as it was.  Rows with the same slot
 * are consecutive tokens of that sequence, in row order.  x, y: rows x C. */
dwconv_status_t dwconv_causal_step(dwconv_causal_t h, const void *x, int64_t ldx, const void *w,
                                   const float *bias, void *state, const int32_t *slots, int n_slots,
                                   int rows, void *y, int64_t ldy, hipStream_t stream);

/* Gradients for dy (as y) and dstate_out (as state_out; NULL: zeros): dx (as
 * x), dw K x C float, dbias C float or NULL, dstate_in (as state_in) or NULL.
 * dw and dbias are overwritten. */
dwconv_status_t dwconv_causal_bwd_workspace(dwconv_causal_t h, int tokens, size_t *bytes);
dwconv_status_t dwconv_causal_bwd(dwconv_causal_t h, const void *x, int64_t ldx, const void *w,
                                  const float *bias, const int32_t *offsets, int seqs, int tokens,
                                  const void *state_in, const void *dy, int64_t lddy,
                                  const void *dstate_out, void *dx, int64_t lddx, float *dw,
                                  float *dbias, void *dstate_in, void *workspace,
                                  hipStream_t stream);

/* ------------------------------------------------------------------------
 * Gated delta rule.  Per value head h (its key head is h / (Hv / Hk)):
 *
 *   S_t = e^{g_t} S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t)
 *   o_t = S_t^T q_t
 *
 * with q_t = scale * q / |q| and k_t = k / |k| where normalize is set
 * (|x| = sqrt(sum x^2 + eps)), else q_t = scale * q, k_t = k.
 *
 *   q, k       tokens x Hk x Dk (dtype), token strides ldq, ldk
 *   v, o       tokens x Hv x Dv (dtype), token strides ldv, ldo
 *   g, beta    tokens x Hv float, dense; g is the logarithm of the decay
 *              (-infinity forgets everything)
 *   state_*    seqs x Hv x Dk x Dv float, dense; NULL state_in: zeros; NULL
 *              state_out: not written; state_out may be state_in itself
 *
 * Forward, a NaN or infinity reaches no token before its own, no other sequence,
 * no other head (from q and k: the value heads of their key head) and, from v or a
 * state, no other column of the state; from its own token on the outputs that
 * depend on it are not finite.  In the gradients it may reach any token of its
 * sequence and the heads that share its key head.
 * ------------------------------------------------------------------------ */

/* Hk, Hv >= 1, Hv a multiple of Hk and at most 65536, 1 <= Dk <= 256, 1 <= Dv <=
 * 4096, dtype F32 / F16 / BF16, finite scale, eps >= 0 and finite. */
dwconv_status_t dwconv_delta_create(dwconv_delta_t *out, int Hk, int Hv, int Dk, int Dv,
                                    dwconv_dtype_t dtype, float scale, int normalize, float eps);
dwconv_status_t dwconv_delta_destroy(dwconv_delta_t h);

/* Bytes of workspace of dwconv_delta_fwd (backward == 0) or dwconv_delta_bwd
 * (backward != 0) for these sizes; the workspace is 16-byte aligned.  The
 * backward pass keeps two matrices of state for each 64 tokens. */
dwconv_status_t dwconv_delta_workspace(dwconv_delta_t h, int seqs, int tokens, int backward,
                                       size_t *bytes);

dwconv_status_t dwconv_delta_fwd(dwconv_delta_t h, const void *q, int64_t ldq, const void *k,
                                 int64_t ldk, const void *v, int64_t ldv, const float *g,
                                 const float *beta, const int32_t *offsets, int seqs, int tokens,
                                 const float *state_in, float *state_out, void *o, int64_t ldo,
                                 void *workspace, hipStream_t stream);

/* One token for each of `rows` sequences, states in a cache of n_slots x Hv x
 * Dk x Dv floats updated in place; slots as for dwconv_causal_step. */
dwconv_status_t dwconv_delta_step(dwconv_delta_t h, const void *q, int64_t ldq, const void *k,
                                  int64_t ldk, const void *v, int64_t ldv, const float *g,
                                  const float *beta, float *state, const int32_t *slots, int n_slots,
                                  int rows, void *o, int64_t ldo, hipStream_t stream);

/* Gradients for d_o (as o) and dstate_out (as state_out; NULL: zeros) of the
 * forward pass from the same inputs (its intermediates are computed again):
 * dq, dk, dv (as q, k, v, token strides lddq, lddk, lddv; a shared key head's
 * gradient is the sum over its value heads), dg and dbeta (as g, beta) and
 * dstate_in (as state_in; it may be dstate_out itself) or NULL. */
dwconv_status_t dwconv_delta_bwd(dwconv_delta_t h, const void *q, int64_t ldq, const void *k,
                                 int64_t ldk, const void *v, int64_t ldv, const float *g,
                                 const float *beta, const int32_t *offsets, int seqs, int tokens,
                                 const float *state_in, const void *d_o, int64_t lddo,
                                 const float *dstate_out, void *dq, int64_t lddq, void *dk,
                                 int64_t lddk, void *dv, int64_t lddv, float *dg, float *dbeta,
                                 float *dstate_in, void *workspace, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Norms around a block.  For each of `rows` rows of D channels:
 *
 *   t = N_after(o) * act(gate)          the block's output, normed and gated
 *   h = residual + scale * t            the new residual stream
 *   y = N_before(h)                     what the next block reads
 *
 *   o, residual, h, y   rows x D (dtype), dense; residual may be NULL
 *   gate                ceil(rows / rows_per_gate) x D (dtype), dense, or NULL:
 *                       row i takes gate row i / rows_per_gate (1: one a row;
 *                       H*W: one an image)
 *   scale               D float or NULL (ones)
 *   w_after, w_before   D float, needed where the norm is not NONE, else
 *                       ignored; b_after, b_before D float or NULL, LAYER only
 *                       (ignored otherwise)
 *   h                   may be NULL if y is given; may be residual or o itself
 *   y                   needed where N_before is not NONE, else ignored; may be
 *                       o itself (if h is not)
 * y is formed from the unrounded h.
 * ------------------------------------------------------------------------ */

/* 1 <= D <= 16384, dtype F32 / F16 / BF16, eps >= 0 and finite. */
dwconv_status_t dwconv_norm_create(dwconv_norm_t *out, int D, dwconv_dtype_t dtype,
                                   dwconv_norm_kind_t after, dwconv_norm_kind_t before,
                                   dwconv_seq_act_t gate_act, float eps);
dwconv_status_t dwconv_norm_destroy(dwconv_norm_t h);

dwconv_status_t dwconv_norm_fwd(dwconv_norm_t p, int rows, const void *o, const void *residual,
                                const void *gate, int rows_per_gate, const float *scale,
                                const float *w_after, const float *b_after, const float *w_before,
                                const float *b_before, void *h, void *y, hipStream_t stream);

/* Gradients for dh and dy (as h and y; dh may be NULL for zeros, dy is needed
 * where N_before is not NONE and ignored otherwise) from the forward pass's
 * inputs: d_o, dresidual, dgate (as o, residual, gate), dscale, dw_after,
 * db_after, dw_before, db_before (D float).  Any of them may be NULL: not
 * wanted; those of absent inputs are ignored. */
dwconv_status_t dwconv_norm_bwd_workspace(dwconv_norm_t p, int rows, int rows_per_gate,
                                          size_t *bytes);
dwconv_status_t dwconv_norm_bwd(dwconv_norm_t p, int rows, const void *o, const void *residual,
                                const void *gate, int rows_per_gate, const float *scale,
                                const float *w_after, const float *b_after, const float *w_before,
                                const float *b_before, const void *dh, const void *dy, void *d_o,
                                void *dresidual, void *dgate, float *dscale, float *dw_after,
                                float *db_after, float *dw_before, float *db_before,
                                void *workspace, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Selective scan.  Per channel c of group g = c / (C / G), with N states:
 *
 *   d_t = softplus(dt_t + dt_bias)          or dt_t + dt_bias without softplus
 *   h_t[n] = e^{d_t a[n]} h_{t-1}[n] + d_t x_t b_t[g, n]
 *   y_t = (sum_n h_t[n] c_t[g, n] + skip x_t) * act(gate_t)
 *
 *   x, dt, y, gate  tokens x C (dtype), token strides ldx, lddt, ldy, ldgate; gate
 *                   may be NULL
 *   a               C x N float: the states' rates, below zero as a rule
 *   b, c            tokens x G x N (dtype), token strides ldb, ldc
 *   skip, dt_bias   C float or NULL (zeros)
 *   state_*         seqs x C x N float, dense; NULL state_in: zeros; NULL
 *                   state_out: not written; state_out may be state_in itself
 *
 * Rates and widths may have any sign: states then grow.  A token's own e^{d a} is an fp32
 * number, though, infinite from d a = 88.8 on, where it makes NaN of a state of zero; that
 * of many tokens together has no such end.
 *
 * Work is laid out by the average length, which is all that the host knows: a sequence
 * many times longer than the others of its call is walked by few CUs where those are as
 * many as fill the card by themselves (C / 64 or more workgroups a sequence, 256 in all).
 * A workgroup has channels of one group: groups of fewer than 64 leave it part empty.
 *
 * Forward, a NaN or infinity reaches no token before its own, no other sequence and,
 * but for those of b and c, no other channel.  In the gradients it may reach any
 * token of its sequence and, through db and dc, the sums over the group's channels.
 * ------------------------------------------------------------------------ */

/* 1 <= C <= 2^24, G >= 1, C a multiple of G, 1 <= N <= 128, dtype F32 / F16 / BF16,
 * gate_act as for a gate above. */
dwconv_status_t dwconv_scan_create(dwconv_scan_t *out, int C, int N, int G, dwconv_dtype_t dtype,
                                   int softplus, dwconv_seq_act_t gate_act);
dwconv_status_t dwconv_scan_destroy(dwconv_scan_t h);

/* Bytes of workspace of dwconv_scan_fwd (backward == 0, 0 for many plans) or
 * dwconv_scan_bwd (backward != 0); the workspace is 16-byte aligned.  The backward
 * pass keeps the states of every 8 tokens. */
dwconv_status_t dwconv_scan_workspace(dwconv_scan_t h, int seqs, int tokens, int backward,
                                      size_t *bytes);

dwconv_status_t dwconv_scan_fwd(dwconv_scan_t h, const void *x, int64_t ldx, const void *dt,
                                int64_t lddt, const float *a, const void *b, int64_t ldb,
                                const void *c, int64_t ldc, const float *skip,
                                const float *dt_bias, const void *gate, int64_t ldgate,
                                const int32_t *offsets, int seqs, int tokens,
                                const float *state_in, float *state_out, void *y, int64_t ldy,
                                void *workspace, hipStream_t stream);

/* One token for each of `rows` sequences, states in a cache of n_slots x C x N
 * floats updated in place; slots as for dwconv_causal_step. */
dwconv_status_t dwconv_scan_step(dwconv_scan_t h, const void *x, int64_t ldx, const void *dt,
                                 int64_t lddt, const float *a, const void *b, int64_t ldb,
                                 const void *c, int64_t ldc, const float *skip,
                                 const float *dt_bias, const void *gate, int64_t ldgate,
                                 float *state, const int32_t *slots, int n_slots, int rows,
                                 void *y, int64_t ldy, hipStream_t stream);

/* Gradients for dy (as y) and dstate_out (as state_out; NULL: zeros) of the forward
 * pass from the same inputs (its intermediates are computed again): dx, ddt, dgate (as
 * x, dt, gate; dgate may be NULL), da (as a), db, dc (as b, c; sums over the
 * channels of the group), dskip, ddt_bias (C float or NULL) and dstate_in (as
 * state_in; it may be dstate_out itself) or NULL. */
dwconv_status_t dwconv_scan_bwd(dwconv_scan_t h, const void *x, int64_t ldx, const void *dt,
                                int64_t lddt, const float *a, const void *b, int64_t ldb,
                                const void *c, int64_t ldc, const float *skip,
                                const float *dt_bias, const void *gate, int64_t ldgate,
                                const int32_t *offsets, int seqs, int tokens,
                                const float *state_in, const void *dy, int64_t lddy,
                                const float *dstate_out, void *dx, int64_t lddx, void *ddt,
                                int64_t ldddt, float *da, void *db, int64_t lddb, void *dc,
                                int64_t lddc, float *dskip, float *ddt_bias, void *dgate,
                                int64_t lddgate, float *dstate_in, void *workspace,
                                hipStream_t stream);

/* ------------------------------------------------------------------------
 * Group norm with an activation.  For each image (or sequence) of `pixels` rows of C
 * channels, and each of its G groups of C / G channels one beside the other:
 *
 *   u = (x - mean) / sqrt(var + eps)        over the group's pixels x C / G values
 *   y = act(u * w + b)
 *
 *   x, y        images x pixels x C (dtype), ldx, ldy elements between two pixels,
 *               images one behind the other; y may be x itself (with ldy == ldx)
 *   w, b        C float or NULL (ones, zeros)
 *
 * Sums over a group are fp32 numbers: a group whose deviations' squares add up to more than
 * 3.4e38 has u = 0 and dx = 0, one whose values do is NaN, and where eps = 0 deviations
 * below 1e-18 lose digits.  A NaN or infinity makes NaN of its image's group, in y and in
 * dx, and of no other one.
 * ------------------------------------------------------------------------ */
typedef enum {
    DWCONV_GROUP_ACT_NONE = 0,   /* identity                                   */
    DWCONV_GROUP_ACT_SILU = 1,   /* z / (1 + exp(-z))                          */
    DWCONV_GROUP_ACT_RELU = 2    /* max(z, 0); slope 0 at 0                    */
} dwconv_group_act_t;

/* C, G >= 1, C a multiple of G and at most 65536, dtype F32 / F16 / BF16, eps >= 0
 * and finite. */
dwconv_status_t dwconv_group_create(dwconv_group_t *out, int C, int G, dwconv_dtype_t dtype,
                                    dwconv_group_act_t act, float eps);
dwconv_status_t dwconv_group_destroy(dwconv_group_t h);

/* Bytes of workspace of dwconv_group_fwd (backward == 0, 0 for small images) or
 * dwconv_group_bwd (backward != 0); the workspace is 16-byte aligned. */
dwconv_status_t dwconv_group_workspace(dwconv_group_t h, int images, int pixels, int backward,
                                       size_t *bytes);

dwconv_status_t dwconv_group_fwd(dwconv_group_t h, int images, int pixels, const void *x,
                                 int64_t ldx, const float *w, const float *b, void *y,
                                 int64_t ldy, void *workspace, hipStream_t stream);

/* Gradients for dy (as y) from the forward pass's inputs: dx (as x; it may be dy itself
 * with lddx == lddy), dw and db (C float, or NULL: not wanted). */
dwconv_status_t dwconv_group_bwd(dwconv_group_t h, int images, int pixels, const void *x,
                                 int64_t ldx, const float *w, const float *b, const void *dy,
                                 int64_t lddy, void *dx, int64_t lddx, float *dw, float *db,
                                 void *workspace, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DWCONV_SEQ_H */
