/*
 * dwconv_seq.h -- C ABI of the sequence operators that stand around a short
 * depthwise convolution in a linear-attention block on MI355X (gfx950):
 *
 *   dwconv_causal_*  causal depthwise 1-D convolution of packed sequences
 *   dwconv_delta_*   the gated delta rule (one matrix of state per head)
 *   dwconv_norm_*    norm after a block, gate, residual scale, residual and
 *                    the norm before the next block, in one pass
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
 *
 * float (fp32) everywhere: biases, scales, norm weights, decays, write
 * strengths, matrix states and the gradients of all of these.  Sums and
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

#ifdef __cplusplus
}
#endif

#endif /* DWCONV_SEQ_H */
