/*
 * adaln_ops.h — C ABI of libadaln.so, second part: the operators around the
 * modulated norm in a training step or a rollout.
 *
 *   adaln_qk_norm_rope_*   RMS norm of the query and key heads and the position
 *                          rotation, in one pass
 *   adaln_embed_*          embedding lookup with scaling; its gradient summed
 *                          over each token's occurrences in a fixed order
 *   adaln_grad_norm/clip   the global norm of a list of gradients; clipping
 *
 * The conventions of adaln.h hold (device pointers, 16-byte alignment, caller-
 * owned buffers, asynchronous on `stream`, order of the checks, status codes),
 * with the differences stated at each call.  No call allocates or synchronizes
 * (the first one of a kernel on a device keeps a small record on the host), and
 * every call can be captured into a CUDA graph.
 * Two calls (or two replayed graphs) that can run at the same time must not
 * share a workspace or an output.  Thread blocks of this part wait on one
 * another only at the hardware barriers of a cluster, whose blocks run together,
 * so no call sets the words adaln_device_error() reads.
 */
#ifndef ADALN_OPS_H
#define ADALN_OPS_H

#include "adaln.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* Norm of queries and keys, with the position rotation                       */
/* ------------------------------------------------------------------------ */

/*
 * Head rows of a tensor [B, S, H, Dh] with dense channels: element
 * (b, s, h, d) is data[b * batch + s * token + h * head + d], strides in
 * elements, >= 0.  A stride of a dimension of size 1 is not used.  The used
 * strides and `data` are multiples of 16 bytes.  [B, H, S, Dh] storage, or a
 * slice of a fused projection's output, is described by its strides.
 */
typedef struct adaln_heads {
    void *data;
    int64_t batch;
    int64_t token;
    int64_t head;
} adaln_heads;

/*
 * adaln_qk_norm_rope_fwd — for every head row x of q and of k:
 *
 *   r    = 1 / sqrt(sum_d x_d^2 / Dh + eps)       fp32
 *   n_d  = x_d * r * w_d                           fp32 (w = wq or wk; NULL: 1)
 *   the first Dr channels in Dr/2 pairs (a, b), pair i turned by angle i of the
 *   row's position p:
 *     a' = a cos[p,i] - b sin[p,i],  b' = a sin[p,i] + b cos[p,i]
 *   interleaved: pair i is channels (2i, 2i+1); otherwise (i, i + Dr/2)
 *   the other Dh - Dr channels are n_d
 *   out  = the result, rounded once to bf16
 *
 *   q [B,S,Hq,Dh], k [B,S,Hk,Dh]  bf16    input head rows
 *   wq, wk [Dh]                   bf16    weights, or NULL
 *   cos, sin [P, Dr/2]            fp32    tables (NULL when Dr == 0)
 *   pos [B, S]   int32, or int64 if pos_is_64; or NULL: row (b, s) has
 *                position s (then S <= P if Dr > 0)
 *   q_out, k_out                  bf16    output head rows of the same sizes
 *
 * A row whose position is outside [0, P) is padding: its outputs are zero,
 * whatever its inputs hold (infinities and NaN included).  Hk == 0: no keys (k,
 * k_out and wk NULL).
 *
 * In place: q_out may describe exactly q's rows (same data and strides), and
 * k_out k's.  Otherwise no output row may overlap an input row or another output
 * row (ADALN_ERR_ALIAS); rows that interleave without overlapping, as in a
 * fused buffer, are fine.  Output strides must nest (each stride at least the
 * extent of the dimensions inside it), so that no two rows of one output share
 * an element; input strides may be 0 (a broadcast dimension).  Memory between
 * output rows is not written.
 *
 * Sizes: Dh a multiple of 8 in [8, 256]; Dr a multiple of 8 in [0, Dh]; 1 <= Hq
 * <= 1024, 0 <= Hk <= 1024; P >= 0; B, S as in adaln.h; B * S * (Hq + Hk) * Dh <
 * 2^40.  The result of a row does not depend on the other rows.
 */
adaln_status adaln_qk_norm_rope_fwd(const adaln_heads *q, const adaln_heads *k, const adaln_bf16 *wq,
                                    const adaln_bf16 *wk, const float *cos, const float *sin, const void *pos,
                                    int pos_is_64, const adaln_heads *q_out, const adaln_heads *k_out, int B, int S,
                                    int Hq, int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream);

/* The same on fp32 head rows and weights (outputs fp32). */
adaln_status adaln_f32_qk_norm_rope_fwd(const adaln_heads *q, const adaln_heads *k, const float *wq, const float *wk,
                                        const float *cos, const float *sin, const void *pos, int pos_is_64,
                                        const adaln_heads *q_out, const adaln_heads *k_out, int B, int S, int Hq,
                                        int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream);

/* Workspace bytes adaln_qk_norm_rope_bwd and adaln_f32_qk_norm_rope_bwd need
 * when dwq_acc or dwk_acc is given (0 otherwise): fp32 partial sums.  0 for
 * sizes that the calls refuse. */
size_t adaln_qk_norm_rope_bwd_workspace_bytes(int B, int S, int Hq, int Hk, int Dh);

/*
 * adaln_qk_norm_rope_bwd — backward of adaln_qk_norm_rope_fwd, from its inputs
 * (nothing is saved by the forward).  With g = the transposed rotation of the
 * row's output gradient:
 *
 *   h_d     = g_d w_d
 *   dx_d    = r (h_d - x_d r^2 (sum_j h_j x_j) / Dh)    one rounding to bf16
 *   dw_d    = sum over the rows of g_d x_d r             fp32
 *
 * A padding row's gradients are zero and it adds nothing to dw.  dw sums the
 * rows of a sample in an order fixed by (S, Hq, Hk, Dh), then the samples in
 * ascending order onto the accumulator (accumulate ? its value : +0), so dw is
 * bitwise independent of how samples are split into accumulating calls.
 *
 *   d_q_out, d_k_out          input: gradients of q_out, k_out (any strides)
 *   q, k, wq, wk, cos, sin, pos    the forward's inputs
 *   d_q, d_k                  output head rows; d_q may be exactly d_q_out, and
 *                             d_k exactly d_k_out (in place); otherwise the
 *                             forward's rule on overlaps
 *   dwq_acc, dwk_acc [Dh]     fp32 in/out, or NULL (not computed)
 *   workspace  >= adaln_qk_norm_rope_bwd_workspace_bytes when either is given
 *
 * B == 0 or S == 0: no rows; the accumulators get their starting value.
 */
adaln_status adaln_qk_norm_rope_bwd(const adaln_heads *d_q_out, const adaln_heads *d_k_out, const adaln_heads *q,
                                    const adaln_heads *k, const adaln_bf16 *wq, const adaln_bf16 *wk,
                                    const float *cos, const float *sin, const void *pos, int pos_is_64,
                                    const adaln_heads *d_q, const adaln_heads *d_k, float *dwq_acc, float *dwk_acc,
                                    int accumulate, void *workspace, size_t workspace_bytes, int B, int S, int Hq,
                                    int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream);

/* The same on fp32 head rows, gradients and weights. */
adaln_status adaln_f32_qk_norm_rope_bwd(const adaln_heads *d_q_out, const adaln_heads *d_k_out, const adaln_heads *q,
                                        const adaln_heads *k, const float *wq, const float *wk, const float *cos,
                                        const float *sin, const void *pos, int pos_is_64, const adaln_heads *d_q,
                                        const adaln_heads *d_k, float *dwq_acc, float *dwk_acc, int accumulate,
                                        void *workspace, size_t workspace_bytes, int B, int S, int Hq, int Hk, int Dh,
                                        int Dr, int P, int interleaved, float eps, void *stream);

/* ------------------------------------------------------------------------ */
/* Embedding lookup with scaling, and its gradient                            */
/* ------------------------------------------------------------------------ */

/*
 * adaln_embed_fwd — out[i, :] = bf16(scale * table[tokens[i], :]), the product in
 * fp32.  The rows that become temb, adaln_proj_fwd's conditioning vector.
 *
 *   tokens [n]     int32, or int64 if tokens_are_64 (16-byte aligned)
 *   table  [V, D]  bf16
 *   out    [n, D]  bf16
 *
 * A token outside [0, V) is padding: its row of out is zero.  D as in adaln.h;
 * 0 <= n <= 2^24; 0 <= V <= 2^24; n * D and V * D < 2^40; scale finite.
 */
adaln_status adaln_embed_fwd(const void *tokens, int tokens_are_64, const adaln_bf16 *table, float scale,
                             adaln_bf16 *out, int n, int V, int D, void *stream);

/* The same on an fp32 table (out fp32). */
adaln_status adaln_f32_embed_fwd(const void *tokens, int tokens_are_64, const float *table, float scale, float *out,
                                 int n, int V, int D, void *stream);

/* Workspace bytes adaln_embed_bwd and adaln_f32_embed_bwd need: the sorted
 * tokens, the list of pieces, and fp32 partial sums of long runs.  0 for sizes
 * that the calls refuse. */
size_t adaln_embed_bwd_workspace_bytes(int n, int V, int D);

/*
 * adaln_embed_bwd — gradient of the table:
 *
 *   s[v, :]  = sum over i with tokens[i] == v of d_out[i, :]     fp32
 *   d_table_acc[v, :] = (accumulate ? d_table_acc[v, :] : +0) + scale * s[v, :]
 *   or d_table[v, :]  = bf16(scale * s[v, :])
 *
 * The occurrences of a token are taken in ascending order of i, in pieces of
 * 32, each summed from +0; the pieces of a token with more than 32 occurrences
 * are the leaves of a tree of fan-out 32, each node the sum of its children in
 * order from +0.  The order therefore depends on the number of the token's
 * occurrences alone: not on n, on the places or on the other tokens.  Padding
 * tokens (outside [0, V)) add nothing.
 *
 *   d_out       [n, D]  bf16
 *   d_table_acc [V, D]  fp32 in/out, or NULL
 *   d_table     [V, D]  bf16 output, or NULL; exactly one of the two is given
 *                       (ADALN_ERR_ARG), d_table only with accumulate == 0
 *
 * Without accumulate every row is written, zero where a token does not occur;
 * with it, only the rows of tokens that occur are read and written.
 */
adaln_status adaln_embed_bwd(const adaln_bf16 *d_out, const void *tokens, int tokens_are_64, float scale,
                             float *d_table_acc, adaln_bf16 *d_table, int accumulate, void *workspace,
                             size_t workspace_bytes, int n, int V, int D, void *stream);

/* The same on an fp32 d_out (the accumulator is required). */
adaln_status adaln_f32_embed_bwd(const float *d_out, const void *tokens, int tokens_are_64, float scale,
                                 float *d_table_acc, int accumulate, void *workspace, size_t workspace_bytes, int n,
                                 int V, int D, void *stream);

/* ------------------------------------------------------------------------ */
/* Global gradient norm, and clipping                                         */
/* ------------------------------------------------------------------------ */

typedef enum adaln_dtype { ADALN_F32 = 0, ADALN_BF16 = 1 } adaln_dtype;

/* One dense tensor of a list: numel elements at data, which is aligned to its
 * element (16-byte alignment is not needed, but faster). */
typedef struct adaln_tensor {
    void *data;
    int64_t numel;
    int32_t dtype; /* adaln_dtype */
    int32_t reserved;
} adaln_tensor;

/* Workspace bytes adaln_grad_norm and adaln_grad_clip need: 8 bytes for each
 * 16 KB of each tensor.  0 for a list that the calls refuse. */
size_t adaln_grad_norm_workspace_bytes(const adaln_tensor *grads, int count);

/*
 * adaln_grad_norm — norm[0] = sqrt(sum over all elements of all tensors of x^2).
 *
 * Squares are summed in fp32 within 16 KB of a tensor (in fp64 where fp32 would
 * overflow or lose them), then in pairs of fp32 with the additions' errors (or in
 * fp64).  The order is fixed by the list's sizes and types alone, not by
 * addresses.  The result is infinite or NaN exactly as the exact norm (rounded
 * to fp32) is.
 *
 *   grads  host array of `count` tensors (0 <= count <= 65536; read before the
 *          call returns), mixed types; numel >= 0, fewer than 2^40 in all.  A
 *          tensor listed twice counts twice.
 *   norm   [1] fp32 output (device)
 */
adaln_status adaln_grad_norm(const adaln_tensor *grads, int count, float *norm, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * adaln_grad_clip — the norm as above, then
 *
 *   coef   = min(1, max_norm / (norm + 1e-6))     fp64, rounded to fp32
 *   out[i] = round(coef * grad[i])                fp32 product, one rounding
 *   stats  = [norm, coef]                         [2] fp32 output (device)
 *
 * coef is formed from the norm before it is rounded to fp32.  An infinity among
 * the elements gives coef 0 (and NaN where it stands), a NaN gives NaN everywhere;
 * with an infinite max_norm coef is 1 unless the norm is NaN.
 * outs[i] has the numel and dtype of grads[i]; its data may be exactly
 * grads[i]'s (in place: with coef 1 nothing is written then) and must not
 * overlap any other tensor of the two lists, stats or the workspace.  max_norm
 * >= 0 (infinity: never clips).
 */
adaln_status adaln_grad_clip(const adaln_tensor *grads, const adaln_tensor *outs, int count, double max_norm,
                             float *stats, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ADALN_OPS_H */
