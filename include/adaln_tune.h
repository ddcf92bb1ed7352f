/*
 * adaln_tune.h — C ABI of libadaln.so, third part: operators of fine-tuning
 * around the modulated norm.
 *
 *   adaln_*ckpt8*   the norm's input kept in 8 bits for the backward pass: the
 *                   forward writes the 8-bit copy in the same pass, the backward
 *                   reads it, the norm's output is taken again from it
 *   adaln_lora_*    low-rank adapters, one for each sample, added to a shared
 *                   projection's result; their gradients
 *
 * The conventions of adaln.h hold (device pointers, 16-byte alignment, caller-
 * owned buffers, asynchronous on `stream`, order of the checks, status codes),
 * with the differences stated at each call.  No call allocates or synchronizes
 * (the first one of a kernel on a device keeps a small record on the host), and
 * every call can be captured into a CUDA graph.  Waits are bounded as in adaln.h;
 * one of the adapters' kernels that runs out sets adaln_device_error's word: 0x401
 * (x A^T or d_out U^T), 0x402 (gradients), 0x403 (out or dx).
 * Two calls (or two replayed graphs) that can run at the same time must not
 * share a workspace, a state or an output.
 */
#ifndef ADALN_TUNE_H
#define ADALN_TUNE_H

#include "adaln.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* Activations in 8 bits                                                      */
/* ------------------------------------------------------------------------ */

/*
 * A row of D channels is kept as one record of
 *
 *     adaln_ckpt8_row_bytes(D) = 16 ceil(D / 16) + 16 ceil(ceil(D / 32) / 16)
 *
 * bytes: the codes [D] (int8), filled up with zeros to a multiple of 16 bytes,
 * then a scale byte for each group of 32 channels (the last group may be short),
 * filled up the same way.  For a group,
 *
 *     k       = the least integer in [-126, 121] with  max |x_d| 2^-k < 127.5
 *               (121 if none has)
 *     code_d  = x_d 2^-k, rounded to the nearest integer, ties to even, at most 127
 *               in magnitude
 *     scale   = k + 127
 *     value_d = code_d 2^k
 *
 * so |value - x| <= 2^(k-1), which is at most 1/127.5 of the group's largest |x|
 * unless k = -126 (2^k at |x| >= 127.5 2^121).  Every value is an exact bf16 (and fp32)
 * number, and no step depends on a rounded division.  A group that holds an
 * infinity or a NaN gets scale 255 and codes 0: its values are NaN.
 *
 * Records lie densely, [rows][row_bytes], 16-byte aligned.  D as in adaln.h (a
 * multiple of 8 up to 8192; the adaln_f32_* calls of the norm up to 4096).
 */

/* Bytes of a record; 0 for a D that the calls refuse. */
size_t adaln_ckpt8_row_bytes(int D);

/*
 * adaln_ckpt8_pack / _unpack — rows of any activation to records and back.
 *   x    [rows, D]          bf16 (adaln_f32_*: fp32)
 *   ckpt [rows, row_bytes]  records
 * 0 <= rows, rows * D < 2^40.  Scale bytes must be 1 to 255.
 */
adaln_status adaln_ckpt8_pack(const adaln_bf16 *x, uint8_t *ckpt, int64_t rows, int D, void *stream);
adaln_status adaln_f32_ckpt8_pack(const float *x, uint8_t *ckpt, int64_t rows, int D, void *stream);
adaln_status adaln_ckpt8_unpack(const uint8_t *ckpt, adaln_bf16 *x, int64_t rows, int D, void *stream);
adaln_status adaln_f32_ckpt8_unpack(const uint8_t *ckpt, float *x, int64_t rows, int D, void *stream);

/*
 * adaln_out_fwd_ckpt8 — adaln_out_fwd, and the records of x.
 *   out, mean, rstd: the bytes of adaln_out_fwd (from x, not from the records)
 *   ckpt [B, S, row_bytes]: the bytes of adaln_ckpt8_pack
 */
adaln_status adaln_out_fwd_ckpt8(const adaln_bf16 *x, const adaln_bf16 *emb, adaln_bf16 *out, float *mean, float *rstd,
                                 uint8_t *ckpt, int B, int S, int D, float eps, void *stream);
adaln_status adaln_f32_out_fwd_ckpt8(const float *x, const float *emb, float *out, float *mean, float *rstd,
                                     uint8_t *ckpt, int B, int S, int D, float eps, void *stream);

/* Workspace bytes adaln_out_bwd_ckpt8 and adaln_f32_out_bwd_ckpt8 need (the
 * tree nodes, as for adaln_out_bwd).  0 for sizes that the calls refuse. */
size_t adaln_out_bwd_ckpt8_workspace_bytes(int B, int S, int D);

/*
 * adaln_out_bwd_ckpt8 — adaln_out_bwd with x taken from its records: dx and
 * d_emb are the bytes of adaln_out_bwd(dy, unpack(ckpt), emb, mean, rstd), mean
 * and rstd being the forward's (of x before it was rounded to 8 bits).  The
 * fp32 form is to adaln_f32_out_bwd what this one is to adaln_out_bwd.
 */
adaln_status adaln_out_bwd_ckpt8(const adaln_bf16 *dy, const uint8_t *ckpt, const adaln_bf16 *emb, const float *mean,
                                 const float *rstd, adaln_bf16 *dx, float *d_emb, void *workspace,
                                 size_t workspace_bytes, int B, int S, int D, void *stream);
adaln_status adaln_f32_out_bwd_ckpt8(const float *dy, const uint8_t *ckpt, const float *emb, const float *mean,
                                     const float *rstd, float *dx, float *d_emb, void *workspace,
                                     size_t workspace_bytes, int B, int S, int D, void *stream);

/*
 * adaln_out_again_ckpt8 — the norm's output from the records: for the weight
 * gradient of the projection that reads it, which then need not be kept.
 *
 *   xhat = fp32(fp32(value - mean) * rstd)
 *   out  = bf16( fp32( fp32(xhat * onep) + shift ) )    onep = bf16(fp32(1 + scale))
 *
 * (fp32 form: onep and out in fp32.)  Rows never interact.
 */
adaln_status adaln_out_again_ckpt8(const uint8_t *ckpt, const adaln_bf16 *emb, const float *mean, const float *rstd,
                                   adaln_bf16 *out, int B, int S, int D, void *stream);
adaln_status adaln_f32_out_again_ckpt8(const uint8_t *ckpt, const float *emb, const float *mean, const float *rstd,
                                       float *out, int B, int S, int D, void *stream);

/* ------------------------------------------------------------------------ */
/* Low-rank adapters of many samples beside a shared projection               */
/* ------------------------------------------------------------------------ */

/*
 * Rows of a tensor [B, S, C] with dense channels: element (b, s, c) is
 * data[b * batch + s * token + c], strides in elements.  A stride of a dimension
 * of size 1 is not used.  The used strides are multiples of 16 bytes, below 2^40
 * bytes, and `data` is 16-byte aligned.
 */
typedef struct adaln_rows {
    void *data;
    int64_t batch;
    int64_t token;
} adaln_rows;

/* Bytes of the state that adaln_lora_fwd leaves for adaln_lora_bwd.  0 for sizes
 * that the calls refuse. */
size_t adaln_lora_state_bytes(int B, int S, int R);

/*
 * adaln_lora_fwd — out = y + scale_a (x A_a^T) U_a with the adapter a = ids[b] of
 * each sample b:
 *
 *   h[b,s,r]   = scale[a] * sum_k x[b,s,k] A[a,r,k]            fp32
 *   out[b,s,n] = y[b,s,n] + sum_r h[b,s,r] U[a,r,n]            fp32, one rounding
 *
 *   x     [B, S, K]   bf16 rows    the projection's input (used strides > 0)
 *   A     [NA, R, K]  bf16         down-projections
 *   U     [NA, R, N]  bf16         up-projections, a row of N for each rank (the
 *                                  transpose of the usual [N, R])
 *   scale [NA]        fp32
 *   ids   [B]         int32, or int64 if ids_are_64.  An id outside [0, NA): no
 *                     adapter, the sample's out is y
 *   lens  [B]         int32, or NULL (all S): the rows of each sample, taken as 0
 *                     below 0 and as S above S.  Rows from lens[b] on are not
 *                     written, and whatever they hold in x (infinities and NaN
 *                     included) changes nothing
 *   y     [B, S, N]   bf16 rows    the projection's result (strides >= 0), or
 *                                  NULL: zero
 *   out   [B, S, N]   bf16 rows    may describe exactly y's rows (in place)
 *   state             written: what adaln_lora_bwd needs, adaln_lora_state_bytes
 *
 * h is held in fp32.  On the tensor cores (bf16, S >= 12 and S R >= 640) what is added
 * to a sum of up to 768 channels is cut off instead of rounded (8e-7 of h, rms, of random
 * signs; these sums are added with rounding), the product with U takes h to 16
 * significant bits (2^-17 relative), and an |h| above bf16's largest finite number,
 * 3.39e38, counts as infinite (a small one is held to 2^-134).  A row's result does
 * not depend on the other samples; its order depends on K, R and S only.  What an
 * infinity or a NaN enters is infinite or NaN, and nothing else changes.
 *
 * Sizes: K, N multiples of 8 in [8, 65536]; R a multiple of 8 in [8, 128] (fill
 * up smaller adapters with zeros); 0 <= NA <= 65535; B, S as in adaln.h; B * S *
 * K and B * S * N < 2^40.
 *
 * out must not overlap x, A, U, scale, ids, lens or state, nor y's rows unless
 * they are the same; its strides must nest (token >= N, batch >= (S - 1) token +
 * N, or the reverse nesting).  B * S == 0 launches nothing.
 */
adaln_status adaln_lora_fwd(const adaln_rows *x, const adaln_bf16 *A, const adaln_bf16 *U, const float *scale,
                            const void *ids, int ids_are_64, const int32_t *lens, const adaln_rows *y,
                            const adaln_rows *out, void *state, size_t state_bytes, int B, int S, int K, int N, int R,
                            int NA, void *stream);

/* The same on fp32 rows and adapters (out fp32; h in fp32). */
adaln_status adaln_f32_lora_fwd(const adaln_rows *x, const float *A, const float *U, const float *scale,
                                const void *ids, int ids_are_64, const int32_t *lens, const adaln_rows *y,
                                const adaln_rows *out, void *state, size_t state_bytes, int B, int S, int K, int N,
                                int R, int NA, void *stream);

/* Workspace bytes of adaln_lora_bwd and adaln_f32_lora_bwd, whichever of the
 * gradients are asked for.  0 for sizes that the calls refuse. */
size_t adaln_lora_bwd_workspace_bytes(int B, int S, int K, int N, int R);
size_t adaln_f32_lora_bwd_workspace_bytes(int B, int S, int K, int N, int R);

/*
 * adaln_lora_bwd — backward of adaln_lora_fwd, with the state that it left and its
 * A, U, scale, ids and lens:
 *
 *   e[b,s,r]  = scale[a] * sum_n d_out[b,s,n] U[a,r,n]          fp32
 *   dx[b,s,k] = dx_base[b,s,k] + sum_r e[b,s,r] A[a,r,k]        as out
 *   dA[a,r,k] = sum over the rows (b,s) with ids[b] == a of e[b,s,r] x[b,s,k]
 *   dU[a,r,n] = the same of h[b,s,r] d_out[b,s,n]               fp32
 *
 *   d_out   [B, S, N]  bf16 rows   gradient of out (used strides > 0); it is also
 *                                  the gradient of y
 *   dx_base [B, S, K]  bf16 rows   what else flows into x (the shared projection's
 *                                  d_out W), or NULL: zero
 *   dx      [B, S, K]  bf16 rows, or NULL (not computed); may be exactly dx_base
 *   dA_acc  [NA, R, K] fp32 in/out, or NULL (not computed)
 *   dU_acc  [NA, R, N] fp32 in/out, or NULL (not computed)
 *
 * dA and dU sum a sample's rows in an order fixed by S, R and the type, in pieces of
 * consecutive rows that each start from +0, and add the pieces, ascending, sample
 * by sample, onto the accumulator (accumulate ? its value : +0): bitwise
 * independent of how samples are split into accumulating calls.  On the tensor cores
 * a piece has up to 512 rows, what is added to its sum is cut off instead of rounded,
 * and h and e are what adaln_lora_fwd describes.  With accumulate only the adapters
 * that occur are read and written; without it all are, with zeros where an adapter
 * does not occur.  Overlaps as adaln_lora_fwd.
 * B * S == 0: the accumulators get their starting value.
 */
adaln_status adaln_lora_bwd(const adaln_rows *d_out, const adaln_rows *x, const void *state, const adaln_bf16 *A,
                            const adaln_bf16 *U, const float *scale, const void *ids, int ids_are_64,
                            const int32_t *lens, const adaln_rows *dx_base, const adaln_rows *dx, float *dA_acc,
                            float *dU_acc, int accumulate, void *workspace, size_t workspace_bytes, int B, int S,
                            int K, int N, int R, int NA, void *stream);
adaln_status adaln_f32_lora_bwd(const adaln_rows *d_out, const adaln_rows *x, const void *state, const float *A,
                                const float *U, const float *scale, const void *ids, int ids_are_64,
                                const int32_t *lens, const adaln_rows *dx_base, const adaln_rows *dx, float *dA_acc,
                                float *dU_acc, int accumulate, void *workspace, size_t workspace_bytes, int B, int S,
                                int K, int N, int R, int NA, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ADALN_TUNE_H */
