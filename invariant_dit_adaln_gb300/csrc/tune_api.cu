// C ABI of libadaln.so, third part (declared in include/adaln_tune.h): the
// host-side argument checks, in the order of api.cu, then the launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "checks.h"
#include "ckpt8.cuh"
#include "common.cuh"
#include "rows.h"
#include "tune.h"

using namespace adaln;

namespace {

constexpr double kMaxElements = 1099511627776.0;  // 2^40
constexpr int kMaxLoraChannels = 65536;
constexpr int kMaxAdapters = 65535;
constexpr int kF32MaxRow = 4096;

bool valid_row(int D, int most) { return D >= 8 && D <= most && D % 8 == 0; }
bool valid_norm(int B, int S, int D, int most) {
    return valid_row(D, most) && B >= 0 && B <= 65535 && S >= 0 && S <= kMaxS && (double)B * S * D < kMaxElements;
}
template <typename T>
constexpr int most_channels() { return sizeof(T) == 2 ? kMaxD : kF32MaxRow; }
bool valid_eps(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }

// the shared end of a checked call
#define ADALN_ON_DEVICE(dev)                          \
    DeviceInfo dev;                                   \
    {                                                 \
        const adaln_status st = check_current_device(&dev); \
        if (st != ADALN_OK) return st;                \
    }

// ---- records -----------------------------------------------------------------

template <typename T, typename F>
adaln_status records(const void *in, size_t in_bytes, void *out, size_t out_bytes, int64_t rows, int D, F launch) {
    if (!valid_row(D, kMaxD) || rows < 0 || (double)rows * D >= kMaxElements) return ADALN_ERR_SHAPE;
    const Buf i = {in, (size_t)rows * in_bytes}, o = {out, (size_t)rows * out_bytes};
    if (missing(i) || missing(o)) return ADALN_ERR_NULL;
    if (!aligned16(in) || !aligned16(out)) return ADALN_ERR_ALIGN;
    if (overlaps(i, o)) return ADALN_ERR_ALIAS;
    ADALN_ON_DEVICE(dev)
    return rows == 0 ? ADALN_OK : from_cuda(launch());
}
template <typename T>
adaln_status pack(const T *x, uint8_t *ckpt, int64_t rows, int D, void *stream) {
    return records<T>(x, (size_t)D * sizeof(T), ckpt, ckpt8_row_bytes(D), rows, D,
                      [&] { return launch_ckpt8_pack<T>(x, ckpt, rows, D, (cudaStream_t)stream); });
}
template <typename T>
adaln_status unpack(const uint8_t *ckpt, T *x, int64_t rows, int D, void *stream) {
    return records<T>(ckpt, ckpt8_row_bytes(D), x, (size_t)D * sizeof(T), rows, D,
                      [&] { return launch_ckpt8_unpack<T>(ckpt, x, rows, D, (cudaStream_t)stream); });
}

template <typename T>
adaln_status fwd_ckpt8(const T *x, const T *emb, T *out, float *mean, float *rstd, uint8_t *ckpt, int B, int S, int D,
                       float eps, void *stream) {
    if (!valid_norm(B, S, D, most_channels<T>())) return ADALN_ERR_SHAPE;
    if (!valid_eps(eps)) return ADALN_ERR_ARG;
    const size_t rows = (size_t)B * S;
    const Buf ins[] = {{x, rows * D * sizeof(T)}, {emb, (size_t)B * 2 * D * sizeof(T)}};
    const Buf outs[] = {{out, rows * D * sizeof(T)}, {mean, rows * 4}, {rstd, rows * 4},
                        {ckpt, rows * ckpt8_row_bytes(D)}};
    if (any_missing(ins, 2) || any_missing(outs, 4)) return ADALN_ERR_NULL;
    if (!aligned16(x) || !aligned16(emb) || !aligned16(out) || !aligned16(mean) || !aligned16(rstd) ||
        !aligned16(ckpt))
        return ADALN_ERR_ALIGN;
    if (any_alias(outs, 4, ins, 2)) return ADALN_ERR_ALIAS;
    ADALN_ON_DEVICE(dev)
    if (rows == 0) return ADALN_OK;
    cudaStream_t s = (cudaStream_t)stream;
    if constexpr (sizeof(T) == 2)
        return from_cuda(launch_out_fwd_ckpt8(x, emb, out, mean, rstd, ckpt, B, S, D, eps, s, dev));
    else
        return from_cuda(launch_f32_out_fwd_ckpt8(x, emb, out, mean, rstd, ckpt, B, S, D, eps, s, dev));
}

template <typename T>
adaln_status bwd_ckpt8(const T *dy, const uint8_t *ckpt, const T *emb, const float *mean, const float *rstd, T *dx,
                       float *d_emb, void *workspace, size_t workspace_bytes, int B, int S, int D, void *stream) {
    if (!valid_norm(B, S, D, most_channels<T>())) return ADALN_ERR_SHAPE;
    const size_t rows = (size_t)B * S, need = adaln_out_bwd_ckpt8_workspace_bytes(B, S, D);
    const Buf ins[] = {{dy, rows * D * sizeof(T)}, {ckpt, rows * ckpt8_row_bytes(D)},
                       {emb, (size_t)B * 2 * D * sizeof(T)}, {mean, rows * 4}, {rstd, rows * 4}};
    const Buf outs[] = {{dx, rows * D * sizeof(T)}, {d_emb, (size_t)B * 2 * D * 4}, {workspace, need}};
    if (any_missing(ins, 5) || any_missing(outs, 2)) return ADALN_ERR_NULL;
    if (!aligned16(dy) || !aligned16(ckpt) || !aligned16(emb) || !aligned16(mean) || !aligned16(rstd) ||
        !aligned16(dx) || !aligned16(d_emb) || !aligned16(workspace))
        return ADALN_ERR_ALIGN;
    if (any_alias(outs, 3, ins, 5)) return ADALN_ERR_ALIAS;
    if (need > 0 && (!workspace || workspace_bytes < need)) return ADALN_ERR_WORKSPACE;
    ADALN_ON_DEVICE(dev)
    if (B == 0) return ADALN_OK;
    cudaStream_t s = (cudaStream_t)stream;
    if constexpr (sizeof(T) == 2)
        return from_cuda(launch_out_bwd_ckpt8(dy, ckpt, emb, mean, rstd, dx, d_emb, workspace, B, S, D, s, dev));
    else
        return from_cuda(launch_f32_out_bwd_ckpt8(dy, ckpt, emb, mean, rstd, dx, d_emb, workspace, B, S, D, s, dev));
}

template <typename T>
adaln_status again_ckpt8(const uint8_t *ckpt, const T *emb, const float *mean, const float *rstd, T *out, int B, int S,
                         int D, void *stream) {
    if (!valid_norm(B, S, D, most_channels<T>())) return ADALN_ERR_SHAPE;
    const size_t rows = (size_t)B * S;
    const Buf ins[] = {{ckpt, rows * ckpt8_row_bytes(D)}, {emb, (size_t)B * 2 * D * sizeof(T)}, {mean, rows * 4},
                       {rstd, rows * 4}};
    const Buf outs[] = {{out, rows * D * sizeof(T)}};
    if (any_missing(ins, 4) || any_missing(outs, 1)) return ADALN_ERR_NULL;
    if (!aligned16(ckpt) || !aligned16(emb) || !aligned16(mean) || !aligned16(rstd) || !aligned16(out))
        return ADALN_ERR_ALIGN;
    if (any_alias(outs, 1, ins, 4)) return ADALN_ERR_ALIAS;
    ADALN_ON_DEVICE(dev)
    if (rows == 0) return ADALN_OK;
    return from_cuda(launch_ckpt8_again<T>(ckpt, emb, mean, rstd, out, B, S, D, (cudaStream_t)stream));
}

// ---- adapters ----------------------------------------------------------------

bool valid_rank(int R) { return R >= 8 && R <= kLoraMaxRank && R % 8 == 0; }
bool valid_tokens(int B, int S) { return B >= 0 && B <= 65535 && S >= 0 && S <= kMaxS; }
bool valid_lora(int B, int S, int K, int N, int R) {
    return valid_rank(R) && valid_row(K, kMaxLoraChannels) && valid_row(N, kMaxLoraChannels) && valid_tokens(B, S) &&
           (double)B * S * K < kMaxElements && (double)B * S * N < kMaxElements;
}

// rows [B, S, C] as head rows of one head
adaln_heads heads(const adaln_rows &r) { return {r.data, r.batch, r.token, 0}; }

struct RowsArg {
    const adaln_rows *rows;
    int C;
    bool required;
    bool strided;  // its used strides must be positive
    bool given() const { return rows && rows->data; }
};

// Sizes and strides, arguments, NULL, alignment, overlaps: ins are row tensors
// that are read, out the one written; flat buffers read and written beside them.
adaln_status check_lora(const LoraCall &c, int es, const RowsArg *ins, int nin, const RowsArg &out, int in_place,
                        const Buf *flat_in, int nfi, const Buf *flat_out, int nfo) {
    const int B = c.B, S = c.S;
    const bool empty = B == 0 || S == 0;
    for (int i = 0; i <= nin && !empty; ++i) {
        const RowsArg &r = i < nin ? ins[i] : out;
        if (!r.rows) continue;
        const int64_t st[2] = {r.rows->batch, r.rows->token};
        const int size[2] = {B, S};
        if (!valid_strides(heads(*r.rows), B, S, 1)) return ADALN_ERR_SHAPE;
        for (int k = 0; k < 2; ++k)
            if (size[k] > 1 && ((r.strided && st[k] <= 0) || st[k] >= ((int64_t)1 << 40) / es)) return ADALN_ERR_SHAPE;
    }
    if ((c.ids_are_64 != 0 && c.ids_are_64 != 1) || (c.accumulate != 0 && c.accumulate != 1)) return ADALN_ERR_ARG;
    for (int i = 0; i <= nin && !empty; ++i) {
        const RowsArg &r = i < nin ? ins[i] : out;
        if (r.required && !r.given()) return ADALN_ERR_NULL;
    }
    if (any_missing(flat_in, nfi)) return ADALN_ERR_NULL;
    for (int i = 0; i <= nin && !empty; ++i) {
        const RowsArg &r = i < nin ? ins[i] : out;
        if (r.given() && !aligned_rows(heads(*r.rows), B, S, 1, es)) return ADALN_ERR_ALIGN;
    }
    for (int i = 0; i < nfi; ++i)
        if (!aligned16(flat_in[i].p)) return ADALN_ERR_ALIGN;
    for (int i = 0; i < nfo; ++i)
        if (!aligned16(flat_out[i].p)) return ADALN_ERR_ALIGN;
    if (any_alias(flat_out, nfo, flat_in, nfi)) return ADALN_ERR_ALIAS;
    if (empty) return ADALN_OK;
    for (int i = 0; i < nin; ++i) {
        if (!ins[i].given()) continue;
        const Lattice l = lattice(heads(*ins[i].rows), B, S, 1, ins[i].C, es);
        for (int k = 0; k < nfo; ++k)
            if (overlaps(Buf{ins[i].rows->data, (size_t)l.extent}, flat_out[k])) return ADALN_ERR_ALIAS;
    }
    if (out.given()) {
        const Lattice o = lattice(heads(*out.rows), B, S, 1, out.C, es);
        if (!o.nested) return ADALN_ERR_ALIAS;
        for (int i = 0; i < nin; ++i) {
            if (!ins[i].given()) continue;
            if (i == in_place && same_rows(heads(*out.rows), heads(*ins[i].rows), B, S, 1)) continue;
            if (lattices_overlap(o, lattice(heads(*ins[i].rows), B, S, 1, ins[i].C, es))) return ADALN_ERR_ALIAS;
        }
        const Buf whole = {out.rows->data, (size_t)o.extent};
        for (int k = 0; k < nfi; ++k)
            if (overlaps(whole, flat_in[k])) return ADALN_ERR_ALIAS;
        for (int k = 0; k < nfo; ++k)
            if (overlaps(whole, flat_out[k])) return ADALN_ERR_ALIAS;
    }
    return ADALN_OK;
}

bool valid_adapters(int NA) { return NA >= 0 && NA <= kMaxAdapters; }

// strides of dimensions of size 1 are not used
adaln_rows used_rows(const adaln_rows *r, int B, int S) {
    if (!r || !r->data) return {nullptr, 0, 0};
    return {r->data, B > 1 ? r->batch : 0, S > 1 ? r->token : 0};
}

template <typename T>
adaln_status lora_fwd(const adaln_rows *x, const T *A, const T *U, const float *scale, const void *ids, int ids_are_64,
                      const int32_t *lens, const adaln_rows *y, const adaln_rows *out, void *state, size_t state_bytes,
                      int B, int S, int K, int N, int R, int NA, void *stream) {
    if (!valid_lora(B, S, K, N, R) || !valid_adapters(NA)) return ADALN_ERR_SHAPE;
    LoraCall c = {};
    c.A = A, c.U = U, c.scale = scale, c.ids = ids, c.ids_are_64 = ids_are_64, c.lens = lens, c.state = state;
    c.B = B, c.S = S, c.K = K, c.N = N, c.R = R, c.NA = NA;
    const size_t need = adaln_lora_state_bytes(B, S, R);
    const bool empty = B == 0 || S == 0;
    const RowsArg ins[] = {{x, K, true, true}, {y, N, false, false}}, o = {out, N, true, true};
    const size_t live = empty ? 0 : 1;
    const Buf fi[] = {{A, live * NA * R * K * sizeof(T)}, {U, live * NA * R * N * sizeof(T)}, {scale, live * NA * 4},
                      {ids, live * B * (ids_are_64 ? 8 : 4)}, {lens, lens ? live * B * 4 : 0}};
    const Buf fo[] = {{state, need}};
    adaln_status st = check_lora(c, sizeof(T), ins, 2, o, 1, fi, 5, fo, 1);
    if (st != ADALN_OK) return st;
    if (need > 0 && (!state || state_bytes < need)) return ADALN_ERR_WORKSPACE;
    ADALN_ON_DEVICE(dev)
    if (empty) return ADALN_OK;
    c.x = used_rows(x, B, S), c.base = used_rows(y, B, S), c.out = used_rows(out, B, S);
    return from_cuda(launch_lora_fwd<T>(c, (cudaStream_t)stream, dev));
}

template <typename T>
size_t bwd_bytes(int B, int S, int K, int N, int R) {
    if (B == 0 || S == 0 || !valid_lora(B, S, K, N, R)) return 0;
    return round256(lora_bwd_ws_bytes<T>(B, S, K, N, R));
}

template <typename T>
adaln_status lora_bwd(const adaln_rows *d_out, const adaln_rows *x, const void *state, const T *A, const T *U,
                      const float *scale, const void *ids, int ids_are_64, const int32_t *lens,
                      const adaln_rows *dx_base, const adaln_rows *dx, float *dA_acc, float *dU_acc, int accumulate,
                      void *workspace, size_t workspace_bytes, int B, int S, int K, int N, int R, int NA,
                      void *stream) {
    if (!valid_lora(B, S, K, N, R) || !valid_adapters(NA)) return ADALN_ERR_SHAPE;
    LoraCall c = {};
    c.A = A, c.U = U, c.scale = scale, c.ids = ids, c.ids_are_64 = ids_are_64, c.lens = lens;
    c.state = const_cast<void *>(state), c.dA = dA_acc, c.dU = dU_acc, c.accumulate = accumulate, c.ws = workspace;
    c.B = B, c.S = S, c.K = K, c.N = N, c.R = R, c.NA = NA;
    const size_t need = bwd_bytes<T>(B, S, K, N, R);
    const bool empty = B == 0 || S == 0;
    const RowsArg ins[] = {{d_out, N, true, true}, {x, K, true, true}, {dx_base, K, false, false}},
                  o = {dx, K, false, true};
    const size_t live = empty ? 0 : 1;
    const Buf fi[] = {{A, live * NA * R * K * sizeof(T)}, {U, live * NA * R * N * sizeof(T)}, {scale, live * NA * 4},
                      {ids, live * B * (ids_are_64 ? 8 : 4)}, {lens, lens ? live * B * 4 : 0},
                      {state, adaln_lora_state_bytes(B, S, R)}};
    const Buf fo[] = {{dA_acc, dA_acc ? (size_t)NA * R * K * 4 : 0}, {dU_acc, dU_acc ? (size_t)NA * R * N * 4 : 0},
                      {workspace, need}};
    adaln_status st = check_lora(c, sizeof(T), ins, 3, o, 2, fi, 6, fo, 3);
    if (st != ADALN_OK) return st;
    if (need > 0 && (!workspace || workspace_bytes < need)) return ADALN_ERR_WORKSPACE;
    ADALN_ON_DEVICE(dev)
    if (empty) {
        // no rows: the gradients are their starting value (+0 unless accumulating)
        cudaError_t e = cudaSuccess;
        for (int i = 0; i < 2 && !accumulate; ++i)
            if (fo[i].bytes > 0 && e == cudaSuccess)
                e = cudaMemsetAsync(const_cast<void *>(fo[i].p), 0, fo[i].bytes, (cudaStream_t)stream);
        return from_cuda(e);
    }
    c.d_out = used_rows(d_out, B, S), c.x = used_rows(x, B, S);
    c.base = used_rows(dx_base, B, S), c.out = used_rows(dx, B, S);
    return from_cuda(launch_lora_bwd<T>(c, (cudaStream_t)stream, dev));
}

}  // namespace

extern "C" {

size_t adaln_ckpt8_row_bytes(int D) { return valid_row(D, kMaxD) ? (size_t)ckpt8_row_bytes(D) : 0; }

adaln_status adaln_ckpt8_pack(const adaln_bf16 *x, uint8_t *ckpt, int64_t rows, int D, void *stream) {
    return pack(x, ckpt, rows, D, stream);
}
adaln_status adaln_f32_ckpt8_pack(const float *x, uint8_t *ckpt, int64_t rows, int D, void *stream) {
    return pack(x, ckpt, rows, D, stream);
}
adaln_status adaln_ckpt8_unpack(const uint8_t *ckpt, adaln_bf16 *x, int64_t rows, int D, void *stream) {
    return unpack(ckpt, x, rows, D, stream);
}
adaln_status adaln_f32_ckpt8_unpack(const uint8_t *ckpt, float *x, int64_t rows, int D, void *stream) {
    return unpack(ckpt, x, rows, D, stream);
}

adaln_status adaln_out_fwd_ckpt8(const adaln_bf16 *x, const adaln_bf16 *emb, adaln_bf16 *out, float *mean, float *rstd,
                                 uint8_t *ckpt, int B, int S, int D, float eps, void *stream) {
    return fwd_ckpt8(x, emb, out, mean, rstd, ckpt, B, S, D, eps, stream);
}
adaln_status adaln_f32_out_fwd_ckpt8(const float *x, const float *emb, float *out, float *mean, float *rstd,
                                     uint8_t *ckpt, int B, int S, int D, float eps, void *stream) {
    return fwd_ckpt8(x, emb, out, mean, rstd, ckpt, B, S, D, eps, stream);
}

size_t adaln_out_bwd_ckpt8_workspace_bytes(int B, int S, int D) {
    if (!valid_norm(B, S, D, kMaxD)) return 0;
    return adaln_out_bwd_workspace_bytes(B, S, D);
}

adaln_status adaln_out_bwd_ckpt8(const adaln_bf16 *dy, const uint8_t *ckpt, const adaln_bf16 *emb, const float *mean,
                                 const float *rstd, adaln_bf16 *dx, float *d_emb, void *workspace,
                                 size_t workspace_bytes, int B, int S, int D, void *stream) {
    return bwd_ckpt8(dy, ckpt, emb, mean, rstd, dx, d_emb, workspace, workspace_bytes, B, S, D, stream);
}
adaln_status adaln_f32_out_bwd_ckpt8(const float *dy, const uint8_t *ckpt, const float *emb, const float *mean,
                                     const float *rstd, float *dx, float *d_emb, void *workspace,
                                     size_t workspace_bytes, int B, int S, int D, void *stream) {
    return bwd_ckpt8(dy, ckpt, emb, mean, rstd, dx, d_emb, workspace, workspace_bytes, B, S, D, stream);
}

adaln_status adaln_out_again_ckpt8(const uint8_t *ckpt, const adaln_bf16 *emb, const float *mean, const float *rstd,
                                   adaln_bf16 *out, int B, int S, int D, void *stream) {
    return again_ckpt8(ckpt, emb, mean, rstd, out, B, S, D, stream);
}
adaln_status adaln_f32_out_again_ckpt8(const uint8_t *ckpt, const float *emb, const float *mean, const float *rstd,
                                       float *out, int B, int S, int D, void *stream) {
    return again_ckpt8(ckpt, emb, mean, rstd, out, B, S, D, stream);
}

size_t adaln_lora_state_bytes(int B, int S, int R) {
    return valid_rank(R) && valid_tokens(B, S) ? lora_state_bytes(B, S, R) : 0;
}

adaln_status adaln_lora_fwd(const adaln_rows *x, const adaln_bf16 *A, const adaln_bf16 *U, const float *scale,
                            const void *ids, int ids_are_64, const int32_t *lens, const adaln_rows *y,
                            const adaln_rows *out, void *state, size_t state_bytes, int B, int S, int K, int N, int R,
                            int NA, void *stream) {
    return lora_fwd(x, A, U, scale, ids, ids_are_64, lens, y, out, state, state_bytes, B, S, K, N, R, NA, stream);
}
adaln_status adaln_f32_lora_fwd(const adaln_rows *x, const float *A, const float *U, const float *scale,
                                const void *ids, int ids_are_64, const int32_t *lens, const adaln_rows *y,
                                const adaln_rows *out, void *state, size_t state_bytes, int B, int S, int K, int N,
                                int R, int NA, void *stream) {
    return lora_fwd(x, A, U, scale, ids, ids_are_64, lens, y, out, state, state_bytes, B, S, K, N, R, NA, stream);
}

size_t adaln_lora_bwd_workspace_bytes(int B, int S, int K, int N, int R) { return bwd_bytes<uint16_t>(B, S, K, N, R); }
size_t adaln_f32_lora_bwd_workspace_bytes(int B, int S, int K, int N, int R) { return bwd_bytes<float>(B, S, K, N, R); }

adaln_status adaln_lora_bwd(const adaln_rows *d_out, const adaln_rows *x, const void *state, const adaln_bf16 *A,
                            const adaln_bf16 *U, const float *scale, const void *ids, int ids_are_64,
                            const int32_t *lens, const adaln_rows *dx_base, const adaln_rows *dx, float *dA_acc,
                            float *dU_acc, int accumulate, void *workspace, size_t workspace_bytes, int B, int S,
                            int K, int N, int R, int NA, void *stream) {
    return lora_bwd(d_out, x, state, A, U, scale, ids, ids_are_64, lens, dx_base, dx, dA_acc, dU_acc, accumulate,
                    workspace, workspace_bytes, B, S, K, N, R, NA, stream);
}
adaln_status adaln_f32_lora_bwd(const adaln_rows *d_out, const adaln_rows *x, const void *state, const float *A,
                                const float *U, const float *scale, const void *ids, int ids_are_64,
                                const int32_t *lens, const adaln_rows *dx_base, const adaln_rows *dx, float *dA_acc,
                                float *dU_acc, int accumulate, void *workspace, size_t workspace_bytes, int B, int S,
                                int K, int N, int R, int NA, void *stream) {
    return lora_bwd(d_out, x, state, A, U, scale, ids, ids_are_64, lens, dx_base, dx, dA_acc, dU_acc, accumulate,
                    workspace, workspace_bytes, B, S, K, N, R, NA, stream);
}

}  // extern "C"
