// Internal host-side interface between the C ABI's third part (tune_api.cu)
// and its kernels (ckpt.cu, lora.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "adaln_tune.h"
#include "internal.h"

namespace adaln {

// ckpt.cu ---------------------------------------------------------------------
template <typename T>
cudaError_t launch_ckpt8_pack(const T *x, uint8_t *ckpt, int64_t rows, int D, cudaStream_t stream);
template <typename T>
cudaError_t launch_ckpt8_unpack(const uint8_t *ckpt, T *x, int64_t rows, int D, cudaStream_t stream);
template <typename T>
cudaError_t launch_ckpt8_again(const uint8_t *ckpt, const T *emb, const float *mean, const float *rstd, T *out, int B,
                               int S, int D, cudaStream_t stream);

// out.cu, f32.cu: the modulated norm with records of its input
cudaError_t launch_out_fwd_ckpt8(const uint16_t *x, const uint16_t *emb, uint16_t *out, float *mean, float *rstd,
                                 uint8_t *ckpt, int B, int S, int D, float eps, cudaStream_t stream,
                                 const DeviceInfo &dev);
cudaError_t launch_out_bwd_ckpt8(const uint16_t *dy, const uint8_t *ckpt, const uint16_t *emb, const float *mean,
                                 const float *rstd, uint16_t *dx, float *d_emb, void *ws, int B, int S, int D,
                                 cudaStream_t stream, const DeviceInfo &dev);
cudaError_t launch_f32_out_fwd_ckpt8(const float *x, const float *emb, float *out, float *mean, float *rstd,
                                     uint8_t *ckpt, int B, int S, int D, float eps, cudaStream_t stream,
                                     const DeviceInfo &dev);
cudaError_t launch_f32_out_bwd_ckpt8(const float *dy, const uint8_t *ckpt, const float *emb, const float *mean,
                                     const float *rstd, float *dx, float *d_emb, void *ws, int B, int S, int D,
                                     cudaStream_t stream, const DeviceInfo &dev);

// lora.cu ---------------------------------------------------------------------
constexpr int kLoraMaxRank = 128;

struct LoraCall {
    adaln_rows x, d_out;     // read; d_out: backward
    adaln_rows base, out;    // y and out, or dx_base and dx; data NULL: none
    const void *A, *U;
    const float *scale;
    const void *ids;
    int ids_are_64;
    const int32_t *lens;
    void *state;             // h
    float *dA, *dU;          // backward: accumulators or NULL
    int accumulate;
    int grads_early;  // the gradients may read before the kernel they follow ends
    void *ws;
    int B, S, K, N, R, NA;
};
// bytes of h or e [B, S, R]
size_t lora_state_bytes(int B, int S, int R);
template <typename T>
size_t lora_bwd_ws_bytes(int B, int S, int K, int N, int R);
template <typename T>
cudaError_t launch_lora_fwd(const LoraCall &c, cudaStream_t stream, const DeviceInfo &dev);
template <typename T>
cudaError_t launch_lora_bwd(const LoraCall &c, cudaStream_t stream, const DeviceInfo &dev);

}  // namespace adaln
