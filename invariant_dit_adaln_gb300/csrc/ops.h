// Internal host-side interface between the C ABI's second part (ops_api.cu)
// and its kernels (heads.cu, embed.cu, grads.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "adaln_ops.h"
#include "internal.h"

namespace adaln {

// heads.cu --------------------------------------------------------------------
struct HeadsCall {
    adaln_heads x[2];   // q, k
    adaln_heads dy[2];  // backward: gradients of the outputs
    adaln_heads out[2]; // forward: outputs; backward: d_q, d_k
    const void *w[2];   // weights or NULL
    const float *cos, *sin;
    const void *pos;
    int pos_is_64;
    int B, S, H[2], Dh, Dr, P;
    int interleaved;
    float eps;
    float *dw[2];  // backward: accumulators or NULL
    int accumulate;
    float *ws;
};
size_t heads_bwd_ws_floats(int B, int S, int Hq, int Hk, int Dh);
template <typename T>
cudaError_t launch_heads_fwd(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev);
template <typename T>
cudaError_t launch_heads_bwd(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev);

// embed.cu --------------------------------------------------------------------
size_t embed_bwd_ws_bytes(int n, int V, int D);
template <typename T>
cudaError_t launch_embed_fwd(const void *tokens, int tokens_are_64, const T *table, float scale, T *out, int n, int V,
                             int D, cudaStream_t stream, const DeviceInfo &dev);
template <typename T>
cudaError_t launch_embed_bwd(const T *d_out, const void *tokens, int tokens_are_64, float scale, float *d_table_acc,
                             uint16_t *d_table, int accumulate, void *ws, int n, int V, int D, cudaStream_t stream,
                             const DeviceInfo &dev);

// grads.cu --------------------------------------------------------------------
// 16 KB pieces of a tensor of `numel` elements
constexpr int64_t kGradPieceBytes = 16384;
inline int64_t grad_pieces(const adaln_tensor &t) {
    const int64_t per = kGradPieceBytes / (t.dtype == ADALN_BF16 ? 2 : 4);
    return (t.numel + per - 1) / per;
}
cudaError_t launch_grad_norm(const adaln_tensor *grads, int count, float *stats, bool clip, double max_norm, void *ws,
                             cudaStream_t stream, const DeviceInfo &dev);
cudaError_t launch_grad_scale(const adaln_tensor *grads, const adaln_tensor *outs, int count, const float *stats,
                              cudaStream_t stream, const DeviceInfo &dev);

}  // namespace adaln
