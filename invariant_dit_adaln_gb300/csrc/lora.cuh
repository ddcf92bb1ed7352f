// What the adapters' kernels share (lora.cu: CUDA cores; lora_tc.cu: tensor cores).
#pragma once

#include "common.cuh"
#include "tune.h"

namespace adaln {

// the adapter of sample b, -1 for none
// L2: from L2, not L1, which may hold what an earlier kernel left there: in kernels that
// read before they have waited for the one they follow.
template <bool L2 = false>
__device__ __forceinline__ int adapter_of(const void *ids, int is64, int b, int NA) {
    const long long *p8 = static_cast<const long long *>(ids) + b;
    const int *p4 = static_cast<const int *>(ids) + b;
    const long long i = is64 ? (L2 ? __ldcg(p8) : *p8) : (L2 ? __ldcg(p4) : *p4);
    return i >= 0 && i < NA ? (int)i : -1;
}
template <bool L2 = false>
__device__ __forceinline__ int rows_of(const int *lens, int b, int S) {
    return lens ? min(max(L2 ? __ldcg(lens + b) : lens[b], 0), S) : S;
}

// one side of the gradients: x with e for dA, d_out with h for dU
struct GradOperand {
    const void *src;
    long long batch, token;
    const float *h;  // [B, S, R]
    float *acc;      // [NA, R, C], NULL: not asked for
    float *part;     // [B][pieces][R][C]
    int C;
    int blocks;      // CTAs along the channels
};

// --------------------------------------------------------------------------
// lora_tc.cu: the tensor-core forms, for bf16 rows and more than 16 tokens a
// sample.  h and e are held as the exact sum of three bf16 parts, transposed:
// [B][3R][Sp], the leading parts of the R ranks, the parts of the rests, theirs;
// Sp = S rounded up to 8.
// --------------------------------------------------------------------------
constexpr int kLoraTcMinTokens = 17;
// Consecutive rows of a sample that a gradient sums from +0.  The tensor core cuts
// off what it adds: with 1024 rows the gradients' error was 1.07e-6 (rank 128), half
// of it from there; the pieces' sums are joined with proper rounding.
constexpr int kLoraTcPiece = 512;
cudaError_t lora_tc_shrink(const adaln_rows &src, const void *W, const LoraCall &c, int C, void *h,
                           cudaStream_t stream, const DeviceInfo &dev);
cudaError_t lora_tc_expand(const void *h, const void *W, const LoraCall &c, int C, cudaStream_t stream,
                           const DeviceInfo &dev);
// every piece by itself into part (in_parts), or each adapter's in order
cudaError_t lora_tc_grads(const GradOperand &o0, const GradOperand &o1, const LoraCall &c, bool in_parts,
                          cudaStream_t stream, const DeviceInfo &dev);

}  // namespace adaln
