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
// lora_tc.cu: the tensor-core forms, for bf16 rows, by S and R (not by B, on which no
// result may depend).  A tile is 128 tokens, so that samples of a few cost them as much
// as long ones, and the CUDA cores' work grows with S R.  Forward and backward, us, on
// the tensor cores and on the CUDA cores:
//     64 samples, 3072 and 3072 channels   rank 8: 48 tokens 72 and 65, 64 tokens 73 and 81;
//       rank 16: 24 tokens 72 and 84, 48 tokens 76 and 107;  rank 32: 16 tokens 71 and 76;
//       rank 64: 8 tokens 118 and 75, 16 tokens 117 and 130;  rank 128: 8 tokens 178 and 131
//     4 samples   rank 16: 24 tokens 32 and 18, 48 tokens 34 and 18, 96 tokens 34 and 22;
//       rank 64: 16 tokens 43 and 26, 64 tokens 40 and 46
// h and e are held as the exact sum of three bf16 parts, transposed:
// [B][3R][Sp], the leading parts of the R ranks, the parts of the rests, theirs;
// Sp = S rounded up to 8.
// --------------------------------------------------------------------------
inline bool lora_tc(int S, int R) { return S >= 12 && S * R >= 640; }
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
