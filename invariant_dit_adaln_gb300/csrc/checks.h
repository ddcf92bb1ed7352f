// Host-side checks shared by the C ABI's translation units (api.cu, ops_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "adaln.h"

namespace adaln {

struct Buf {
    const void *p;
    size_t bytes;
};

inline bool overlaps(const Buf &a, const Buf &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Every output against every input, every other output and the workspace.
inline bool any_alias(const Buf *outs, int nout, const Buf *ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlaps(outs[i], ins[j])) return true;
        for (int j = i + 1; j < nout; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

inline bool aligned16(const void *p) { return p == nullptr || ((uintptr_t)p & 15u) == 0; }

// a buffer with bytes > 0 needs a pointer
inline bool missing(const Buf &b) { return b.bytes > 0 && b.p == nullptr; }
inline bool any_missing(const Buf *bufs, int n) {
    for (int i = 0; i < n; ++i)
        if (missing(bufs[i])) return true;
    return false;
}

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

inline adaln_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return ADALN_OK;
    cudaGetLastError();  // clear a non-sticky launch error
    return ADALN_ERR_CUDA;
}

}  // namespace adaln
