// Activations in 8 bits (include/adaln_tune.h): rows to records and back, and
// the modulated norm's output from the records.  The norm's own forward and
// backward with records are forms of its kernels (out.cu, f32.cu).
//
// Everything here streams: a row's channels are read once and written once, and
// a lane's arithmetic is a few instructions for each.
#include "ckpt8.cuh"
#include "tune.h"

namespace adaln {

namespace {

template <typename T>
struct Eight;  // 8 channels of a row
template <>
struct Eight<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const uint16_t *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ uint32_t max_bits() const { return ckpt8_max(v); }
    __device__ __forceinline__ void pairs(px2 (&x)[4]) const {
        x[0] = px_bf16(v.x), x[1] = px_bf16(v.y), x[2] = px_bf16(v.z), x[3] = px_bf16(v.w);
    }
    static __device__ __forceinline__ void store(uint16_t *p, const px2 (&x)[4]) {
        __stcs(reinterpret_cast<uint4 *>(p),
               make_uint4(px_to_bf16x2(x[0]), px_to_bf16x2(x[1]), px_to_bf16x2(x[2]), px_to_bf16x2(x[3])));
    }
    // (1 + scale) rounded to the activations' type
    static __device__ __forceinline__ px2 one_plus(px2 s) {
        return px_bf16(px_to_bf16x2(px_add(px_splat(1.0f), s)));
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void load(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ uint32_t max_bits() const { return ckpt8_max(a, b); }
    __device__ __forceinline__ void pairs(px2 (&x)[4]) const {
        x[0] = px_make(a.x, a.y), x[1] = px_make(a.z, a.w), x[2] = px_make(b.x, b.y), x[3] = px_make(b.z, b.w);
    }
    static __device__ __forceinline__ void store(float *p, const px2 (&x)[4]) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(px_lo(x[0]), px_hi(x[0]), px_lo(x[1]), px_hi(x[1])));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(px_lo(x[2]), px_hi(x[2]), px_lo(x[3]), px_hi(x[3])));
    }
    static __device__ __forceinline__ px2 one_plus(px2 s) { return px_add(px_splat(1.0f), s); }
};

constexpr int kVecs = 4;  // vectors of 8 channels a lane has in flight

// A warp takes 32 kVecs vectors of a row; V is rounded up to whole groups.
template <typename T>
__global__ void __launch_bounds__(256)
ckpt8_pack_kernel(const T *__restrict__ x, unsigned char *__restrict__ ckpt, long long rows, int D) {
    const int lane = threadIdx.x & 31;
    const int V = D >> 3, Vg = (V + 3) & ~3, parts = (Vg + 32 * kVecs - 1) / (32 * kVecs), P = ckpt8_row_bytes(D);
    pdl_wait();
    pdl_trigger();
    for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < rows * parts;
         task += (long long)gridDim.x * 8) {
        const long long row = task / parts;
        const int v0 = (int)(task - row * parts) * 32 * kVecs + lane;
        Eight<T> e[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            e[j].zero();
            if (v0 + 32 * j < V) e[j].load(x + row * D + (size_t)(v0 + 32 * j) * 8);
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (v0 - lane + 32 * j >= Vg) break;  // the whole warp
            px2 p[4];
            e[j].pairs(p);
            ckpt8_put(ckpt + row * P, D, V, v0 + 32 * j, e[j].max_bits(), p);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
ckpt8_unpack_kernel(const unsigned char *__restrict__ ckpt, T *__restrict__ x, long long rows, int D) {
    const int lane = threadIdx.x & 31;
    const int V = D >> 3, parts = (V + 32 * kVecs - 1) / (32 * kVecs), P = ckpt8_row_bytes(D);
    const int at = ckpt8_code_bytes(D);
    pdl_wait();
    pdl_trigger();
    for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < rows * parts;
         task += (long long)gridDim.x * 8) {
        const long long row = task / parts;
        const int v0 = (int)(task - row * parts) * 32 * kVecs + lane;
        const unsigned char *rec = ckpt + row * P;
        uint2 c[kVecs];
        uint32_t s[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int v = v0 + 32 * j;
            c[j] = make_uint2(0u, 0u), s[j] = 1u;
            if (v < V) c[j] = __ldcs(reinterpret_cast<const uint2 *>(rec + (size_t)v * 8)), s[j] = rec[at + (v >> 2)];
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int v = v0 + 32 * j;
            if (v >= V) continue;
            const px2 step = px_splat(ckpt8_step(s[j]));
            px2 p[4];
            ckpt8_floats(c[j].x, p[0], p[1]);
            ckpt8_floats(c[j].y, p[2], p[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q] = px_mul(p[q], step);
            Eight<T>::store(x + row * D + (size_t)v * 8, p);
        }
    }
}

// A lane keeps the modulation of one vector of 8 channels in registers for a run
// of a sample's rows.
constexpr int kAgainRows = 16;  // rows a warp takes
constexpr int kAgainFlight = 4; // of them in flight

template <typename T>
__global__ void __launch_bounds__(256)
ckpt8_again_kernel(const unsigned char *__restrict__ ckpt, const T *__restrict__ emb, const float *__restrict__ mean,
                   const float *__restrict__ rstd, T *__restrict__ out, int S, int D) {
    const int V = D >> 3, P = ckpt8_row_bytes(D), at = ckpt8_code_bytes(D);
    const int v = blockIdx.x * 32 + (threadIdx.x & 31);
    const int b = blockIdx.z;
    const int s0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kAgainRows;
    pdl_wait();
    pdl_trigger();
    if (v >= V || s0 >= S) return;
    px2 onep[4], shift[4];
    {
        Eight<T> e;
        e.load(emb + (size_t)b * 2 * D + (size_t)v * 8);
        e.pairs(onep);
#pragma unroll
        for (int q = 0; q < 4; ++q) onep[q] = Eight<T>::one_plus(onep[q]);
        e.load(emb + (size_t)b * 2 * D + D + (size_t)v * 8);
        e.pairs(shift);
    }
    const int n = min(kAgainRows, S - s0);
    for (int i0 = 0; i0 < n; i0 += kAgainFlight) {
        uint2 c[kAgainFlight];
        uint32_t s[kAgainFlight];
        float mu[kAgainFlight], rs[kAgainFlight];
#pragma unroll
        for (int i = 0; i < kAgainFlight; ++i) {
            c[i] = make_uint2(0u, 0u), s[i] = 1u, mu[i] = rs[i] = 0.0f;
            if (i0 + i < n) {
                const size_t row = (size_t)b * S + s0 + i0 + i;
                const unsigned char *rec = ckpt + row * P;
                c[i] = __ldcs(reinterpret_cast<const uint2 *>(rec + (size_t)v * 8));
                s[i] = rec[at + (v >> 2)];
                mu[i] = mean[row], rs[i] = rstd[row];
            }
        }
#pragma unroll
        for (int i = 0; i < kAgainFlight; ++i) {
            if (i0 + i >= n) break;
            const px2 step = px_splat(ckpt8_step(s[i])), nmu = px_splat(-mu[i]), r2 = px_splat(rs[i]);
            px2 p[4];
            ckpt8_floats(c[i].x, p[0], p[1]);
            ckpt8_floats(c[i].y, p[2], p[3]);
            // the value is code * step exactly, so the fused form is fp32(value - mean)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const px2 xhat = px_mul(px_fma(p[q], step, nmu), r2);
                // rounded before the shift is added: scalar products, since a packed one may be fused into the add
                const px2 m = px_make(__fmul_rn(px_lo(xhat), px_lo(onep[q])), __fmul_rn(px_hi(xhat), px_hi(onep[q])));
                p[q] = px_add(m, shift[q]);
            }
            Eight<T>::store(out + ((size_t)b * S + s0 + i0 + i) * D + (size_t)v * 8, p);
        }
    }
}

unsigned grid_of(long long ctas) { return (unsigned)(ctas < (1 << 30) ? ctas : (1 << 30)); }

}  // namespace

template <typename T>
cudaError_t launch_ckpt8_pack(const T *x, uint8_t *ckpt, int64_t rows, int D, cudaStream_t stream) {
    const int Vg = (D / 8 + 3) & ~3, parts = (Vg + 32 * kVecs - 1) / (32 * kVecs);
    return launch_pdl(ckpt8_pack_kernel<T>, dim3(grid_of((rows * parts + 7) / 8)), dim3(256), 0, stream, x, ckpt,
                      (long long)rows, D);
}

template <typename T>
cudaError_t launch_ckpt8_unpack(const uint8_t *ckpt, T *x, int64_t rows, int D, cudaStream_t stream) {
    const int parts = (D / 8 + 32 * kVecs - 1) / (32 * kVecs);
    return launch_pdl(ckpt8_unpack_kernel<T>, dim3(grid_of((rows * parts + 7) / 8)), dim3(256), 0, stream, ckpt, x,
                      (long long)rows, D);
}

template <typename T>
cudaError_t launch_ckpt8_again(const uint8_t *ckpt, const T *emb, const float *mean, const float *rstd, T *out, int B,
                               int S, int D, cudaStream_t stream) {
    const dim3 grid((D / 8 + 31) / 32, (S + 8 * kAgainRows - 1) / (8 * kAgainRows), B);
    return launch_pdl(ckpt8_again_kernel<T>, grid, dim3(256), 0, stream, ckpt, emb, mean, rstd, out, S, D);
}

#define ADALN_CKPT8(T)                                                                                                 \
    template cudaError_t launch_ckpt8_pack<T>(const T *, uint8_t *, int64_t, int, cudaStream_t);                       \
    template cudaError_t launch_ckpt8_unpack<T>(const uint8_t *, T *, int64_t, int, cudaStream_t);                     \
    template cudaError_t launch_ckpt8_again<T>(const uint8_t *, const T *, const float *, const float *, T *, int,     \
                                               int, int, cudaStream_t);
ADALN_CKPT8(uint16_t)
ADALN_CKPT8(float)

}  // namespace adaln
