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
    __device__ __forceinline__ void load_kept(const uint16_t *p) { v = ldg16(p); }
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
    __device__ __forceinline__ void load_kept(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
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

// Where a lane's vectors lie.  In rows of more than 512 channels a warp takes 32 kVecs
// vectors (part blockIdx.y) of a row (C == kVecs); in shorter ones C == 2 or 1 steps end
// the row and the next rows follow, and up to 128 channels a row has 4, 8 or 16 lanes (2^lg)
// and several rows share a step.  (104218 rows of 72 channels with a warp a row: pack 39
// us, unpack 17, most of it empty lanes; 11 and 6 so.)
template <int C>
struct Place {
    int sub, v0;           // this lane's row within a step, and its first vector
    int rows;              // rows of a step
    __device__ __forceinline__ explicit Place(int lg) {
        const int lane = threadIdx.x & 31;
        sub = C == 1 ? lane >> lg : 0, rows = C == 1 ? 32 >> lg : 1;
        v0 = C == 1 ? lane & ((1 << lg) - 1) : C == kVecs ? blockIdx.y * 32 * kVecs + lane : lane;
    }
    // the warp's rows, from `first()` on by `step()`; there are `left` steps of rows at `row` (this lane's first)
    __device__ __forceinline__ int taken() const { return kVecs / C * rows; }
    __device__ __forceinline__ long long first() const {
        return ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * taken() + sub;
    }
    __device__ __forceinline__ long long step() const { return (long long)gridDim.x * 8 * taken(); }
    __device__ __forceinline__ int left(long long row, long long all) const {
        const int n = (int)min(all - row, (long long)taken());
        return (n + rows - 1) / rows;
    }
};

// The arithmetic is 30 to 60 instructions a vector: with a division for the place of a
// task, and the halves' largest value by emulated 16-bit maxima, pack issued 154.
template <typename T, int C>
__global__ void __launch_bounds__(256)
ckpt8_pack_kernel(const T *__restrict__ x, unsigned char *__restrict__ ckpt, long long rows, int D, int lg) {
    const int V = D >> 3, P = ckpt8_row_bytes(D), code_bytes = ckpt8_code_bytes(D);
    const Place<C> at(lg);
    const int v0 = at.v0;
    pdl_wait();
    pdl_trigger();
    for (long long row = at.first(); row - at.sub < rows; row += at.step()) {
        const int left = C == kVecs ? 1 : at.left(row, rows);
        const T *src = x + row * D + v0 * 8;
        Eight<T> e[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            e[j].zero();
            if (j / C < left && v0 + 32 * (j % C) < V) e[j].load(src + (long long)(j / C * at.rows) * D + 256 * (j % C));
        }
        uint32_t top[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) top[j] = e[j].max_bits();
        ckpt8_put<kVecs, 8, C>(ckpt + row * P, code_bytes, V, v0, top, [&](int j, px2 (&p)[4]) { e[j].pairs(p); },
                               (size_t)at.rows * P, left);
    }
}

template <typename T, int C>
__global__ void __launch_bounds__(256)
ckpt8_unpack_kernel(const unsigned char *__restrict__ ckpt, T *__restrict__ x, long long rows, int D, int lg) {
    const int V = D >> 3, P = ckpt8_row_bytes(D);
    const Place<C> place(lg);
    const int v0 = place.v0, at = ckpt8_code_bytes(D) + (v0 >> 2);
    pdl_wait();
    pdl_trigger();
    for (long long row = place.first(); row - place.sub < rows; row += place.step()) {
        const int left = C == kVecs ? 1 : place.left(row, rows);
        uint2 c[kVecs];
        uint32_t s[kVecs];
        auto live = [&](int j) { return j / C < left && v0 + 32 * (j % C) < V; };
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            c[j] = make_uint2(0u, 0u), s[j] = 1u;
            if (live(j)) {
                const unsigned char *rec = ckpt + (row + j / C * place.rows) * P;
                c[j] = __ldcs(reinterpret_cast<const uint2 *>(rec + v0 * 8) + 32 * (j % C));
                s[j] = rec[at + 8 * (j % C)];
            }
        }
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            if (!live(j)) continue;
            const px2 step = px_splat(ckpt8_step(s[j]));
            px2 p[4];
            ckpt8_floats(c[j].x, p[0], p[1]);
            ckpt8_floats(c[j].y, p[2], p[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q] = px_mul(p[q], step);
            Eight<T>::store(x + (row + j / C * place.rows) * D + v0 * 8 + 256 * (j % C), p);
        }
    }
}

// A warp takes kAgainRows rows of 256 channels, all requested at once; a lane keeps the
// modulation of its 8 channels in registers, and lane i brings row i's statistics.
// (16 rows, 4 of them requested at once: 21 us for 8192 rows of 3072 channels; the
// modulation read and formed again for each row: 28, bound by issue.)
constexpr int kAgainRows = 8;

template <typename T>
__global__ void __launch_bounds__(256)
ckpt8_again_kernel(const unsigned char *__restrict__ ckpt, const T *__restrict__ emb, const float *__restrict__ mean,
                   const float *__restrict__ rstd, T *__restrict__ out, int S, int D) {
    const int lane = threadIdx.x & 31;
    const int V = D >> 3, P = ckpt8_row_bytes(D);
    const int v = blockIdx.x * 32 + lane, b = blockIdx.z;
    const int s0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kAgainRows;
    pdl_wait();
    pdl_trigger();
    if (s0 >= S) return;  // the whole warp
    const int n = min(kAgainRows, S - s0);
    const bool live = v < V;
    const size_t row0 = (size_t)b * S + s0;
    const unsigned char *rec = ckpt + row0 * P + v * 8, *scales = ckpt + row0 * P + ckpt8_code_bytes(D) + (v >> 2);
    uint2 c[kAgainRows];
    uint32_t s[kAgainRows];
#pragma unroll
    for (int i = 0; i < kAgainRows; ++i) {
        c[i] = make_uint2(0u, 0u), s[i] = 1u;
        if (live && i < n) {
            c[i] = __ldcs(reinterpret_cast<const uint2 *>(rec + (size_t)i * P));
            s[i] = scales[(size_t)i * P];
        }
    }
    float mu = 0.0f, rs = 0.0f;
    if (lane < n) mu = mean[row0 + lane], rs = rstd[row0 + lane];
    px2 onep[4], shift[4];
    {
        Eight<T> e, f;
        e.zero(), f.zero();
        if (live) {
            e.load_kept(emb + (size_t)b * 2 * D + (size_t)v * 8);
            f.load_kept(emb + (size_t)b * 2 * D + D + (size_t)v * 8);
        }
        e.pairs(onep);
        f.pairs(shift);
#pragma unroll
        for (int q = 0; q < 4; ++q) onep[q] = Eight<T>::one_plus(onep[q]);
    }
    T *o = out + row0 * D + (size_t)v * 8;
#pragma unroll
    for (int i = 0; i < kAgainRows; ++i) {
        const px2 nmu = px_splat(-__shfl_sync(0xFFFFFFFFu, mu, i)), r2 = px_splat(__shfl_sync(0xFFFFFFFFu, rs, i)),
                  step = px_splat(ckpt8_step(s[i]));
        if (!live || i >= n) continue;
        px2 p[4];
        ckpt8_floats(c[i].x, p[0], p[1]);
        ckpt8_floats(c[i].y, p[2], p[3]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // the value is code * step exactly, so the fused form is fp32(value - mean)
            const px2 xhat = px_mul(px_fma(p[q], step, nmu), r2);
            p[q] = px_add(px_mul_rounded(xhat, onep[q]), shift[q]);
        }
        Eight<T>::store(o + (size_t)i * D, p);
    }
}

// pack or unpack `rows` rows of V vectors (those of a record's groups included)
template <typename K1, typename K2, typename K4, typename... Args>
cudaError_t launch_rows(K1 k1, K2 k2, K4 k4, int64_t rows, int V, cudaStream_t stream, Args... args) {
    int lg = 2;  // lanes of a row: 4 to 32
    while (lg < 5 && (1 << lg) < V) ++lg;
    const int steps = V <= 32 ? 1 : V <= 64 ? 2 : kVecs;  // of a row
    const int taken = kVecs / steps * (steps == 1 ? 32 >> lg : 1);  // rows of a warp
    const int64_t x = (rows + 8 * taken - 1) / (8 * taken);  // in turns where they are more than a grid has room for
    const dim3 grid((unsigned)(x < (1 << 30) ? x : (1 << 30)), (unsigned)((V + 32 * kVecs - 1) / (32 * kVecs)));
    auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(256), 0, stream, args..., lg); };
    return steps == 1 ? go(k1) : steps == 2 ? go(k2) : go(k4);
}

}  // namespace

template <typename T>
cudaError_t launch_ckpt8_pack(const T *x, uint8_t *ckpt, int64_t rows, int D, cudaStream_t stream) {
    // whole groups: 8 bytes of padding behind the codes are a lane's too
    return launch_rows(ckpt8_pack_kernel<T, 1>, ckpt8_pack_kernel<T, 2>, ckpt8_pack_kernel<T, kVecs>, rows,
                       (D / 8 + 3) & ~3, stream, x, ckpt, (long long)rows, D);
}

template <typename T>
cudaError_t launch_ckpt8_unpack(const uint8_t *ckpt, T *x, int64_t rows, int D, cudaStream_t stream) {
    return launch_rows(ckpt8_unpack_kernel<T, 1>, ckpt8_unpack_kernel<T, 2>, ckpt8_unpack_kernel<T, kVecs>, rows, D / 8,
                       stream, ckpt, x, (long long)rows, D);
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
