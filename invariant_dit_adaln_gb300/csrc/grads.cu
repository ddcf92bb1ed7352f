// Global gradient norm over a list of tensors, and clipping (contract:
// include/adaln_ops.h).
//
//   norm = sqrt(sum x^2),  coef = min(1, max_norm / (norm + 1e-6)),  out = coef x
//
// Bound by HBM: the norm reads every byte once, clipping reads it again and
// writes it.  One CTA takes one 16 KB piece of one tensor (4 16-byte loads in
// flight per thread; with 32 KB 60 ragged tensors of 120 MB take 76 us instead of
// 72, and 1.2 GB 607 instead of 611); the list travels in the kernel's parameters, so nothing
// is copied to the device first and the launch can be captured.  A piece's
// squares are summed in fp32 (8 or 4 terms in each of a thread's four chains,
// then a fixed butterfly), the pieces' sums in compensated fp32 pairs (one SM
// adds fp64 at a few values a cycle: in fp64 the join of 36,864 sums took 20
// us), and in fp64 where the range asks for it.  An element's thread and chain
// depend on its index in the tensor alone, never on an address.
#include "common.cuh"
#include "ops.h"

namespace adaln {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = kGradPieceBytes / 16 / kThreads;  // 16-byte vectors of a thread: 4

// Tensors of one launch; first[i] is the index of tensor i's first piece.
template <int N>
struct GradList {
    const void *in[N];
    void *out[N];
    long long numel[N];
    int first[N + 1];
    unsigned char bf16[N];
    int count;
    int in_place;    // out is in, for every tensor
    long long base;  // pieces of the launches before this one
    float2 *part;  // a piece's sum is x * 2^y, y = 0 but for sums outside fp32's range
    const float *stats;
};

template <int N>
__device__ __forceinline__ int find_tensor(const GradList<N> &a, int piece) {
    int lo = 0, hi = a.count;  // first[lo] <= piece < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.first[mid] <= piece)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// 16 bytes at p, which is aligned to its element of E bytes only, from within
// [base, end): two aligned loads shifted together, or single elements where
// an aligned load would leave the tensor.
template <int E>
__device__ __forceinline__ uint4 load16_any(const char *p, const char *base, const char *end) {
    const unsigned sh = (unsigned)((uintptr_t)p & 15u);
    if (sh == 0) return *reinterpret_cast<const uint4 *>(p);
    const char *q = p - sh;
    uint32_t o[4];
    if (q >= base && q + 32 <= end) {
        const uint4 a = *reinterpret_cast<const uint4 *>(q);
        const uint4 b = *reinterpret_cast<const uint4 *>(q + 16);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const unsigned r = (sh & 3u) * 8u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // sh / 4 == k, the same for the whole tensor
            if ((int)(sh >> 2) == k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[k + i], w[k + i + 1], r);
            }
        }
    } else if (E == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = reinterpret_cast<const uint32_t *>(p)[i];
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (uint32_t)h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// vector j of a piece whose bytes are [p, p + bytes): its 16 bytes, or what is
// left of them and zeros
template <int E>
__device__ __forceinline__ uint4 piece_vec(const char *p, int j, int bytes, const char *base, const char *end) {
    const int at = 16 * j;
    if (at + 16 <= bytes) return load16_any<E>(p + at, base, end);
    uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16 / E; ++i) {
        if (at + i * E + E <= bytes) {
            if (E == 4)
                o[i] = *reinterpret_cast<const uint32_t *>(p + at + 4 * i);
            else
                o[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + at + 2 * i) << (16 * (i & 1));
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int E>
__device__ __forceinline__ void add_squares(float (&acc)[4], uint32_t &any, const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (E == 4) {
            const float f = __uint_as_float(w[i]);
            acc[i] = __fmaf_rn(f, f, acc[i]);
            any |= w[i] & 0x7FFFFFFFu;
        } else {
            const float lo = bf16lo(w[i]), hi = bf16hi(w[i]);
            acc[i] = __fmaf_rn(hi, hi, __fmaf_rn(lo, lo, acc[i]));
            any |= w[i] & 0x7FFF7FFFu;
        }
    }
}

template <int E>
__device__ __forceinline__ double squares_f64(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (E == 4) {
            const double f = (double)__uint_as_float(w[i]);
            s += f * f;
        } else {
            const double lo = (double)bf16lo(w[i]), hi = (double)bf16hi(w[i]);
            s += lo * lo;
            s += hi * hi;
        }
    }
    return s;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Below this a piece's fp32 sum may have lost squares to underflow: a square
// that fp32 rounds or flushes is off by at most 2^-126, 2^13 of them by
// 2^-113, which is 2^-33 of the smallest sum kept.
constexpr float kLeastSum = 0x1p-80f;

// A piece's sum in fp64, read again: rare, so it holds no registers elsewhere.
template <int E>
__device__ __noinline__ void piece_norm_f64(const char *p, int bytes, const char *base, const char *end,
                                            float2 *part) {
    __shared__ double red64[kThreads / 32];
    double d = 0.0;
    for (int i = 0; i < kVecs; ++i) d += squares_f64<E>(piece_vec<E>(p, i * kThreads + threadIdx.x, bytes, base, end));
    d = warp_sum_f64(d);
    if ((threadIdx.x & 31) == 0) red64[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        d = red64[0];
        for (int i = 1; i < kThreads / 32; ++i) d += red64[i];
        int y = 0;
        if (d > 0.0 && d <= 1.7e308) d = frexp(d, &y);
        *part = make_float2((float)d, (float)y);
    }
}

template <int E>
__device__ __forceinline__ void piece_norm(const char *base, long long numel, int piece, float2 *part) {
    __shared__ float red[kThreads / 32];
    __shared__ uint32_t red_any[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const char *p = base + (long long)piece * kGradPieceBytes, *end = base + numel * E;
    const int bytes = (int)min((long long)kGradPieceBytes, (long long)(end - p));
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t any = 0;
    if (bytes == kGradPieceBytes && ((uintptr_t)p & 15u) == 0) {
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = *reinterpret_cast<const uint4 *>(p + 16 * (i * kThreads + threadIdx.x));
#pragma unroll
        for (int i = 0; i < kVecs; ++i) add_squares<E>(acc, any, v[i]);
    } else {
#pragma unroll 2
        for (int i = 0; i < kVecs; ++i)
            add_squares<E>(acc, any, piece_vec<E>(p, i * kThreads + threadIdx.x, bytes, base, end));
    }
    const float s = warp_sum(__fadd_rn(__fadd_rn(acc[0], acc[1]), __fadd_rn(acc[2], acc[3])));
    any = __reduce_or_sync(0xFFFFFFFFu, any);
    if (lane == 0) {
        red[warp] = s;
        red_any[warp] = any;
    }
    __syncthreads();
    float sum = red[0];
    any = red_any[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) {
        sum = __fadd_rn(sum, red[i]);
        any |= red_any[i];
    }
    // the same for every thread: an overflow (or an infinity or NaN of the
    // input), or squares too small for fp32
    if (!(sum <= 3.0e38f) || (any != 0 && sum < kLeastSum))
        piece_norm_f64<E>(p, bytes, base, end, part);
    else if (threadIdx.x == 0)
        *part = make_float2(sum, 0.0f);
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ GradList<N> a) {
    const int t = find_tensor(a, (int)blockIdx.x);
    const int piece = (int)blockIdx.x - a.first[t];
    float2 *part = a.part + a.base + blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (a.bf16[t])
        piece_norm<2>(static_cast<const char *>(a.in[t]), a.numel[t], piece, part);
    else
        piece_norm<4>(static_cast<const char *>(a.in[t]), a.numel[t], piece, part);
}

// the warp's pairs s + c, joined by a fixed butterfly; the same in every lane
__device__ __forceinline__ void warp_twosum(float &s, float &c) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float so = __shfl_xor_sync(0xFFFFFFFFu, s, off);
        c = __fadd_rn(c, __shfl_xor_sync(0xFFFFFFFFu, c, off));
        float t = lane & off ? so : s;  // one order in both lanes
        twosum(t, c, lane & off ? s : so);
        s = t;
    }
}

// The pieces' sums in a fixed order (thread i takes i, i + 1024, ..., then a
// butterfly and the warps), the norm and, with clip, the coefficient.  A sum is
// a pair s + c with the error of every addition in c.
__global__ void __launch_bounds__(1024) grad_norm_kernel(const float2 *__restrict__ part, int n, float *stats,
                                                         int clip, double max_norm) {
    __shared__ float red_s[32], red_c[32];
    __shared__ double red64[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    float s = 0.0f, c = 0.0f;
    bool scaled = false;
    for (int i = threadIdx.x; i < n; i += 16 * 1024) {
        float2 v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = part[min(i + k * 1024, n - 1)];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const bool in = i + k * 1024 < n;
            scaled |= in && v[k].y != 0.0f;
            twosum(s, c, in ? v[k].x : 0.0f);
        }
    }
    warp_twosum(s, c);
    if (lane == 0) red_s[warp] = s, red_c[warp] = c;
    scaled = __syncthreads_or(scaled);  // also publishes red_s, red_c
    s = red_s[lane], c = red_c[lane];
    warp_twosum(s, c);  // every warp: the same for all
    double total = (double)s + (double)c;
    if (scaled || !(s <= 3.0e38f)) {
        total = 0.0;
        for (int i = threadIdx.x; i < n; i += 1024) total += scalbn((double)part[i].x, (int)part[i].y);
        total = warp_sum_f64(total);
        if (lane == 0) red64[warp] = total;
        __syncthreads();
        total = warp_sum_f64(red64[lane]);
    }
    if (threadIdx.x == 0) {
        const double norm = sqrt(total);
        stats[0] = (float)norm;
        if (clip) {
            // an infinite max_norm clips nothing; a NaN norm passes on
            const double f = isinf(max_norm) && norm == norm ? 1.0 : max_norm / (norm + 1e-6);
            stats[1] = f >= 1.0 ? 1.0f : (float)f;
        }
    }
}

template <int E>
__device__ __forceinline__ uint4 scaled(const uint4 &v, float c) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (E == 4)
            w[i] = __float_as_uint(__fmul_rn(__uint_as_float(w[i]), c));
        else
            w[i] = pack_bf16x2(__fmul_rn(bf16lo(w[i]), c), __fmul_rn(bf16hi(w[i]), c));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int E>
__device__ __forceinline__ void scale_one(const char *src, char *dst, float c) {
    if (E == 4)
        *reinterpret_cast<float *>(dst) = __fmul_rn(*reinterpret_cast<const float *>(src), c);
    else
        *reinterpret_cast<uint16_t *>(dst) = bf16_bits(__fmul_rn(bf16f(*reinterpret_cast<const uint16_t *>(src)), c));
}

// One piece of out = c * in: the elements before the first 16-byte boundary
// of out, whole vectors of out, and the rest.
template <int E>
__device__ void piece_scale(const char *base, char *out, long long numel, int piece, float c) {
    const long long off = (long long)piece * kGradPieceBytes;
    const char *src = base + off, *end = base + numel * E;
    char *dst = out + off;
    const int bytes = (int)min((long long)kGradPieceBytes, (long long)(end - src));
    const int head = min(bytes, (int)((16u - (unsigned)((uintptr_t)dst & 15u)) & 15u));
    const int vecs = (bytes - head) / 16, tail = head + 16 * vecs;
    // vectors of this thread: vec = threadIdx.x + i * kThreads
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int j = i * kThreads + threadIdx.x;
        if (j < vecs) v[i] = load16_any<E>(src + head + 16 * j, base, end);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int j = i * kThreads + threadIdx.x;
        if (j < vecs) *reinterpret_cast<uint4 *>(dst + head + 16 * j) = scaled<E>(v[i], c);
    }
    const int at = (int)threadIdx.x * E;  // fewer than 16 bytes on either side
    if (at < head) scale_one<E>(src + at, dst + at, c);
    if (tail + at < bytes) scale_one<E>(src + tail + at, dst + tail + at, c);
}

// One CTA a piece here too: as many CTAs as the device holds, each over several
// pieces, took 660 us instead of 607 for 1.2 GB.
template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ GradList<N> a) {
    pdl_wait();
    pdl_trigger();
    const float c = __ldcg(a.stats + 1);
    if (c == 1.0f && a.in_place) return;
    // last pieces first: the norm read them last, so L2 still holds them
    const int at = (int)(gridDim.x - 1 - blockIdx.x);
    const int t = find_tensor(a, at);
    const int piece = at - a.first[t];
    if (c == 1.0f && a.in[t] == a.out[t]) return;
    if (a.bf16[t])
        piece_scale<2>(static_cast<const char *>(a.in[t]), static_cast<char *>(a.out[t]), a.numel[t], piece, c);
    else
        piece_scale<4>(static_cast<const char *>(a.in[t]), static_cast<char *>(a.out[t]), a.numel[t], piece, c);
}

// Fills a list from tensors [from, from + N) with elements; returns the first
// tensor not taken.  Tensors without elements take no entry.
template <int N>
int fill(GradList<N> &a, const adaln_tensor *in, const adaln_tensor *out, int from, int count) {
    a.count = 0;
    a.in_place = 1;
    a.first[0] = 0;
    int i = from;
    for (; i < count && a.count < N; ++i) {
        if (in[i].numel == 0) continue;
        const int64_t pieces = grad_pieces(in[i]);
        if ((int64_t)a.first[a.count] + pieces > 0x7FFFFFFF) break;
        a.in[a.count] = in[i].data;
        a.out[a.count] = out ? out[i].data : nullptr;
        if (a.out[a.count] != a.in[a.count]) a.in_place = 0;
        a.numel[a.count] = in[i].numel;
        a.bf16[a.count] = in[i].dtype == ADALN_BF16;
        a.first[a.count + 1] = a.first[a.count] + (int)pieces;
        ++a.count;
    }
    return i;
}

// One launch per N tensors (at most 2^31 - 1 pieces): squares, or scaling when
// outs is given.
template <int N>
cudaError_t run(const adaln_tensor *in, const adaln_tensor *out, int count, float2 *part, const float *stats,
                cudaStream_t stream) {
    GradList<N> a;
    a.base = 0;
    a.part = part;
    a.stats = stats;
    for (int i = 0; i < count;) {
        i = fill(a, in, out, i, count);
        if (a.count == 0) break;
        const dim3 grid((unsigned)a.first[a.count]);
        const cudaError_t e = out ? launch_pdl(grad_scale_kernel<N>, grid, dim3(kThreads), 0, stream, a)
                                  : launch_pdl(grad_squares_kernel<N>, grid, dim3(kThreads), 0, stream, a);
        if (e != cudaSuccess) return e;
        a.base += a.first[a.count];
    }
    return cudaSuccess;
}

// The parameter block is copied at every launch, so short lists take a short one.
cudaError_t run_any(const adaln_tensor *in, const adaln_tensor *out, int count, float2 *part, const float *stats,
                    cudaStream_t stream) {
    if (count <= 16) return run<16>(in, out, count, part, stats, stream);
    if (count <= 128) return run<128>(in, out, count, part, stats, stream);
    return run<1024>(in, out, count, part, stats, stream);
}

}  // namespace

cudaError_t launch_grad_norm(const adaln_tensor *grads, int count, float *stats, bool clip, double max_norm, void *ws,
                             cudaStream_t stream, const DeviceInfo &) {
    float2 *part = static_cast<float2 *>(ws);
    cudaError_t e = run_any(grads, nullptr, count, part, nullptr, stream);
    if (e != cudaSuccess) return e;
    long long pieces = 0;
    for (int i = 0; i < count; ++i) pieces += grad_pieces(grads[i]);
    return launch_pdl(grad_norm_kernel, dim3(1), dim3(1024), 0, stream, (const float2 *)part, (int)pieces, stats,
                      clip ? 1 : 0, max_norm);
}

cudaError_t launch_grad_scale(const adaln_tensor *grads, const adaln_tensor *outs, int count, const float *stats,
                              cudaStream_t stream, const DeviceInfo &) {
    return run_any(grads, outs, count, nullptr, stats, stream);
}

}  // namespace adaln
