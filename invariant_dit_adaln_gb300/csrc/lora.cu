// Low-rank adapters, one for each sample, beside a shared projection
// (include/adaln_tune.h): forward, and the gradients.
//
// With W = A or U, [NA, R, C] in both directions, three products make up a call:
//     shrink   h[b,s,:] = scale_a W_a src[b,s,:]           (x with A; d_out with U)
//     expand   out[b,s,:] = base[b,s,:] + h[b,s,:] W_a     (h with U; e with A)
//     grad     dW_a = sum over rows of h[b,s,:] src[b,s,:]^T
// 2 R flop for each channel read or written: bound by memory for bf16 on the
// tensor cores; on the CUDA cores (fp32, and samples of a few tokens) by issue
// from R = 16 or so on.
#include "common.cuh"
#include "tune.h"

namespace adaln {

namespace {

constexpr int kRB = 8;           // ranks a warp (shrink) or a thread (grad) holds
constexpr int kGradPiece = 256;  // consecutive rows of a sample that the gradient sums from +0

template <typename T>
struct Vec;  // 16 bytes of a row as pairs
template <>
struct Vec<uint16_t> {
    static constexpr int E = 8;
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const uint16_t *p) { v = ldg16(p); }
    __device__ __forceinline__ void pairs(px2 (&x)[4]) const {
        x[0] = px_bf16(v.x), x[1] = px_bf16(v.y), x[2] = px_bf16(v.z), x[3] = px_bf16(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const px2 (&x)[4]) {
        return make_uint4(px_to_bf16x2(x[0]), px_to_bf16x2(x[1]), px_to_bf16x2(x[2]), px_to_bf16x2(x[3]));
    }
};
template <>
struct Vec<float> {
    static constexpr int E = 4;
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const float *p) { v = ldg16(p); }
    __device__ __forceinline__ void pairs(px2 (&x)[2]) const {
        x[0] = px_make(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = px_make(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const px2 (&x)[2]) {
        return make_uint4(__float_as_uint(px_lo(x[0])), __float_as_uint(px_hi(x[0])), __float_as_uint(px_lo(x[1])),
                          __float_as_uint(px_hi(x[1])));
    }
};

// the adapter of sample b, -1 for none
__device__ __forceinline__ int adapter_of(const void *ids, int is64, int b, int NA) {
    const long long i = is64 ? static_cast<const long long *>(ids)[b] : static_cast<const int *>(ids)[b];
    return i >= 0 && i < NA ? (int)i : -1;
}
__device__ __forceinline__ int rows_of(const int *lens, int b, int S) { return lens ? min(max(lens[b], 0), S) : S; }

// NV values of every lane summed over the warp by a transposed butterfly: lane l
// ends with value l mod NV.  The order of a sum does not depend on NV.
template <int NV>
__device__ __forceinline__ float scatter_sum(float (&a)[NV], int lane) {
    static_assert(NV >= 1 && NV <= 32 && (NV & (NV - 1)) == 0, "a power of two");
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        if (off >= NV) {
#pragma unroll
            for (int q = 0; q < NV; ++q) a[q] = __fadd_rn(a[q], __shfl_xor_sync(0xFFFFFFFFu, a[q], off));
        } else {
            const bool up = (lane & off) != 0;
#pragma unroll
            for (int q = 0; q < off; ++q) {
                const float keep = up ? a[q + off] : a[q], give = up ? a[q] : a[q + off];
                a[q] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, off));
            }
        }
    }
    return a[0];
}

// --------------------------------------------------------------------------
// shrink: a warp (KS == 1) or the CTA's four warps (KS == 4, the channels split
// among them) form kRB ranks of TOK tokens of a sample.  A lane takes the 16-byte
// vectors of its share in ascending order, even and odd channels in the halves of
// a packed accumulator; halves, butterfly, warps ascending.  State fp32 [B,S,R].
// --------------------------------------------------------------------------
template <typename T, int TOK, int KS>
__global__ void __launch_bounds__(128)
lora_shrink_kernel(const T *__restrict__ src, long long batch, long long token, const T *__restrict__ W,
                   const float *__restrict__ scale, const void *ids, int is64, const int *lens,
                   float *__restrict__ h, int S, int C, int R, int NA) {
    constexpr int E = Vec<T>::E, V = TOK * kRB;
    __shared__ float part[KS][V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, r0 = blockIdx.y * kRB;
    const int s0 = (KS == 4 ? blockIdx.x : blockIdx.x * 4 + warp) * TOK;
    pdl_wait();
    pdl_trigger();
    const int a = adapter_of(ids, is64, b, NA);
    const int n = a < 0 ? 0 : min(TOK, rows_of(lens, b, S) - s0);
    px2 acc[TOK][kRB];
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
        for (int r = 0; r < kRB; ++r) acc[i][r] = 0ull;
    if (n > 0) {
        const T *w = W + ((long long)a * R + r0) * C, *x = src + b * batch + s0 * token;
        for (int v = KS == 4 ? (int)threadIdx.x : lane; v < C / E; v += KS == 4 ? 128 : 32) {
            Vec<T> xv[TOK];
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                xv[i].zero();
                if (i < n) xv[i].load(x + i * token + (long long)v * E);
            }
            px2 xp[TOK][E / 2];
#pragma unroll
            for (int i = 0; i < TOK; ++i) xv[i].pairs(xp[i]);
#pragma unroll
            for (int r = 0; r < kRB; ++r) {
                Vec<T> wv;
                wv.load(w + (long long)r * C + (long long)v * E);
                px2 wp[E / 2];
                wv.pairs(wp);
#pragma unroll
                for (int i = 0; i < TOK; ++i)
#pragma unroll
                    for (int q = 0; q < E / 2; ++q) acc[i][r] = px_fma(xp[i][q], wp[q], acc[i][r]);
            }
        }
    }
    float sum[V];
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
        for (int r = 0; r < kRB; ++r) sum[i * kRB + r] = __fadd_rn(px_lo(acc[i][r]), px_hi(acc[i][r]));
    float mine = scatter_sum<V>(sum, lane);
    if (KS == 4) {
        if (lane < V) part[warp & (KS - 1)][lane] = mine;
        __syncthreads();
        if (warp > 0) return;
        if (lane < V)
            for (int k = 1; k < KS; ++k) mine = __fadd_rn(mine, part[k][lane]);
    }
    // every row of the state is written: zeros where there is no adapter or no row
    if (lane < V && s0 + lane / kRB < S) {
        const float c = a < 0 ? 0.0f : scale[a];
        h[((long long)b * S + s0 + lane / kRB) * R + r0 + lane % kRB] = lane / kRB < n ? __fmul_rn(c, mine) : 0.0f;
    }
}

// --------------------------------------------------------------------------
// expand: a thread holds 16 bytes of channels of TOK tokens; the ranks ascending,
// then the base, one rounding.
// --------------------------------------------------------------------------
template <typename T, int TOK>
__global__ void __launch_bounds__(128)
lora_expand_kernel(const float *__restrict__ h, const T *__restrict__ W, const void *ids, int is64, const int *lens,
                   const T *base, long long base_batch, long long base_token, T *out, long long batch, long long token,
                   int S, int C, int R, int NA) {
    constexpr int E = Vec<T>::E;
    __shared__ float hs[TOK][kLoraMaxRank];
    const int b = blockIdx.z, s0 = blockIdx.y * TOK;
    const int c0 = (blockIdx.x * 128 + threadIdx.x) * E;
    pdl_wait();
    pdl_trigger();
    const int n = min(TOK, rows_of(lens, b, S) - s0);
    if (n <= 0) return;
    const int a = adapter_of(ids, is64, b, NA);
    if (a < 0 && base == out) return;
    for (int i = threadIdx.x; i < TOK * R; i += 128)
        hs[i / R][i % R] = i / R < n ? h[((long long)b * S + s0) * R + i] : 0.0f;
    __syncthreads();
    if (c0 >= C) return;
    px2 acc[TOK][E / 2];
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
        for (int q = 0; q < E / 2; ++q) acc[i][q] = 0ull;
    if (a >= 0) {
        const T *w = W + (long long)a * R * C + c0;
#pragma unroll 4
        for (int r = 0; r < R; ++r) {
            Vec<T> wv;
            wv.load(w + (long long)r * C);
            px2 wp[E / 2];
            wv.pairs(wp);
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                const px2 hr = px_splat(hs[i][r]);
#pragma unroll
                for (int q = 0; q < E / 2; ++q) acc[i][q] = px_fma(hr, wp[q], acc[i][q]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
        if (i >= n) break;
        if (base) {
            Vec<T> y;
            // not the read-only path: base may be out
            y.v = *reinterpret_cast<const uint4 *>(base + b * base_batch + (s0 + i) * base_token + c0);
            px2 yp[E / 2];
            y.pairs(yp);
#pragma unroll
            for (int q = 0; q < E / 2; ++q) acc[i][q] = px_add(yp[q], acc[i][q]);
        }
        stg16(out + b * batch + (s0 + i) * token + c0, Vec<T>::pack(acc[i]));
    }
}

// --------------------------------------------------------------------------
// grad: a thread holds 4 channels of kRB ranks.  A piece is kGradPiece
// consecutive rows of a sample, summed from +0 by fused multiply-adds in
// ascending order; the pieces are added in ascending order, sample by sample.
//
// Two schedules of the same sums.  OWNER: the CTA takes every piece of an
// adapter and writes the accumulator.  Otherwise each CTA takes one piece, writes
// its sum to the workspace, and lora_join_kernel adds them.  The second has as
// many CTAs as there are pieces, and moves R fp32 for each channel of a piece
// twice.
// --------------------------------------------------------------------------
struct GradOperand {
    const void *src;
    long long batch, token;
    const float *h;  // [B, S, R]
    float *acc;      // [NA, R, C], NULL: not asked for
    float *part;     // [B][pieces][R][C]
    int C;
    int blocks;      // CTAs along the channels
};

template <typename T>
__device__ __forceinline__ void load4(const T *p, px2 (&x)[2]);
template <>
__device__ __forceinline__ void load4<uint16_t>(const uint16_t *p, px2 (&x)[2]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = px_bf16(v.x), x[1] = px_bf16(v.y);
}
template <>
__device__ __forceinline__ void load4<float>(const float *p, px2 (&x)[2]) {
    const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = px_make(v.x, v.y), x[1] = px_make(v.z, v.w);
}

// rows [s0, s1) of a sample into acc, from what it holds
template <typename T>
__device__ __forceinline__ void grad_rows(const GradOperand &o, int b, int s0, int s1, int S, int R, int r0, int c0,
                                          px2 (&acc)[kRB][2]) {
    const T *x = static_cast<const T *>(o.src) + b * o.batch + s0 * o.token + c0;
    const float *h = o.h + ((long long)b * S + s0) * R + r0;
#pragma unroll 4
    for (int s = s0; s < s1; ++s, x += o.token, h += R) {
        px2 xp[2];
        load4<T>(x, xp);
        const float4 ha = __ldg(reinterpret_cast<const float4 *>(h)), hb = __ldg(reinterpret_cast<const float4 *>(h) + 1);
        const float hr[kRB] = {ha.x, ha.y, ha.z, ha.w, hb.x, hb.y, hb.z, hb.w};
#pragma unroll
        for (int r = 0; r < kRB; ++r) {
            const px2 e = px_splat(hr[r]);
            acc[r][0] = px_fma(e, xp[0], acc[r][0]);
            acc[r][1] = px_fma(e, xp[1], acc[r][1]);
        }
    }
}

template <typename T, bool OWNER>
__global__ void __launch_bounds__(128)
lora_grad_kernel(const GradOperand o0, const GradOperand o1, const void *ids, int is64, const int *lens, int accumulate,
                 int B, int S, int R, int NA, int pieces) {
    const int rb = R / kRB;
    const bool first = (int)blockIdx.x < o0.blocks * rb;
    const GradOperand &o = first ? o0 : o1;
    const int at = first ? blockIdx.x : blockIdx.x - o0.blocks * rb;
    const int r0 = at / o.blocks * kRB, c0 = (at % o.blocks * 128 + threadIdx.x) * 4;
    const bool live = c0 < o.C;
    pdl_wait();
    pdl_trigger();
    px2 sum[kRB][2], acc[kRB][2];
    if (!OWNER) {
        const int b = blockIdx.z, s0 = blockIdx.y * kGradPiece;
        const int s1 = min(rows_of(lens, b, S), s0 + kGradPiece);
        if (s0 >= s1 || adapter_of(ids, is64, b, NA) < 0 || !live) return;
#pragma unroll
        for (int r = 0; r < kRB; ++r) acc[r][0] = acc[r][1] = 0ull;
        grad_rows<T>(o, b, s0, s1, S, R, r0, c0, acc);
        float *p = o.part + (((long long)b * pieces + blockIdx.y) * R + r0) * o.C + c0;
#pragma unroll
        for (int r = 0; r < kRB; ++r)
            stg16f(p + (long long)r * o.C,
                   make_float4(px_lo(acc[r][0]), px_hi(acc[r][0]), px_lo(acc[r][1]), px_hi(acc[r][1])));
        return;
    }
    const int a = blockIdx.y;
    float *p = o.acc + ((long long)a * R + r0) * o.C + c0;
    bool any = false;
#pragma unroll
    for (int r = 0; r < kRB; ++r) sum[r][0] = sum[r][1] = 0ull;
    __shared__ int found[128];
    __shared__ int count[4];
    for (int b0 = 0; b0 < B; b0 += 128) {
        // the samples of adapter a among the next 128, in order
        const int b = b0 + threadIdx.x;
        const bool mine = b < B && adapter_of(ids, is64, b, NA) == a;
        const unsigned vote = __ballot_sync(0xFFFFFFFFu, mine);
        if ((threadIdx.x & 31) == 0) count[threadIdx.x >> 5] = __popc(vote);
        __syncthreads();
        int before = 0, total = 0;
        for (int w = 0; w < 4; ++w) {
            if (w < (int)(threadIdx.x >> 5)) before += count[w];
            total += count[w];
        }
        if (mine) found[before + __popc(vote & ((1u << (threadIdx.x & 31)) - 1u))] = b;
        __syncthreads();
        if (live) {
            if (total > 0 && !any) {
                any = true;
                if (accumulate)
#pragma unroll
                    for (int r = 0; r < kRB; ++r) {
                        const float4 v = *reinterpret_cast<const float4 *>(p + (long long)r * o.C);
                        sum[r][0] = px_make(v.x, v.y), sum[r][1] = px_make(v.z, v.w);
                    }
            }
            for (int i = 0; i < total; ++i) {
                const int bb = found[i], n = rows_of(lens, bb, S);
                for (int s0 = 0; s0 < n; s0 += kGradPiece) {
#pragma unroll
                    for (int r = 0; r < kRB; ++r) acc[r][0] = acc[r][1] = 0ull;
                    grad_rows<T>(o, bb, s0, min(n, s0 + kGradPiece), S, R, r0, c0, acc);
#pragma unroll
                    for (int r = 0; r < kRB; ++r)
                        sum[r][0] = px_add(sum[r][0], acc[r][0]), sum[r][1] = px_add(sum[r][1], acc[r][1]);
                }
            }
        }
        __syncthreads();
    }
    if (live && (any || !accumulate))
#pragma unroll
        for (int r = 0; r < kRB; ++r)
            stg16f(p + (long long)r * o.C,
                   make_float4(px_lo(sum[r][0]), px_hi(sum[r][0]), px_lo(sum[r][1]), px_hi(sum[r][1])));
}

// The pieces' sums onto the accumulators: a thread holds 4 channels of a rank.
__global__ void __launch_bounds__(128)
lora_join_kernel(const GradOperand o0, const GradOperand o1, const void *ids, int is64, const int *lens, int accumulate,
                 int B, int S, int R, int NA, int pieces, int piece_rows) {
    const int n0 = o0.acc ? R * (o0.C / 4) : 0, n1 = o1.acc ? R * (o1.C / 4) : 0;
    int i = blockIdx.x * 128 + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (i >= n0 + n1) return;
    const GradOperand &o = i < n0 ? o0 : o1;
    if (i >= n0) i -= n0;
    const int a = blockIdx.y;
    const long long size = (long long)R * o.C;  // of a piece
    float4 *p = reinterpret_cast<float4 *>(o.acc + a * size) + i;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool any = false;
    for (int b = 0; b < B; ++b) {
        if (adapter_of(ids, is64, b, NA) != a) continue;
        if (!any && accumulate) s = *p;
        any = true;
        const int k = (rows_of(lens, b, S) + piece_rows - 1) / piece_rows;
        const float4 *q = reinterpret_cast<const float4 *>(o.part + (long long)b * pieces * size) + i;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const float4 v = __ldcs(q + j * (size / 4));
            s = make_float4(__fadd_rn(s.x, v.x), __fadd_rn(s.y, v.y), __fadd_rn(s.z, v.z), __fadd_rn(s.w, v.w));
        }
    }
    if (any || !accumulate) *p = s;
}

// --------------------------------------------------------------------------
// launchers
// --------------------------------------------------------------------------
template <typename T>
cudaError_t shrink(const adaln_rows &src, const T *W, const LoraCall &c, int C, float *h, cudaStream_t stream) {
    const T *p = static_cast<const T *>(src.data);
    const dim3 grid(1, c.R / kRB, c.B);
    auto go = [&](auto kern, int ctas) {
        return launch_pdl(kern, dim3(ctas, grid.y, grid.z), dim3(128), 0, stream, p, (long long)src.batch,
                          (long long)src.token, W, c.scale, c.ids, c.ids_are_64, c.lens, h, c.S, C, c.R, c.NA);
    };
    // few tokens a sample: the channels over four warps
    if (c.S == 1) return go(lora_shrink_kernel<T, 1, 4>, 1);
    if (c.S <= 16) return go(lora_shrink_kernel<T, 4, 4>, (c.S + 3) / 4);
    return go(lora_shrink_kernel<T, 4, 1>, (c.S + 15) / 16);
}

template <typename T>
cudaError_t expand(const float *h, const T *W, const LoraCall &c, int C, cudaStream_t stream) {
    constexpr int E = Vec<T>::E;
    const int x = (C / E + 127) / 128;
    auto go = [&](auto kern, int tok) {
        return launch_pdl(kern, dim3(x, (c.S + tok - 1) / tok, c.B), dim3(128), 0, stream, h, W, c.ids, c.ids_are_64,
                          c.lens, static_cast<const T *>(c.base.data), (long long)c.base.batch,
                          (long long)c.base.token, static_cast<T *>(c.out.data), (long long)c.out.batch,
                          (long long)c.out.token, c.S, C, c.R, c.NA);
    };
    if (c.S == 1) return go(lora_expand_kernel<T, 1>, 1);
    return go(lora_expand_kernel<T, 8>, 8);
}

// Pieces in parallel, where their sums are no more than what is read anyway
bool grad_in_parts(int S, int R, int es, int piece) {
    return (long long)((S + piece - 1) / piece) * R * 4 <= (long long)S * es;
}

template <typename T>
cudaError_t grads(const float *h, const float *e, float *part, const LoraCall &c, cudaStream_t stream) {
    const int pieces = (c.S + kGradPiece - 1) / kGradPiece, rb = c.R / kRB;
    GradOperand o0 = {c.x.data, c.x.batch, c.x.token, e, c.dA, part, c.K, c.dA ? (c.K + 511) / 512 : 0};
    GradOperand o1 = {c.d_out.data, c.d_out.batch, c.d_out.token, h, c.dU,
                      part + (long long)c.B * pieces * c.R * c.K, c.N, c.dU ? (c.N + 511) / 512 : 0};
    const unsigned x = (unsigned)((o0.blocks + o1.blocks) * rb);
    if (!grad_in_parts(c.S, c.R, sizeof(T), kGradPiece))
        return launch_pdl(lora_grad_kernel<T, true>, dim3(x, c.NA), dim3(128), 0, stream, o0, o1, c.ids, c.ids_are_64,
                          c.lens, c.accumulate, c.B, c.S, c.R, c.NA, pieces);
    cudaError_t err = launch_pdl(lora_grad_kernel<T, false>, dim3(x, pieces, c.B), dim3(128), 0, stream, o0, o1, c.ids,
                                 c.ids_are_64, c.lens, c.accumulate, c.B, c.S, c.R, c.NA, pieces);
    if (err != cudaSuccess) return err;
    const long long n = (long long)c.R * ((c.dA ? c.K : 0) + (c.dU ? c.N : 0)) / 4;
    return launch_pdl(lora_join_kernel, dim3((unsigned)((n + 127) / 128), c.NA), dim3(128), 0, stream, o0, o1, c.ids,
                      c.ids_are_64, c.lens, c.accumulate, c.B, c.S, c.R, c.NA, pieces, kGradPiece);
}

}  // namespace

size_t lora_state_bytes(int B, int S, int R) { return (size_t)B * R * ((S + 7) / 8 * 8) * 4; }

template <typename T>
size_t lora_bwd_ws_bytes(int B, int S, int K, int N, int R) {
    const size_t pieces = grad_in_parts(S, R, sizeof(T), kGradPiece) ? (S + kGradPiece - 1) / kGradPiece : 0;
    return lora_state_bytes(B, S, R) + (size_t)B * pieces * R * ((size_t)K + N) * 4;
}

template <typename T>
cudaError_t launch_lora_fwd(const LoraCall &c, cudaStream_t stream, const DeviceInfo &) {
    float *h = static_cast<float *>(c.state);
    const cudaError_t err = shrink<T>(c.x, static_cast<const T *>(c.A), c, c.K, h, stream);
    if (err != cudaSuccess) return err;
    return expand<T>(h, static_cast<const T *>(c.U), c, c.N, stream);
}

template <typename T>
cudaError_t launch_lora_bwd(const LoraCall &c, cudaStream_t stream, const DeviceInfo &) {
    const float *h = static_cast<const float *>(c.state);
    float *e = static_cast<float *>(c.ws);
    cudaError_t err = cudaSuccess;
    if (c.dA || c.out.data) err = shrink<T>(c.d_out, static_cast<const T *>(c.U), c, c.N, e, stream);
    if (err == cudaSuccess && c.out.data) err = expand<T>(e, static_cast<const T *>(c.A), c, c.K, stream);
    if (err == cudaSuccess && (c.dA || c.dU) && c.NA > 0)
        err = grads<T>(h, e, e + lora_state_bytes(c.B, c.S, c.R) / 4, c, stream);
    return err;
}

#define ADALN_LORA(T)                                                                                                  \
    template size_t lora_bwd_ws_bytes<T>(int, int, int, int, int);                                                     \
    template cudaError_t launch_lora_fwd<T>(const LoraCall &, cudaStream_t, const DeviceInfo &);                       \
    template cudaError_t launch_lora_bwd<T>(const LoraCall &, cudaStream_t, const DeviceInfo &);
ADALN_LORA(uint16_t)
ADALN_LORA(float)

}  // namespace adaln
