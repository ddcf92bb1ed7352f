// Low-rank adapters, one for each sample, beside a shared projection
// (include/adaln_tune.h): forward, and the gradients.
//
// With W = A or U, [NA, R, C] in both directions, three products make up a call:
//     shrink   h[b,s,:] = scale_a W_a src[b,s,:]           (x with A; d_out with U)
//     expand   out[b,s,:] = base[b,s,:] + h[b,s,:] W_a     (h with U; e with A)
//     grad     dW_a = sum over rows of h[b,s,:] src[b,s,:]^T
// 2 R flop for each channel read or written: bf16 on the tensor cores where a sample
// has work for them (lora_tc.cu); here on the CUDA cores, fp32 and samples of a few
// tokens.  These calls are small, and a chain of latencies more than anything else:
// what a kernel can read before the one it follows has ended, it does.  Cold, at 257
// samples of a token, 3072 and 6144 channels, 4 adapters of rank 16: shrink 11 and 16 us,
// expand 9 and 7, the gradients 17 to 20; at 64 samples replayed from a graph 7.0 for
// both kernels of the forward.
#include "lora.cuh"

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
    __device__ __forceinline__ void load_l2(const uint16_t *p) { v = __ldcg(reinterpret_cast<const uint4 *>(p)); }
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
    __device__ __forceinline__ void load_l2(const float *p) { v = __ldcg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void pairs(px2 (&x)[2]) const {
        x[0] = px_make(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = px_make(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const px2 (&x)[2]) {
        return make_uint4(__float_as_uint(px_lo(x[0])), __float_as_uint(px_hi(x[0])), __float_as_uint(px_lo(x[1])),
                          __float_as_uint(px_hi(x[1])));
    }
};

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
// shrink: the CTA's KS warps, the channels split among them, form kRB ranks of TOK
// tokens of a sample.  A lane takes the 16-byte
// vectors of its share in ascending order (NV of them requested at once), even and
// odd channels in the halves of a packed accumulator; halves, butterfly, warps
// ascending.  State fp32 [B,S,R].
// --------------------------------------------------------------------------
template <typename T, int TOK, int KS, int NV>
__global__ void __launch_bounds__(KS * 32)
lora_shrink_kernel(const T *__restrict__ src, long long batch, long long token, const T *__restrict__ W,
                   const float *__restrict__ scale, const void *ids, int is64, const int *lens,
                   float *__restrict__ h, int S, int C, int R, int NA) {
    constexpr int E = Vec<T>::E, V = TOK * kRB, kStep = KS * 32;
    __shared__ float part[KS][V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, r0 = blockIdx.y * kRB;
    const int s0 = blockIdx.x * TOK;
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
        for (int v0 = threadIdx.x; v0 < C / E; v0 += NV * kStep) {
            Vec<T> xv[NV][TOK], wv[NV][kRB];
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const long long at = (long long)(v0 + u * kStep) * E;
                const bool in = v0 + u * kStep < C / E;
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    xv[u][i].zero();
                    if (in && i < n) xv[u][i].load(x + i * token + at);
                }
#pragma unroll
                for (int r = 0; r < kRB; ++r) {
                    wv[u][r].zero();
                    if (in) wv[u][r].load(w + (long long)r * C + at);
                }
            }
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                px2 xp[TOK][E / 2];
#pragma unroll
                for (int i = 0; i < TOK; ++i) xv[u][i].pairs(xp[i]);
#pragma unroll
                for (int r = 0; r < kRB; ++r) {
                    px2 wp[E / 2];
                    wv[u][r].pairs(wp);
#pragma unroll
                    for (int i = 0; i < TOK; ++i)
#pragma unroll
                        for (int q = 0; q < E / 2; ++q) acc[i][r] = px_fma(xp[i][q], wp[q], acc[i][r]);
                }
            }
        }
    }
    float sum[V];
#pragma unroll
    for (int i = 0; i < TOK; ++i)
#pragma unroll
        for (int r = 0; r < kRB; ++r) sum[i * kRB + r] = __fadd_rn(px_lo(acc[i][r]), px_hi(acc[i][r]));
    float mine = scatter_sum<V>(sum, lane);
    if (lane < V) part[warp][lane] = mine;
    __syncthreads();
    if (warp > 0) return;
    if (lane < V)
        for (int k = 1; k < KS; ++k) mine = __fadd_rn(mine, part[k][lane]);
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
    // With adapters this kernel follows shrink, which waited for all that came before:
    // only the state is not there yet.
    if (NA == 0) pdl_wait();
    const int n = min(TOK, rows_of<true>(lens, b, S) - s0);
    const int a = adapter_of<true>(ids, is64, b, NA);
    const T *w = W + (long long)max(a, 0) * R * C + c0;
    Vec<T> y[TOK], wv[kRB];
#pragma unroll
    for (int r = 0; r < kRB; ++r) {
        wv[r].zero();
        if (a >= 0 && c0 < C) wv[r].load_l2(w + (long long)r * C);
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
        y[i].zero();
        if (base && i < n && c0 < C) y[i].load_l2(base + b * base_batch + (s0 + i) * base_token + c0);
    }
    if (NA > 0) pdl_wait();
    pdl_trigger();
    if (n <= 0 || (a < 0 && base == out)) return;
    if (a >= 0)
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
        for (int r0 = 0; r0 < R; r0 += kRB) {
            if (r0 > 0)
#pragma unroll
                for (int r = 0; r < kRB; ++r) wv[r].load(w + (long long)(r0 + r) * C);
#pragma unroll
            for (int r = 0; r < kRB; ++r) {
                px2 wp[E / 2];
                wv[r].pairs(wp);
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    const px2 hr = px_splat(hs[i][r0 + r]);
#pragma unroll
                    for (int q = 0; q < E / 2; ++q) acc[i][q] = px_fma(hr, wp[q], acc[i][q]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
        if (i >= n) break;
        uint4 o = y[i].v;  // without an adapter the base as it is (a zero added would lose the sign of -0)
        if (a >= 0) {
            px2 yp[E / 2];
            y[i].pairs(yp);
#pragma unroll
            for (int q = 0; q < E / 2; ++q) acc[i][q] = px_add(yp[q], acc[i][q]);
            o = Vec<T>::pack(acc[i]);
        }
        stg16(out + b * batch + (s0 + i) * token + c0, o);
    }
}

// --------------------------------------------------------------------------
// grad: a lane holds 4 channels of kRB ranks.  A piece is kGradPiece consecutive
// rows of a sample, summed by fused multiply-adds, ascending, from +0; the pieces
// are added in ascending order, sample by sample.
//
// Two schedules, chosen by S, R and the type.  lora_grad_parts_kernel: a CTA takes
// one piece (a warp its rows s mod 4 == w, kFlight of them requested at once; the
// four sums are added in order of w) and writes its sum to the workspace, and
// lora_join_kernel adds them: as many CTAs as there are pieces, and R fp32 for each
// channel of a piece moved twice.  lora_grad_owner_kernel: a thread takes every
// piece of an adapter and writes the accumulator.
// --------------------------------------------------------------------------
constexpr int kFlight = 16;  // rows of a warp requested at once (5 x 333 rows, fp32: 14 us; 8 rows 17)

template <typename T>
struct Four;  // 4 channels of a row
template <>
struct Four<uint16_t> {
    uint2 v;
    __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
    __device__ __forceinline__ void load(const uint16_t *p) { v = __ldcg(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void pairs(px2 (&x)[2]) const { x[0] = px_bf16(v.x), x[1] = px_bf16(v.y); }
};
template <>
struct Four<float> {
    float4 v;
    __device__ __forceinline__ void zero() { v = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void load(const float *p) { v = __ldcg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void pairs(px2 (&x)[2]) const { x[0] = px_make(v.x, v.y), x[1] = px_make(v.z, v.w); }
};

// NR ranks of 4 channels
template <int NR>
using RankAcc = px2[NR][2];
template <int NR>
__device__ __forceinline__ void zero_acc(RankAcc<NR> &a) {
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r][0] = a[r][1] = 0ull;
}
template <int NR>
__device__ __forceinline__ void add_acc(RankAcc<NR> &a, const RankAcc<NR> &b) {
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r][0] = px_add(a[r][0], b[r][0]), a[r][1] = px_add(a[r][1], b[r][1]);
}
// a row's products: x of 4 channels, h of NR ranks in shared memory
template <int NR, typename T>
__device__ __forceinline__ void add_row(RankAcc<NR> &a, const Four<T> &x, const float *h) {
    px2 xp[2];
    x.pairs(xp);
#pragma unroll
    for (int r4 = 0; r4 < NR; r4 += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(h + r4);
        const float hr[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const px2 e = px_splat(hr[r]);
            a[r4 + r][0] = px_fma(e, xp[0], a[r4 + r][0]);
            a[r4 + r][1] = px_fma(e, xp[1], a[r4 + r][1]);
        }
    }
}
template <int NR>
__device__ __forceinline__ float4 of_acc(const RankAcc<NR> &a, int r) {
    return make_float4(px_lo(a[r][0]), px_hi(a[r][0]), px_lo(a[r][1]), px_hi(a[r][1]));
}

// the operand, rank block and first channel of a CTA; rb blocks of `ranks` ranks, blocks of `width` channels
__device__ __forceinline__ const GradOperand &grad_place(const GradOperand &o0, const GradOperand &o1, int ranks, int rb,
                                                         int width, int &r0, int &c0) {
    const bool first = (int)blockIdx.x < o0.blocks * rb;
    const GradOperand &o = first ? o0 : o1;
    const int at = first ? blockIdx.x : blockIdx.x - o0.blocks * rb;
    r0 = at / o.blocks * ranks, c0 = at % o.blocks * width;
    return o;
}

template <typename T>
__global__ void __launch_bounds__(128)
lora_grad_parts_kernel(const GradOperand o0, const GradOperand o1, const void *ids, int is64, const int *lens, int early,
                       int S, int R, int NA, int pieces) {
    __shared__ __align__(16) float hs[kGradPiece][kRB];
    __shared__ float4 sums[3][kRB][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int r0, c0;
    const GradOperand &o = grad_place(o0, o1, kRB, R / kRB, 128, r0, c0);
    c0 += lane * 4;
    if (!early) pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z, s0 = blockIdx.y * kGradPiece;
    const int n = min(rows_of<true>(lens, b, S) - s0, kGradPiece);
    if (n <= 0 || adapter_of<true>(ids, is64, b, NA) < 0) {
        pdl_wait();
        return;
    }
    const float *h = o.h + ((long long)b * S + s0) * R + r0;
    for (int i = threadIdx.x; i < n * 2; i += 128)
        *reinterpret_cast<float4 *>(&hs[i >> 1][(i & 1) * 4]) =
            __ldcg(reinterpret_cast<const float4 *>(h + (long long)(i >> 1) * R + (i & 1) * 4));
    __syncthreads();
    RankAcc<kRB> acc;
    zero_acc<kRB>(acc);
    if (c0 < o.C) {
        const T *x = static_cast<const T *>(o.src) + b * o.batch + s0 * o.token + c0;
        for (int s = warp; s < n; s += 4 * kFlight) {
            Four<T> v[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k)
                if (s + 4 * k < n) v[k].load(x + (s + 4 * k) * o.token);
#pragma unroll
            for (int k = 0; k < kFlight; ++k)
                if (s + 4 * k < n) add_row<kRB>(acc, v[k], hs[s + 4 * k]);
        }
    }
    if (warp > 0)
#pragma unroll
        for (int r = 0; r < kRB; ++r) sums[warp - 1][r][lane] = of_acc<kRB>(acc, r);
    pdl_wait();  // in every CTA: the next kernel takes this one's end for that of all before it
    __syncthreads();
    if (warp > 0 || c0 >= o.C) return;
    float *p = o.part + (((long long)b * pieces + blockIdx.y) * R + r0) * o.C + c0;
#pragma unroll
    for (int r = 0; r < kRB; ++r) {
        float4 v = of_acc<kRB>(acc, r);
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            const float4 u = sums[w][r][lane];
            v = make_float4(__fadd_rn(v.x, u.x), __fadd_rn(v.y, u.y), __fadd_rn(v.z, u.z), __fadd_rn(v.w, u.w));
        }
        stg16f(p + (long long)r * o.C, v);
    }
}

// The rows of the adapter's samples, S for each, as one sequence: 1024 samples are
// looked through at a time, h of 128 rows goes through shared memory, and FLIGHT rows
// of x are requested at once, of one sample or of several.  A thread holds 4 ranks: few
// samples of an adapter make a chain of latencies, which more warps hide (257 samples of
// one token, 4 adapters of rank 16, 3072 and 6144 channels: 54 us with one row requested
// after the other, 30 with 8 rows and 8 ranks, 23 with 16 and 4.  A whole backward there,
// and of 32 samples of 8 tokens: 28 and 22 us with 16 rows, 31 and 22 with 8, 27 and 26
// with 32.)
constexpr int kWindow = 128;
constexpr int kLook = 1024;
constexpr int kOwnerRanks = 4;  // of a thread
template <typename T, int FLIGHT>
__global__ void __launch_bounds__(128)
lora_grad_owner_kernel(const GradOperand o0, const GradOperand o1, const void *ids, int is64, const int *lens,
                       int early, int accumulate, int B, int S, int R, int NA) {
    __shared__ __align__(16) float hs[kWindow][kOwnerRanks];
    __shared__ int place_b[kWindow], place_s[kWindow];  // sample and row, -1 past its end
    __shared__ int found[kLook], count[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int r0, c0;
    const GradOperand &o = grad_place(o0, o1, kOwnerRanks, R / kOwnerRanks, 512, r0, c0);
    c0 += threadIdx.x * 4;
    const bool live = c0 < o.C;
    if (!early) pdl_wait();
    pdl_trigger();
    const int a = blockIdx.y;
    float *p = o.acc + ((long long)a * R + r0) * o.C + c0;
    const T *src = static_cast<const T *>(o.src) + c0;
    RankAcc<kOwnerRanks> total, acc;
    zero_acc<kOwnerRanks>(total);
    bool any = false, open = false;
    for (int b0 = 0; b0 < B; b0 += kLook) {
        // the samples of adapter a among the next ones, in order; a warp looks through a quarter of them
        unsigned mine[kLook / 128];
        int here = 0;
#pragma unroll
        for (int j = 0; j < kLook / 128; ++j) {
            const int b = b0 + warp * (kLook / 4) + j * 32 + lane;
            mine[j] = __ballot_sync(0xFFFFFFFFu, b < B && adapter_of<true>(ids, is64, b, NA) == a);
            here += __popc(mine[j]);
        }
        if (lane == 0) count[warp] = here;
        __syncthreads();
        int before = 0, samples = 0;
        for (int w = 0; w < 4; ++w) {
            if (w < warp) before += count[w];
            samples += count[w];
        }
#pragma unroll
        for (int j = 0; j < kLook / 128; ++j) {
            if (mine[j] >> lane & 1u)
                found[before + __popc(mine[j] & ((1u << lane) - 1u))] = b0 + warp * (kLook / 4) + j * 32 + lane;
            before += __popc(mine[j]);
        }
        __syncthreads();
        if (samples > 0 && !any) {
            any = true;
            if (accumulate && live)
#pragma unroll
                for (int r = 0; r < kOwnerRanks; ++r) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + (long long)r * o.C));
                    total[r][0] = px_make(v.x, v.y), total[r][1] = px_make(v.z, v.w);
                }
        }
        for (long long i0 = 0; i0 < (long long)samples * S; i0 += kWindow) {
            const int rows = (int)min((long long)kWindow, (long long)samples * S - i0);
            if (threadIdx.x < rows) {
                const int i = threadIdx.x, bb = found[(i0 + i) / S], s = (int)((i0 + i) % S);
                const bool real = s < rows_of<true>(lens, bb, S);
                place_b[i] = bb, place_s[i] = real ? s : -1;
                if (real)
                    *reinterpret_cast<float4 *>(hs[i]) =
                        __ldcg(reinterpret_cast<const float4 *>(o.h + ((long long)bb * S + s) * R + r0));
            }
            __syncthreads();
            if (live)
                for (int i = 0; i < rows; i += FLIGHT) {
                    Four<T> v[FLIGHT];
                    int s[FLIGHT];
#pragma unroll
                    for (int k = 0; k < FLIGHT; ++k) {
                        s[k] = i + k < rows ? place_s[i + k] : -1;
                        if (s[k] >= 0) v[k].load(src + place_b[i + k] * o.batch + s[k] * o.token);
                    }
#pragma unroll
                    for (int k = 0; k < FLIGHT; ++k) {
                        if (s[k] < 0) continue;
                        if (s[k] % kGradPiece == 0) {  // a new piece
                            if (open) add_acc<kOwnerRanks>(total, acc);
                            open = true;
                            zero_acc<kOwnerRanks>(acc);
                        }
                        add_row<kOwnerRanks>(acc, v[k], hs[i + k]);
                    }
                }
            __syncthreads();
        }
    }
    if (open) add_acc<kOwnerRanks>(total, acc);
    pdl_wait();
    if (live && (any || !accumulate))
#pragma unroll
        for (int r = 0; r < kOwnerRanks; ++r) stg16f(p + (long long)r * o.C, of_acc<kOwnerRanks>(total, r));
}

// The pieces' sums onto the accumulators: a thread holds 4 channels of a rank.
__global__ void __launch_bounds__(128)
lora_join_kernel(const GradOperand o0, const GradOperand o1, const void *ids, int is64, const int *lens, int accumulate,
                 int B, int S, int R, int NA, int pieces, int piece_rows) {
    const int n0 = o0.acc ? R * (o0.C / 4) : 0, n1 = o1.acc ? R * (o1.C / 4) : 0;
    int i = blockIdx.x * 128 + threadIdx.x;
    pdl_trigger();
    const bool live = i < n0 + n1;
    const GradOperand &o = i < n0 ? o0 : o1;
    if (i >= n0) i -= n0;
    const int a = blockIdx.y;
    const long long size = (long long)R * o.C;  // of a piece
    float4 *p = reinterpret_cast<float4 *>(o.acc + a * size) + i;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool any = false;
    const int lane = threadIdx.x & 31;
    constexpr int kSide = 8;  // pieces requested at once, of one sample or of several
    const float4 *at[kSide];
    int k = 0;
    auto add = [&] {
        pdl_wait();  // until here only what was there before the call is read
        float4 v[kSide];
#pragma unroll
        for (int j = 0; j < kSide; ++j)
            if (live && j < k) v[j] = __ldcs(at[j]);
#pragma unroll
        for (int j = 0; j < kSide; ++j)
            if (j < k)
                s = make_float4(__fadd_rn(s.x, v[j].x), __fadd_rn(s.y, v[j].y), __fadd_rn(s.z, v[j].z),
                                __fadd_rn(s.w, v[j].w));
        k = 0;
    };
    // sample b's adapter and rows, by a lane each; the next 32 samples' on their way
    auto id_of = [&](int b) { return b < B ? adapter_of<true>(ids, is64, b, NA) : -1; };
    auto n_of = [&](int b) { return b < B ? rows_of<true>(lens, b, S) : 0; };
    int next_id = id_of(lane), next_n = n_of(lane);
    for (int b0 = 0; b0 < B; b0 += 32) {
        unsigned left = __ballot_sync(0xFFFFFFFFu, next_id == a);  // those of adapter a
        const int n = next_n;
        next_id = id_of(b0 + 32 + lane), next_n = n_of(b0 + 32 + lane);
        for (; left; left &= left - 1) {
            const int b = b0 + __ffs(left) - 1;
            const int here = (__shfl_sync(0xFFFFFFFFu, n, b - b0) + piece_rows - 1) / piece_rows;
            if (!any && accumulate && live) s = __ldcg(p);
            any = true;
            const float4 *q = reinterpret_cast<const float4 *>(o.part + (long long)b * pieces * size) + i;
            for (int j = 0; j < here; ++j, q += size / 4) {
#pragma unroll
                for (int m = 0; m < kSide; ++m)
                    if (m == k) at[m] = q;
                if (++k == kSide) add();
            }
        }
    }
    add();
    if (!live) return;
    if (any || !accumulate) *p = s;
}

// --------------------------------------------------------------------------
// launchers
// --------------------------------------------------------------------------
template <typename T>
cudaError_t shrink(const adaln_rows &src, const T *W, const LoraCall &c, int C, float *h, cudaStream_t stream) {
    const T *p = static_cast<const T *>(src.data);
    const dim3 grid(1, c.R / kRB, c.B);
    auto go = [&](auto kern, int ctas, int warps) {
        return launch_pdl(kern, dim3(ctas, grid.y, grid.z), dim3(32 * warps), 0, stream, p, (long long)src.batch,
                          (long long)src.token, W, c.scale, c.ids, c.ids_are_64, c.lens, h, c.S, C, c.R, c.NA);
    };
    // no more tokens a thread than a sample has, here and in expand: those that are not
    // there cost as much (forward of 160 samples of 2 tokens, 3896 and 2496 channels, rank
    // 56: 28.7 us with 4 and 8 tokens, 18.5 with 2; of 70 samples of 4, 3832 and 5072: 21.6
    // with 8 in expand, 16.6 with 4)
    if (c.S == 1) return go(lora_shrink_kernel<T, 1, 4, 3>, 1, 4);
    if (c.S == 2) return go(lora_shrink_kernel<T, 2, 4, 2>, 1, 4);
    return go(lora_shrink_kernel<T, 4, 4, 1>, (c.S + 3) / 4, 4);
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
    if (c.S == 2) return go(lora_expand_kernel<T, 2>, 2);
    if (c.S <= 4) return go(lora_expand_kernel<T, 4>, 4);
    return go(lora_expand_kernel<T, 8>, 8);
}

template <typename T>
bool on_tensor_cores(int S, int R) { return sizeof(T) == 2 && lora_tc(S, R); }

// Pieces in parallel, where their sums are no more than what is read anyway
bool grad_in_parts(int S, int R, int es, int piece) {
    return (long long)((S + piece - 1) / piece) * R * 4 <= (long long)S * es;
}

// rows of a piece
template <typename T>
int piece_rows(int S, int R) { return on_tensor_cores<T>(S, R) ? kLoraTcPiece : kGradPiece; }

template <typename T>
cudaError_t grads(const float *h, const float *e, float *part, const LoraCall &c, cudaStream_t stream,
                  const DeviceInfo &dev) {
    const int rows = piece_rows<T>(c.S, c.R), pieces = (c.S + rows - 1) / rows;
    const bool in_parts = grad_in_parts(c.S, c.R, sizeof(T), rows);
    const int width = in_parts ? 128 : 512;  // channels of a CTA
    GradOperand o0 = {c.x.data, c.x.batch, c.x.token, e, c.dA, part, c.K, c.dA ? (c.K + width - 1) / width : 0};
    GradOperand o1 = {c.d_out.data, c.d_out.batch, c.d_out.token, h, c.dU,
                      part + (long long)c.B * pieces * c.R * c.K, c.N, c.dU ? (c.N + width - 1) / width : 0};
    const unsigned x = (unsigned)((o0.blocks + o1.blocks) * (c.R / (in_parts ? kRB : kOwnerRanks)));
    cudaError_t err;
    if (on_tensor_cores<T>(c.S, c.R))
        err = lora_tc_grads(o0, o1, c, in_parts, stream, dev);
    else if (in_parts)
        err = launch_pdl(lora_grad_parts_kernel<T>, dim3(x, pieces, c.B), dim3(128), 0, stream, o0, o1, c.ids,
                         c.ids_are_64, c.lens, c.grads_early, c.S, c.R, c.NA, pieces);
    else
        err = launch_pdl(lora_grad_owner_kernel<T, sizeof(T) == 2 ? 16 : 8>, dim3(x, c.NA), dim3(128), 0, stream, o0,
                         o1, c.ids, c.ids_are_64, c.lens, c.grads_early, c.accumulate, c.B, c.S, c.R, c.NA);
    if (err != cudaSuccess || !in_parts) return err;
    const long long n = (long long)c.R * ((c.dA ? c.K : 0) + (c.dU ? c.N : 0)) / 4;
    return launch_pdl(lora_join_kernel, dim3((unsigned)((n + 127) / 128), c.NA), dim3(128), 0, stream, o0, o1, c.ids,
                      c.ids_are_64, c.lens, c.accumulate, c.B, c.S, c.R, c.NA, pieces, rows);
}

}  // namespace

// fp32, or three bf16 parts (lora.cuh)
size_t lora_state_bytes(int B, int S, int R) { return (size_t)B * R * ((S + 7) / 8 * 8) * 6; }

template <typename T>
size_t lora_bwd_ws_bytes(int B, int S, int K, int N, int R) {
    const int rows = piece_rows<T>(S, R);
    const size_t pieces = grad_in_parts(S, R, sizeof(T), rows) ? (S + rows - 1) / rows : 0;
    return lora_state_bytes(B, S, R) + (size_t)B * pieces * R * ((size_t)K + N) * 4;
}

template <typename T>
static cudaError_t down(const adaln_rows &src, const void *W, const LoraCall &c, int C, void *h, cudaStream_t stream,
                 const DeviceInfo &dev) {
    if (c.NA == 0) return cudaSuccess;  // nothing reads h
    if (on_tensor_cores<T>(c.S, c.R)) return lora_tc_shrink(src, W, c, C, h, stream, dev);
    return shrink<T>(src, static_cast<const T *>(W), c, C, static_cast<float *>(h), stream);
}
template <typename T>
static cudaError_t up(const void *h, const void *W, const LoraCall &c, int C, cudaStream_t stream,
                      const DeviceInfo &dev) {
    if (on_tensor_cores<T>(c.S, c.R)) return lora_tc_expand(h, W, c, C, stream, dev);
    return expand<T>(static_cast<const float *>(h), static_cast<const T *>(W), c, C, stream);
}

template <typename T>
cudaError_t launch_lora_fwd(const LoraCall &c, cudaStream_t stream, const DeviceInfo &dev) {
    const cudaError_t err = down<T>(c.x, c.A, c, c.K, c.state, stream, dev);
    return err != cudaSuccess ? err : up<T>(c.state, c.U, c, c.N, stream, dev);
}

template <typename T>
cudaError_t launch_lora_bwd(const LoraCall &call, cudaStream_t stream, const DeviceInfo &dev) {
    // Behind expand, which waited for shrink, which waited for all before it, the
    // gradients find both states and their rows ready: they start beside expand's end.
    LoraCall c = call;
    c.grads_early = c.out.data != nullptr;
    const float *h = static_cast<const float *>(c.state);
    float *e = static_cast<float *>(c.ws);
    cudaError_t err = cudaSuccess;
    if (c.dA || c.out.data) err = down<T>(c.d_out, c.U, c, c.N, e, stream, dev);
    if (err == cudaSuccess && c.out.data) err = up<T>(e, c.A, c, c.K, stream, dev);
    if (err == cudaSuccess && (c.dA || c.dU) && c.NA > 0)
        err = grads<T>(h, e, e + lora_state_bytes(c.B, c.S, c.R) / 4, c, stream, dev);
    return err;
}

#define ADALN_LORA(T)                                                                                                  \
    template size_t lora_bwd_ws_bytes<T>(int, int, int, int, int);                                                     \
    template cudaError_t launch_lora_fwd<T>(const LoraCall &, cudaStream_t, const DeviceInfo &);                       \
    template cudaError_t launch_lora_bwd<T>(const LoraCall &, cudaStream_t, const DeviceInfo &);
ADALN_LORA(uint16_t)
ADALN_LORA(float)

}  // namespace adaln
