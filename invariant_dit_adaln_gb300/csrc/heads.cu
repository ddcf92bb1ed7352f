// RMS norm of query and key heads with the position rotation, forward and
// backward (contract: include/adaln_ops.h).
//
// Mathematics, for one head row x of Dh channels with weights w:
//   r = 1 / sqrt(sum x^2 / Dh + eps),  n = x r w,  y = R n
// R turns channel pairs by the angles of the row's position (orthogonal), so
//   g = R^T dy,  h = g w,  dx = r (h - x r^2 (sum h x) / Dh),  dw = sum g x r.
// Neither direction needs anything but its tensors once: the backward forms r
// again from x.
//
// Layout: a row is held by LPR = Dh/8 lanes, rounded up to a power of two (at
// least 4), 8 channels a lane, so both reductions are butterflies inside the
// row's lanes.
// A lane's 8 channels are chosen so that both members of every pair it touches
// are its own: interleaved, channels 8l .. 8l+7; halves, channels 4l .. 4l+3
// and Dr/2 + 4l .. Dr/2 + 4l + 3.  The rotation therefore exchanges nothing
// between lanes, and lane l needs the angles 4l .. 4l+3 in either form.
#include "common.cuh"
#include "ops.h"

namespace adaln {

namespace {

constexpr int kWarps = 4;  // warps of a CTA

struct HeadsArgs {
    const void *x[2], *dy[2];
    void *out[2];
    const void *w[2];
    long long xs[2][3], dys[2][3], os[2][3];  // batch, token, head strides in elements
    const float *cos, *sin;
    const void *pos;
    int pos_is_64;
    int S, H[2], Dh, Dr, P;
    int chunks[2];      // groups of heads of a token: q's, k's
    float eps;
    // forward: the tokens of this launch, of all B * S
    long long token0;
    unsigned ntok;
    // backward
    float *part;        // [B][tiles][2][Dh]
    int tile, tiles;    // tokens of a tile, tiles of a sample
};

__device__ __forceinline__ long long position(const HeadsArgs &a, long long token, int s) {
    if (a.pos == nullptr) return s;
    return a.pos_is_64 ? static_cast<const long long *>(a.pos)[token] : static_cast<const int *>(a.pos)[token];
}

// The 8 channels of a lane: two runs of four, at lo and hi.
struct Slot {
    int lo, hi;
    bool live, turned;
};
template <bool INTER>
__device__ __forceinline__ Slot lane_slot(int l, int Dh, int Dr) {
    Slot s;
    s.live = 8 * l < Dh;
    s.turned = 8 * l < Dr;
    s.lo = (INTER || !s.turned) ? 8 * l : 4 * l;
    s.hi = (INTER || !s.turned) ? 8 * l + 4 : Dr / 2 + 4 * l;
    return s;
}

// A lane's 8 channels as they lie in memory, and their values.  Plain
// (coherent) loads: in place, a row is read by the lanes that write it.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
    uint2 a, b;
};
template <>
struct Raw<float> {
    float4 a, b;
};
template <bool INTER>
__device__ __forceinline__ Raw<uint16_t> load8(const uint16_t *p, const Slot &s) {
    if (INTER) {
        const uint4 t = *reinterpret_cast<const uint4 *>(p + s.lo);
        return {make_uint2(t.x, t.y), make_uint2(t.z, t.w)};
    }
    return {*reinterpret_cast<const uint2 *>(p + s.lo), *reinterpret_cast<const uint2 *>(p + s.hi)};
}
template <bool INTER>
__device__ __forceinline__ Raw<float> load8(const float *p, const Slot &s) {
    return {*reinterpret_cast<const float4 *>(p + s.lo), *reinterpret_cast<const float4 *>(p + s.hi)};
}
__device__ __forceinline__ void clear(Raw<uint16_t> &r) { r.a = r.b = make_uint2(0, 0); }
__device__ __forceinline__ void clear(Raw<float> &r) { r.a = r.b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

// The values as four packed pairs: the first members of the lane's four channel
// pairs in v[0], v[1], the second members in v[2], v[3].  Both rotations then
// are the same arithmetic; an interleaved bf16 word is taken apart as it is
// widened, which costs nothing.
template <bool INTER>
__device__ __forceinline__ void values(px2 (&v)[4], const Raw<uint16_t> &r) {
    if (INTER) {
        v[0] = px_make(bf16lo(r.a.x), bf16lo(r.a.y)), v[1] = px_make(bf16lo(r.b.x), bf16lo(r.b.y));
        v[2] = px_make(bf16hi(r.a.x), bf16hi(r.a.y)), v[3] = px_make(bf16hi(r.b.x), bf16hi(r.b.y));
    } else {
        v[0] = px_bf16(r.a.x), v[1] = px_bf16(r.a.y), v[2] = px_bf16(r.b.x), v[3] = px_bf16(r.b.y);
    }
}
template <bool INTER>
__device__ __forceinline__ void values(px2 (&v)[4], const Raw<float> &r) {
    if (INTER) {
        v[0] = px_make(r.a.x, r.a.z), v[1] = px_make(r.b.x, r.b.z);
        v[2] = px_make(r.a.y, r.a.w), v[3] = px_make(r.b.y, r.b.w);
    } else {
        v[0] = px_make(r.a.x, r.a.y), v[1] = px_make(r.a.z, r.a.w);
        v[2] = px_make(r.b.x, r.b.y), v[3] = px_make(r.b.z, r.b.w);
    }
}
// the column of value i (0 .. 7) of such four pairs
template <bool INTER>
__device__ __forceinline__ int column(int i, const Slot &s) {
    if (INTER) return s.lo + 2 * (i & 3) + (i >> 2);
    return i < 4 ? s.lo + i : s.hi + i - 4;
}
// Streaming stores: the output of a large call does not fit L2 beside its inputs.
template <bool INTER>
__device__ __forceinline__ void store8(uint16_t *p, const px2 (&v)[4], const Slot &s) {
    if (INTER) {
        __stcs(reinterpret_cast<uint4 *>(p + s.lo),
               make_uint4(pack_bf16x2(px_lo(v[0]), px_lo(v[2])), pack_bf16x2(px_hi(v[0]), px_hi(v[2])),
                          pack_bf16x2(px_lo(v[1]), px_lo(v[3])), pack_bf16x2(px_hi(v[1]), px_hi(v[3]))));
    } else {
        __stcs(reinterpret_cast<uint2 *>(p + s.lo), make_uint2(px_to_bf16x2(v[0]), px_to_bf16x2(v[1])));
        __stcs(reinterpret_cast<uint2 *>(p + s.hi), make_uint2(px_to_bf16x2(v[2]), px_to_bf16x2(v[3])));
    }
}
template <bool INTER>
__device__ __forceinline__ void store8(float *p, const px2 (&v)[4], const Slot &s) {
    float4 a, b;
    if (INTER) {
        a = make_float4(px_lo(v[0]), px_lo(v[2]), px_hi(v[0]), px_hi(v[2]));
        b = make_float4(px_lo(v[1]), px_lo(v[3]), px_hi(v[1]), px_hi(v[3]));
    } else {
        a = make_float4(px_lo(v[0]), px_hi(v[0]), px_lo(v[1]), px_hi(v[1]));
        b = make_float4(px_lo(v[2]), px_hi(v[2]), px_lo(v[3]), px_hi(v[3]));
    }
    __stcs(reinterpret_cast<float4 *>(p + s.lo), a);
    __stcs(reinterpret_cast<float4 *>(p + s.hi), b);
}
template <bool INTER, typename T>
__device__ __forceinline__ void store_zero(T *p, const Slot &s) {
    const px2 zero[4] = {0, 0, 0, 0};
    store8<INTER>(p, zero, s);
}

// the lane's weights (1 without weights, and in idle lanes)
template <typename T, bool INTER>
__device__ __forceinline__ void load_weights(px2 (&w)[4], const void *p, const Slot &s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = px_splat(1.0f);
    if (s.live && p != nullptr) values<INTER>(w, load8<INTER>(static_cast<const T *>(p), s));
}

// The lane's four angles: cosines and sines, from 16-byte aligned places.
struct Angles {
    px2 c[2], s[2];
};
__device__ __forceinline__ Angles make_angles(const float4 &c, const float4 &s) {
    return {{px_make(c.x, c.y), px_make(c.z, c.w)}, {px_make(s.x, s.y), px_make(s.z, s.w)}};
}
// Turn the lane's pairs by its angles (BACK: by the negative angles).
template <bool BACK>
__device__ __forceinline__ void turn(px2 (&v)[4], const Angles &t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const px2 a = v[i], b = v[2 + i];
        const px2 as = px_mul(a, t.s[i]), bs = px_mul(b, t.s[i]);
        v[i] = BACK ? px_fma(a, t.c[i], bs) : px_sub(px_mul(a, t.c[i]), bs);
        v[2 + i] = BACK ? px_sub(px_mul(b, t.c[i]), as) : px_fma(b, t.c[i], as);
    }
}

// sum over the lane's 8 values of a b
__device__ __forceinline__ float dot8(const px2 (&a)[4], const px2 (&b)[4]) {
    const px2 t = px_fma(a[3], b[3], px_fma(a[2], b[2], px_fma(a[1], b[1], px_mul(a[0], b[0]))));
    return __fadd_rn(px_lo(t), px_hi(t));
}
// sum over a row's lanes
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// --------------------------------------------------------------------------
// Forward: a warp takes U * 32/LPR heads of one token, so the token's angles
// are loaded once for them, and all their loads are in flight together.
// --------------------------------------------------------------------------
template <typename T, int LPR, int U, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) heads_fwd_kernel(const __grid_constant__ HeadsArgs a) {
    constexpr int RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const Slot slot = lane_slot<INTER>(l, a.Dh, a.Dr);
    const unsigned nchunk = a.chunks[0] + a.chunks[1];
    const unsigned task = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const unsigned tk = task / nchunk;
    int chunk = (int)(task - tk * nchunk);
    const int t = chunk >= a.chunks[0];
    if (t) chunk -= a.chunks[0];
    const long long token = a.token0 + tk;
    const long long b = (token >> 32) ? token / a.S : (unsigned)token / (unsigned)a.S;
    const int s = (int)(token - b * a.S);
    const int h0 = chunk * (U * RPW) + sub;
    const long long xstep = RPW * a.xs[t][2], ostep = RPW * a.os[t][2];
    const T *x = static_cast<const T *>(a.x[t]) + b * a.xs[t][0] + s * a.xs[t][1] + h0 * a.xs[t][2];
    T *o = static_cast<T *>(a.out[t]) + b * a.os[t][0] + s * a.os[t][1] + h0 * a.os[t][2];
    const int rows = slot.live ? (a.H[t] - h0 + RPW - 1) / RPW : 0;  // the lane's heads: u < rows
    pdl_wait();
    pdl_trigger();
    if (tk >= a.ntok) return;
    const long long p = position(a, token, s);
    Raw<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        clear(raw[u]);
        if (u < rows) raw[u] = load8<INTER>(x + u * xstep, slot);
    }
    px2 w[4];
    load_weights<T, INTER>(w, a.w[t], slot);
    if (p < 0 || p >= a.P) {  // padding
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < rows) store_zero<INTER>(o + u * ostep, slot);
        return;
    }
    Angles ang = {};
    if (slot.turned) {
        const long long at = p * (a.Dr / 2) + 4 * l;
        ang = make_angles(__ldg(reinterpret_cast<const float4 *>(a.cos + at)),
                          __ldg(reinterpret_cast<const float4 *>(a.sin + at)));
    }
    const float inv = __fdiv_rn(1.0f, (float)a.Dh);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        px2 v[4];
        values<INTER>(v, raw[u]);
        const float ss = row_sum<LPR>(dot8(v, v));
        const px2 r = px_splat(rsqrtf(__fmaf_rn(ss, inv, a.eps)));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = px_mul(px_mul(v[i], r), w[i]);
        if (slot.turned) turn<false>(v, ang);
        if (u < rows) store8<INTER>(o + u * ostep, v, slot);
    }
}

// --------------------------------------------------------------------------
// Tiles: one CTA per (tile of tokens, q or k, sample), for the backward and for
// large forward calls.  Each warp takes an equal share of the tile's (token,
// U * 32/LPR heads) tasks, in order, and copies their rows asynchronously into
// a ring of kStages tasks of its own, so that the bytes in flight are not held
// in registers.  Padded rows are copied too.  A token's angles travel with its tasks; its position is read
// one token ahead.
//
// Measured at B=2, S=4096, 24 + 24 heads of 128 in bf16, back to back: forward
// 34.1 us (203 MB, 6.0 TB/s), backward 57.1 us with the join of dw (304 MB, 5.3
// TB/s).  With the rows in registers the backward was bound by load latency at
// 18 warps an SM: 70 us.  2 and 4 rows a lane and 3 or 4 stages differ by 2 %;
// any register spilled in the loop costs 10 us, hence the launch bounds.
//
// Backward: each lane keeps the dw sums of its 8 channels, joined over the CTA
// in a fixed order into the tile's partial.
// --------------------------------------------------------------------------
constexpr int kStages = 3;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros without reading
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The rows of one task of one tensor: the lane's 8 channels of rows src, src +
// step, ... to dst, dst + (a warp's rows), ...; `all`: every lane has all U of them,
// otherwise u < rows.  A row that a lane does not have lies behind the heads: its
// zeros name `base`, an address of the tensor, as their source.
template <typename T, int U>
__device__ __forceinline__ void copy_rows(uint32_t dst, const T *src, const T *base, long long step, bool all,
                                          int rows) {
    constexpr int E = 16 / (int)sizeof(T);
    if (all) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < 8 / E; ++j)
                cp_async16(dst + u * 256 * (int)sizeof(T) + 16 * j, src + u * step + E * j);
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < 8 / E; ++j)
                cp_async16_if(dst + u * 256 * (int)sizeof(T) + 16 * j, u < rows ? src + u * step + E * j : base,
                              u < rows);
        }
    }
}

// A stage of the ring: the task's rows of x (and dy), then its token's cosines
// and sines, 4 LPR floats each; in bytes.
template <typename T, int LPR, int U, bool BWD>
struct Stage {
    static constexpr int kRows = U * 256 * (int)sizeof(T);
    static constexpr int kAngles = (BWD ? 2 : 1) * kRows;
    static constexpr int kBytes = kAngles + 32 * LPR;
    static constexpr size_t kSmem = (size_t)kWarps * kStages * kBytes;
};

template <typename T, int LPR, int U, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? (BWD ? (LPR == 32 ? 4 : 5) : 7) : 4)
heads_tile_kernel(const __grid_constant__ HeadsArgs a) {
    using St = Stage<T, LPR, U, BWD>;
    constexpr int RPW = 32 / LPR;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
    const Slot slot = lane_slot<INTER>(l, a.Dh, a.Dr);
    const int t = blockIdx.y;
    const int nchunk = a.chunks[t];
    if (nchunk == 0) return;  // no keys
    unsigned char *ring = ring_bytes + warp * (kStages * St::kBytes);
    const int s0 = blockIdx.x * a.tile;
    const int ntask = min(a.tile, a.S - s0) * nchunk;
    const long long b = blockIdx.z;
    const int first = ntask * warp / kWarps, end = ntask * (warp + 1) / kWarps;
    const int heads = slot.live ? (a.H[t] - sub + RPW - 1) / RPW : 0;  // the lane's heads of a token
    px2 dw[4] = {0, 0, 0, 0};
    pdl_wait();
    pdl_trigger();
    if (first < end) {
        const float inv = __fdiv_rn(1.0f, (float)a.Dh);
        const int last = s0 + (end - 1) / nchunk;  // the warp's last token
        // a token's position, or -1: padding
        const auto where = [&](int s) {
            const long long p = position(a, b * a.S + s, s);
            return p >= 0 && p < a.P ? (int)p : -1;
        };
        // Copies run kStages - 1 tasks ahead, at chunk cc of token cs; its position
        // is known one token before.  Pointers advance by a chunk, and by what is
        // left of the token's stride behind its last chunk.
        int cs = s0 + first / nchunk, cc = first % nchunk, chunk = cc, todo = end - first;
        const int whole = (8 * LPR == a.Dh) ? a.H[t] / (U * RPW) : 0;  // chunks with a row for every lane
        const long long xrow = RPW * a.xs[t][2], grow = RPW * a.dys[t][2], orow = RPW * a.os[t][2];
        const long long xwrap = a.xs[t][1] - nchunk * U * xrow, gwrap = a.dys[t][1] - nchunk * U * grow,
                        owrap = a.os[t][1] - nchunk * U * orow;
        const T *xsrc = static_cast<const T *>(a.x[t]) + b * a.xs[t][0] + cs * a.xs[t][1] + cc * U * xrow +
                        sub * a.xs[t][2] + 8 * l;
        const T *gsrc = nullptr;
        if (BWD)
            gsrc = static_cast<const T *>(a.dy[t]) + b * a.dys[t][0] + cs * a.dys[t][1] + cc * U * grow +
                   sub * a.dys[t][2] + 8 * l;
        T *o = static_cast<T *>(a.out[t]) + b * a.os[t][0] + cs * a.os[t][1] + cc * U * orow + sub * a.os[t][2];
        int p = where(cs), p_next = where(min(cs + 1, last));
        unsigned real = 0;  // bit i: stage i holds a real token's task
        const uint32_t lane_dst = smem_u32(ring) + lane * 8 * (int)sizeof(T);
        const uint32_t angle_dst = smem_u32(ring) + St::kAngles + 16 * l;
        const auto copy_next = [&](int stage, bool more) {
            if (more) {
                const int rows = heads - cc * U;  // the lane's heads: u < rows
                const uint32_t dst = lane_dst + stage * St::kBytes;
                const bool all = cc < whole;
                copy_rows<T, U>(dst, xsrc, static_cast<const T *>(a.x[t]), xrow, all, rows);
                if (BWD) copy_rows<T, U>(dst + St::kRows, gsrc, static_cast<const T *>(a.dy[t]), grow, all, rows);
                if (sub == 0 && slot.turned && p >= 0) {
                    const long long at = (long long)p * (a.Dr / 2) + 4 * l;
                    cp_async16(angle_dst + stage * St::kBytes, a.cos + at);
                    cp_async16(angle_dst + stage * St::kBytes + 16 * LPR, a.sin + at);
                }
                real = p >= 0 ? real | 1u << stage : real & ~(1u << stage);
                xsrc += U * xrow;
                if (BWD) gsrc += U * grow;
                if (++cc == nchunk) {
                    cc = 0, ++cs;
                    xsrc += xwrap;
                    if (BWD) gsrc += gwrap;
                    p = p_next;
                    if (cs < last) p_next = where(cs + 1);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy_next(i, i < todo);
        px2 w[4];
        load_weights<T, INTER>(w, a.w[t], slot);
        int stage = 0;
#pragma unroll 1
        for (; todo > 0; --todo) {
            cp_async_wait<kStages - 2>();
            __syncwarp();  // the stage is whole, and every lane has read the one before it
            copy_next(stage == 0 ? kStages - 1 : stage - 1, todo > kStages - 1);
            const unsigned char *at = ring + stage * St::kBytes;
            const bool known = real >> stage & 1u;
            if (++stage == kStages) stage = 0;
            const int rows = heads - chunk * U;
            if (known) {
                const Angles ang = make_angles(*reinterpret_cast<const float4 *>(at + St::kAngles + 16 * l),
                                               *reinterpret_cast<const float4 *>(at + St::kAngles + 16 * (LPR + l)));
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const T *row = reinterpret_cast<const T *>(at) + (u * RPW + sub) * LPR * 8;
                    px2 v[4];
                    values<INTER>(v, load8<INTER>(row, slot));
                    const float ss = row_sum<LPR>(dot8(v, v));
                    if (BWD) {
                        px2 g[4], gx[4];
                        values<INTER>(g, load8<INTER>(row + St::kRows / (int)sizeof(T), slot));
                        if (slot.turned) turn<true>(g, ang);
#pragma unroll
                        for (int i = 0; i < 4; ++i) gx[i] = px_mul(g[i], v[i]);
                        const float hx = row_sum<LPR>(dot8(gx, w));
                        // lanes without a row: 0, where r would be infinite at eps = 0
                        const float r = u < rows ? rsqrtf(__fmaf_rn(ss, inv, a.eps)) : 0.0f;
                        const px2 rr = px_splat(r);
                        const px2 k = px_splat(-__fmul_rn(__fmul_rn(__fmul_rn(r, r), inv), hx));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            dw[i] = px_fma(gx[i], rr, dw[i]);
                            v[i] = px_mul(px_fma(v[i], k, px_mul(g[i], w[i])), rr);
                        }
                    } else {
                        const px2 r = px_splat(rsqrtf(__fmaf_rn(ss, inv, a.eps)));
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = px_mul(px_mul(v[i], r), w[i]);
                        if (slot.turned) turn<false>(v, ang);
                    }
                    if (u < rows) store8<INTER>(o + u * orow, v, slot);
                }
            } else {  // padding
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < rows) store_zero<INTER>(o + u * orow, slot);
            }
            o += U * orow;
            if (++chunk == nchunk) chunk = 0, o += owrap;
        }
        cp_async_wait<0>();
    }
    if (!BWD || a.part == nullptr) return;
    __syncthreads();  // the rings are free
    float(*red)[LPR * 8] = reinterpret_cast<float(*)[LPR * 8]>(ring_bytes);
    // the warp's row groups, then the warps in ascending order
    float sums[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[2 * i] = px_lo(dw[i]), sums[2 * i + 1] = px_hi(dw[i]);
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[i] = __fadd_rn(sums[i], __shfl_xor_sync(0xFFFFFFFFu, sums[i], off));
    }
    if (sub == 0 && slot.live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[warp][column<INTER>(i, slot)] = sums[i];
    }
    __syncthreads();
    float *part = a.part + ((b * a.tiles + blockIdx.x) * 2 + t) * a.Dh;
    for (int d = threadIdx.x; d < a.Dh; d += 32 * kWarps) {
        float sum = red[0][d];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) sum = __fadd_rn(sum, red[i][d]);
        part[d] = sum;
    }
}

// --------------------------------------------------------------------------
// dw of a sample: its tiles' partials.  A CTA takes 8 columns (one 32-byte
// sector of a partial) and 128 groups of tiles: group g adds the tiles g, g +
// 128, ... in order, then the groups are joined by a fixed tree.  The order
// is fixed by the number of tiles, that is by S, H, Dh.
//   DIRECT: a CTA takes all samples (at most kDirectSamples) and adds them onto
//   the accumulator itself, which saves a launch; otherwise blockIdx.z is the
//   sample and its sum goes to sums [B][2][Dh].
// --------------------------------------------------------------------------
constexpr int kDirectSamples = 6;

struct FoldArgs {
    const float *part;
    float *sums;
    float *dw[2];
    int B, tiles, Dh, accumulate;
};

template <bool DIRECT>
__global__ void __launch_bounds__(1024) heads_fold_kernel(const FoldArgs a) {
    constexpr int NB = DIRECT ? kDirectSamples : 1;
    __shared__ float red[NB][32][8];
    __shared__ float sums[NB][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane & 7, grp = threadIdx.x >> 3;
    const int t = blockIdx.y, d = blockIdx.x * 8 + col;
    const long long b0 = DIRECT ? 0 : blockIdx.z;
    const int nb = DIRECT ? a.B : 1;
    float *dw = a.dw[t];
    pdl_wait();
    pdl_trigger();
    if (dw == nullptr) return;
    const long long sample = (long long)a.tiles * 2 * a.Dh;
    const float *p = a.part + b0 * sample + t * a.Dh + d;
    float sum[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) sum[k] = 0.0f;
    for (int i0 = grp; i0 < a.tiles; i0 += 2 * 128) {
        float v[NB][2];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = i0 + j * 128;
                v[k][j] = 0.0f;  // +0 behind the end: adding it changes no sum begun from +0
                if (k < nb && i < a.tiles) v[k][j] = __ldcg(p + k * sample + (long long)i * 2 * a.Dh);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int k = 0; k < NB; ++k) sum[k] = __fadd_rn(sum[k], v[k][j]);
        }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        sum[k] = __fadd_rn(sum[k], __shfl_xor_sync(0xFFFFFFFFu, sum[k], 8));
        sum[k] = __fadd_rn(sum[k], __shfl_xor_sync(0xFFFFFFFFu, sum[k], 16));
        if (lane < 8) red[k][warp][col] = sum[k];
    }
    __syncthreads();
    if (warp < NB) {  // warp k joins the 32 warps' sums of sample k, 8 to a quarter
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v = __fadd_rn(v, red[warp][(lane >> 3) * 8 + i][col]);
        v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
        v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
        if (lane < 8) sums[warp][col] = v;
    }
    if (DIRECT) __syncthreads();
    if (threadIdx.x >= 8) return;
    if (DIRECT) {
        float acc = a.accumulate ? dw[d] : 0.0f;
#pragma unroll
        for (int k = 0; k < NB; ++k)
            if (k < nb) acc = __fadd_rn(acc, sums[k][col]);
        dw[d] = acc;
    } else {
        a.sums[(b0 * 2 + t) * a.Dh + d] = sums[0][col];
    }
}

// the samples' sums onto the accumulators, in ascending order
__global__ void __launch_bounds__(256) heads_samples_kernel(const FoldArgs a) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (i >= 2 * a.Dh) return;
    float *dw = a.dw[i / a.Dh];
    if (dw == nullptr) return;
    float acc = a.accumulate ? dw[i % a.Dh] : 0.0f;
#pragma unroll 16
    for (long long b = 0; b < a.B; ++b) acc = __fadd_rn(acc, __ldcg(a.sums + b * 2 * a.Dh + i));
    dw[i % a.Dh] = acc;
}

int lanes_per_row(int Dh) {
    int l = 4;  // smaller rows leave lanes idle
    while (8 * l < Dh) l *= 2;
    return l;
}

HeadsArgs make_args(const HeadsCall &c, int group) {
    HeadsArgs a = {};
    for (int t = 0; t < 2; ++t) {
        a.x[t] = c.x[t].data;
        a.dy[t] = c.dy[t].data;
        a.out[t] = c.out[t].data;
        a.w[t] = c.w[t];
        a.H[t] = c.H[t];
        a.chunks[t] = (c.H[t] + group - 1) / group;
        const adaln_heads *h[3] = {&c.x[t], &c.dy[t], &c.out[t]};
        long long *s[3] = {a.xs[t], a.dys[t], a.os[t]};
        for (int i = 0; i < 3; ++i) {
            s[i][0] = h[i]->batch;
            s[i][1] = h[i]->token;
            s[i][2] = h[i]->head;
        }
    }
    a.cos = c.cos;
    a.sin = c.sin;
    a.pos = c.pos;
    a.pos_is_64 = c.pos_is_64;
    a.S = c.S;
    a.Dh = c.Dh;
    a.Dr = c.Dr;
    // without positions and without a rotation every row is real
    a.P = (c.pos == nullptr && c.Dr == 0) ? 0x7FFFFFFF : c.P;
    a.eps = c.eps;
    return a;
}

// rows a lane in a tile's task: 2 where a token has heads for them
int tile_rows(int Hq, int Hk, int Dh) {
    const int h = Hq > Hk ? Hq : Hk;
    return h > 32 / lanes_per_row(Dh) ? 2 : 1;
}

// Tokens of a tile with about `tasks` tasks; fewer where a sample has few, so
// that it still spreads over the SMs.
int tile_tokens(int tasks, int S, int Hq, int Hk, int Dh) {
    const int group = tile_rows(Hq, Hk, Dh) * (32 / lanes_per_row(Dh)), h = Hq > Hk ? Hq : Hk;
    const int chunks = (h + group - 1) / group;
    const int most = chunks >= tasks ? 1 : tasks / chunks, spread = S < 64 ? 1 : S / 64;
    return most < spread ? most : spread;
}
// Backward: 48 tasks a CTA, 12 a warp, fill the ring and pay for joining dw (24:
// 4 us more, 96: 5 us more at the size above).  It is fixed by S, the head
// counts and the head size, and with it the order of dw.
int bwd_tile(int S, int Hq, int Hk, int Dh) { return tile_tokens(48, S, Hq, Hk, Dh); }
// Forward: 24, for a finer tail (fp32, 4593 tokens of 20 + 4 heads of 96: 14.6 us
// from a graph against 15.8 with 48).
int fwd_tile(int S, int Hq, int Hk, int Dh) { return tile_tokens(24, S, Hq, Hk, Dh); }

template <typename T, int LPR, int U, bool INTER, bool BWD>
cudaError_t run_tile(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev) {
    HeadsArgs a = make_args(c, U * (32 / LPR));
    a.tile = (BWD ? bwd_tile : fwd_tile)(c.S, c.H[0], c.H[1], c.Dh);
    a.tiles = (c.S + a.tile - 1) / a.tile;
    a.part = BWD && (c.dw[0] || c.dw[1]) ? c.ws : nullptr;
    constexpr size_t smem = Stage<T, LPR, U, BWD>::kSmem;
    const cudaError_t e = ensure_smem_attr((const void *)heads_tile_kernel<T, LPR, U, INTER, BWD>, smem, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(heads_tile_kernel<T, LPR, U, INTER, BWD>, dim3(a.tiles, 2, c.B), dim3(32 * kWarps), smem, stream,
                      a);
}
template <typename T, int LPR, bool BWD>
cudaError_t pick_tile(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev) {
    if (tile_rows(c.H[0], c.H[1], c.Dh) == 2)
        return c.interleaved ? run_tile<T, LPR, 2, true, BWD>(c, stream, dev)
                             : run_tile<T, LPR, 2, false, BWD>(c, stream, dev);
    return c.interleaved ? run_tile<T, LPR, 1, true, BWD>(c, stream, dev)
                         : run_tile<T, LPR, 1, false, BWD>(c, stream, dev);
}

template <typename T, int LPR, int U>
cudaError_t run_direct(const HeadsCall &c, cudaStream_t stream) {
    HeadsArgs a = make_args(c, U * (32 / LPR));
    // tasks of a launch are counted in 31 bits
    const long long tokens = (long long)c.B * c.S, nchunk = a.chunks[0] + a.chunks[1];
    const long long most = 0x7FFFFFFFll / nchunk;
    for (; a.token0 < tokens; a.token0 += a.ntok) {
        a.ntok = (unsigned)(tokens - a.token0 < most ? tokens - a.token0 : most);
        const dim3 grid((unsigned)((a.ntok * nchunk + kWarps - 1) / kWarps)), block(32 * kWarps);
        const cudaError_t e = c.interleaved ? launch_pdl(heads_fwd_kernel<T, LPR, U, true>, grid, block, 0, stream, a)
                                            : launch_pdl(heads_fwd_kernel<T, LPR, U, false>, grid, block, 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int LPR>
cudaError_t pick_fwd(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev) {
    // Few rows go one a lane straight through registers, for the shortest path
    // through the kernel (8 tokens of 24 + 24 heads: 3.6 us of kernel); from 16
    // warps an SM on 4 a lane, or through the ring where a tile has 4 tasks or
    // more for each warp (at the size above 34.1 us against 41).
    const long long rows = (long long)c.B * c.S * (c.H[0] + c.H[1]);
    if (rows / (4 * (32 / LPR)) < 16ll * dev.sm_count) return run_direct<T, LPR, 1>(c, stream);
    const int tile = fwd_tile(c.S, c.H[0], c.H[1], c.Dh), group = tile_rows(c.H[0], c.H[1], c.Dh) * (32 / LPR);
    if ((long long)tile * ((c.H[0] + group - 1) / group) < 4 * kWarps) return run_direct<T, LPR, 4>(c, stream);
    return pick_tile<T, LPR, false>(c, stream, dev);
}

}  // namespace

size_t heads_bwd_ws_floats(int B, int S, int Hq, int Hk, int Dh) {
    const int tile = bwd_tile(S, Hq, Hk, Dh);
    const size_t tiles = ((size_t)S + tile - 1) / tile;
    return (size_t)B * (tiles + 1) * 2 * Dh;
}

template <typename T>
cudaError_t launch_heads_fwd(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev) {
    switch (lanes_per_row(c.Dh)) {
        case 4: return pick_fwd<T, 4>(c, stream, dev);
        case 8: return pick_fwd<T, 8>(c, stream, dev);
        case 16: return pick_fwd<T, 16>(c, stream, dev);
        default: return pick_fwd<T, 32>(c, stream, dev);
    }
}

template <typename T>
cudaError_t launch_heads_bwd(const HeadsCall &c, cudaStream_t stream, const DeviceInfo &dev) {
    cudaError_t e;
    switch (lanes_per_row(c.Dh)) {
        case 4: e = pick_tile<T, 4, true>(c, stream, dev); break;
        case 8: e = pick_tile<T, 8, true>(c, stream, dev); break;
        case 16: e = pick_tile<T, 16, true>(c, stream, dev); break;
        default: e = pick_tile<T, 32, true>(c, stream, dev); break;
    }
    if (e != cudaSuccess || (!c.dw[0] && !c.dw[1])) return e;
    FoldArgs f = {};
    f.part = c.ws;
    f.dw[0] = c.dw[0];
    f.dw[1] = c.dw[1];
    f.B = c.B;
    f.Dh = c.Dh;
    f.accumulate = c.accumulate;
    const int tile = bwd_tile(c.S, c.H[0], c.H[1], c.Dh);
    f.tiles = (c.S + tile - 1) / tile;
    f.sums = c.ws + (size_t)c.B * f.tiles * 2 * c.Dh;
    const unsigned cols = c.Dh / 8;
    if (c.B <= kDirectSamples) return launch_pdl(heads_fold_kernel<true>, dim3(cols, 2), dim3(1024), 0, stream, f);
    e = launch_pdl(heads_fold_kernel<false>, dim3(cols, 2, c.B), dim3(1024), 0, stream, f);
    if (e != cudaSuccess) return e;
    return launch_pdl(heads_samples_kernel, dim3((2 * c.Dh + 255) / 256), dim3(256), 0, stream, f);
}

template cudaError_t launch_heads_fwd<uint16_t>(const HeadsCall &, cudaStream_t, const DeviceInfo &);
template cudaError_t launch_heads_fwd<float>(const HeadsCall &, cudaStream_t, const DeviceInfo &);
template cudaError_t launch_heads_bwd<uint16_t>(const HeadsCall &, cudaStream_t, const DeviceInfo &);
template cudaError_t launch_heads_bwd<float>(const HeadsCall &, cudaStream_t, const DeviceInfo &);

}  // namespace adaln
