// The 8-bit record of a row (include/adaln_tune.h): codes, scale bytes.
#pragma once

#include "common.cuh"

namespace adaln {

constexpr int kCkptGroup = 32;  // channels a scale byte covers

__host__ __device__ constexpr int ckpt8_code_bytes(int D) { return (D + 15) / 16 * 16; }
__host__ __device__ constexpr int ckpt8_groups(int D) { return (D + kCkptGroup - 1) / kCkptGroup; }
__host__ __device__ constexpr int ckpt8_row_bytes(int D) { return ckpt8_code_bytes(D) + (ckpt8_groups(D) + 15) / 16 * 16; }

// The scale byte of a group from the fp32 bits of its largest magnitude m 2^e,
// 1 <= m < 2: k = e - 6 brings it to 64 m < 128, and from m = 127.5 / 64 (mantissa
// bits 0x7F0000) on it is one more, which is a carry into the exponent.  k ends at
// 121: with 122 the code 64 would stand for 2^128.
constexpr uint32_t kCkptLastScale = 121 + 127;
__device__ __forceinline__ uint32_t ckpt8_scale(uint32_t max_bits) {
    if (max_bits >= 0x7F800000u) return 255u;
    const int s = (int)((max_bits + 0x10000u) >> 23) - 6;
    return s < 1 ? 1u : min((uint32_t)s, kCkptLastScale);
}
// 2^k of a scale byte k + 127 (255: infinity, which makes every value 0 * inf = NaN)
__device__ __forceinline__ float ckpt8_step(uint32_t scale) { return __uint_as_float(scale << 23); }
// 2^-k (scale bytes 1 .. 253)
__device__ __forceinline__ float ckpt8_inverse(uint32_t scale) { return __uint_as_float((254u - scale) << 23); }

// Four codes, low byte first: x 2^-k rounded to an integer by adding 1.5 * 2^23
// (the product with a power of two is exact, and the fused form rounds once, to
// even); the integer stands in the low bits, in two's complement.
__device__ __forceinline__ uint32_t ckpt8_codes(px2 lo, px2 hi, px2 inv) {
    const px2 magic = px_splat(12582912.0f);
    const px2 a = px_fma(lo, inv, magic), b = px_fma(hi, inv, magic);
    const uint32_t p = __byte_perm(__float_as_uint(px_lo(a)), __float_as_uint(px_hi(a)), 0x0040);
    const uint32_t q = __byte_perm(__float_as_uint(px_lo(b)), __float_as_uint(px_hi(b)), 0x0040);
    return __byte_perm(p, q, 0x5410);
}

// Four codes of a group with that scale byte (not 255)
__device__ __forceinline__ uint32_t ckpt8_clamped(px2 (&x)[2], uint32_t scale) {
    if (scale == kCkptLastScale) {  // values from 127.5 2^121 on would round to 128: 127
        const float most = 127.0f * 0x1p121f;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            x[q] = px_make(fminf(fmaxf(px_lo(x[q]), -most), most), fminf(fmaxf(px_hi(x[q]), -most), most));
    }
    return ckpt8_codes(x[0], x[1], px_splat(ckpt8_inverse(scale)));
}

// Four codes as exact fp32 pairs: byte + 128 in the low bits of 2^23, less 2^23 + 128
__device__ __forceinline__ void ckpt8_floats(uint32_t w, px2 &lo, px2 &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const px2 less = px_splat(-8388736.0f);
    lo = px_add(px_make(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)),
                        __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541))), less);
    hi = px_add(px_make(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)),
                        __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543))), less);
}

// the largest magnitude's bits among 8 channels, bf16 (as 16-bit halves) or fp32
// (a NaN wins, in either)
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t ckpt8_max(const uint4 &v) {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = bf16x2_max(bf16x2_max(v.x & m, v.y & m), bf16x2_max(v.z & m, v.w & m));
    return max(a << 16, a & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t ckpt8_max(const float4 &a, const float4 &b) {
    const uint32_t m = 0x7FFFFFFFu;
    const uint32_t x = max(max(__float_as_uint(a.x) & m, __float_as_uint(a.y) & m),
                           max(__float_as_uint(a.z) & m, __float_as_uint(a.w) & m));
    const uint32_t y = max(max(__float_as_uint(b.x) & m, __float_as_uint(b.y) & m),
                           max(__float_as_uint(b.z) & m, __float_as_uint(b.w) & m));
    return max(x, y);
}

// Parts of a record, by the lanes of a warp that hold the row: vector v0 + 32 j (j <
// N, v0 mod 32 the lane) has E channels, LANES = 32 / E neighbouring lanes, the first
// with v a multiple of LANES, hold a group; V vectors in the row, past them
// max_bits[j] is 0 and pairs(j, p) gives zeros.  The whole warp runs this; steps j
// with 32 j past the row's last group do nothing.  Fills the record's padding as well.
//
// C < N: the row ends after C steps, and the steps go on in the next row, row_step
// bytes of records further; the first `left` of these N / C rows are there (the
// others' max_bits 0, their pairs zeros).
//
// A step's chain (maximum, exchanges, scale, codes) is long and its work short, so the
// N chains run side by side, without branches, but where a group holds an infinity,
// a NaN or ends at the last scale: then the row's part is written one by one.
template <int N, int E, int C = N, typename F>
__device__ __forceinline__ void ckpt8_put(unsigned char *rec, int code_bytes, int V, int v0, uint32_t (&max_bits)[N],
                                          F pairs, size_t row_step = 0, int left = 1) {
    constexpr int LANES = kCkptGroup / E;
    static_assert(E == 8 || E == 4, "8 bytes of codes a lane, or 4");
#pragma unroll
    for (int d = 1; d < LANES; d *= 2)
#pragma unroll
        for (int j = 0; j < N; ++j) max_bits[j] = max(max_bits[j], __shfl_xor_sync(0xFFFFFFFFu, max_bits[j], d));
    uint32_t scale[N], most = 0u;
#pragma unroll
    for (int j = 0; j < N; ++j) scale[j] = ckpt8_scale(max_bits[j]), most = max(most, scale[j]);
    auto store = [&](int j, const uint32_t (&c)[E / 4]) {
        if (C < N && j / C >= left) return;
        unsigned char *to = rec + (j / C) * row_step;
        const int v = v0 + 32 * (j % C);
        if (v * E < code_bytes) {
            if (E == 8)
                *reinterpret_cast<uint2 *>(to + (size_t)v * E) = make_uint2(c[0], c[E / 4 - 1]);
            else
                *reinterpret_cast<uint32_t *>(to + (size_t)v * E) = c[0];
        }
        if (v % LANES == 0 && v < V) to[code_bytes + v / LANES] = (unsigned char)scale[j];
    };
    if (!__any_sync(0xFFFFFFFFu, most >= kCkptLastScale)) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            px2 x[E / 2];
            pairs(j, x);
            const px2 inv = px_splat(ckpt8_inverse(scale[j]));
            uint32_t c[E / 4];
#pragma unroll
            for (int q = 0; q < E / 4; ++q) c[q] = ckpt8_codes(x[2 * q], x[2 * q + 1], inv);
            store(j, c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            px2 x[E / 2];
            pairs(j, x);
            uint32_t c[E / 4];
#pragma unroll
            for (int q = 0; q < E / 4; ++q) {
                px2 y[2] = {x[2 * q], x[2 * q + 1]};
                c[q] = scale[j] == 255u ? 0u : ckpt8_clamped(y, scale[j]);
            }
            store(j, c);
        }
    }
    // the scales' padding, by the lane of the last group
    const int last = (V - 1) / LANES * LANES;
    if (last >= v0 && (last - v0) % 32 == 0 && (last - v0) / 32 < C)
        for (int r = 0; r < (C < N ? left : 1); ++r)
            for (int i = last / LANES + 1; i & 15; ++i) rec[r * row_step + code_bytes + i] = 0;
}

}  // namespace adaln
