// Embedding lookup with scaling, and the table's gradient (contract:
// include/adaln_ops.h).
//
//   out[i] = scale * table[t_i];   dT[v] = scale * sum over i, t_i = v, of d_out[i]
//
// Both are bound by HBM: rows read and rows written.  The gradient groups the
// tokens first, so that every row of d_out is read once, every row of dT is
// written once by one owner, and no floating-point atomic decides an order:
//   1. a stable radix sort of (token, place), 8 bits a pass, as many passes as
//      V has bytes;  n <= kSmall: one CTA, in shared memory, otherwise a
//      histogram and a scatter kernel per pass;
//   2. the runs of equal tokens cut into pieces of 32 places.  Which list entry
//      a piece gets is left to an integer atomic: it decides who computes
//      the piece, not what;
//   3. a warp per (piece, group of columns) adds the piece's rows in ascending order;
//      a token with one piece is written at once, the pieces of longer runs
//      go to partial sums.  The same kernel writes the zero rows;
//   4. the partial sums of the long runs.
#include "common.cuh"
#include "ops.h"

namespace adaln {

namespace {

constexpr int kSmall = 4096;      // tokens that one CTA sorts
constexpr int kPiece = 32;        // places of a piece
constexpr int kDigits = 256;      // 8 bits a pass
constexpr int kTileMin = 2048;    // tokens of a sorting CTA
constexpr int kMaxTiles = 256;    // ... and the number of such CTAs

struct Piece {
    int token, start, len;
    int slot;  // partial sum, or -1: the token's only piece
};
struct Run {
    int token, slot, pieces;
};
struct Counts {
    int pieces, runs, slots;
};

__device__ __forceinline__ uint32_t token_key(const void *tokens, int is64, int i, int V) {
    const long long t = is64 ? static_cast<const long long *>(tokens)[i] : static_cast<const int *>(tokens)[i];
    return t >= 0 && t < V ? (uint32_t)t : (uint32_t)V;  // padding sorts last
}

// --------------------------------------------------------------------------
// lookup: a warp takes 4 vectors of 16 bytes a lane of one row
// --------------------------------------------------------------------------
__device__ __forceinline__ uint4 scale16(uint4 v, float c, uint16_t) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(__fmul_rn(bf16lo(w[i]), c), __fmul_rn(bf16hi(w[i]), c));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 scale16(uint4 v, float c, float) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__fmul_rn(__uint_as_float(w[i]), c));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void __launch_bounds__(256)
embed_fwd_kernel(const void *tokens, int is64, const T *__restrict__ table, float scale, T *__restrict__ out, int n,
                 int V, int D) {
    constexpr int E = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int vecs = D / E, groups = (vecs + 127) / 128;
    const long long total = (long long)n * groups;
    pdl_wait();
    pdl_trigger();
    for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < total;
         task += (long long)gridDim.x * 8) {
        const int i = (int)(task / groups), v0 = (int)(task % groups) * 128 + lane;
        const uint32_t key = token_key(tokens, is64, i, V);
        const bool real = key < (uint32_t)V;
        const uint4 *src = reinterpret_cast<const uint4 *>(table + (long long)(real ? key : 0) * D);
        uint4 *dst = reinterpret_cast<uint4 *>(out + (long long)i * D);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (real && v0 + 32 * j < vecs) v[j] = __ldg(src + v0 + 32 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v0 + 32 * j < vecs) dst[v0 + 32 * j] = real ? scale16(v[j], scale, T()) : v[j];
    }
}

// --------------------------------------------------------------------------
// sorting
// --------------------------------------------------------------------------
// lanes of the warp with the same digit (among the lanes of `active`)
__device__ __forceinline__ unsigned same_digit(unsigned active, int digit) { return __match_any_sync(active, digit); }

// Exclusive scan of one value per thread over the first 256 threads of a CTA
// (all threads call it; the others pass 0 and ignore the result).
__device__ int scan256(int v, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
        if (lane >= off) inc += o;
    }
    if (warp < 8 && lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < warp && i < 8; ++i) before += warp_sums[i];
    __syncthreads();
    return before + inc - v;
}

// First index of keys[0, n) (ascending) whose key is >= k.
__device__ __forceinline__ int lower_bound(const uint32_t *keys, int n, uint32_t k) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (keys[mid] < k)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Pieces of the run that begins at sorted place i, if one does.  Called by
// whole warps: long runs are written by all lanes together.
__device__ void plan_place(const uint32_t *keys, int n, int V, int i, Piece *pieces, Run *runs, Counts *counts) {
    const int lane = threadIdx.x & 31;
    int len = 0;
    uint32_t key = (uint32_t)V;
    if (i < n) {
        key = keys[i];
        if (key < (uint32_t)V && (i == 0 || keys[i - 1] != key)) {
            // the end: nearby for most tokens, otherwise by bisection
            int e = i + 1;
            while (e < n && e < i + 4 && keys[e] == key) ++e;
            if (e == i + 4 && e < n && keys[e] == key) e += lower_bound(keys + e, n - e, key + 1);
            len = e - i;
        }
    }
    const int np = (len + kPiece - 1) / kPiece;
    // one atomic per warp and counter
    int inc = np, slots = np > 1 ? np : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int a = __shfl_up_sync(0xFFFFFFFFu, inc, off), b = __shfl_up_sync(0xFFFFFFFFu, slots, off);
        if (lane >= off) inc += a, slots += b;
    }
    const int all = __shfl_sync(0xFFFFFFFFu, inc, 31), all_slots = __shfl_sync(0xFFFFFFFFu, slots, 31);
    if (all == 0) return;
    const unsigned longs = __ballot_sync(0xFFFFFFFFu, np > 1);
    int base = 0, slot_base = 0, run_base = 0;
    if (lane == 0) {
        base = atomicAdd(&counts->pieces, all);
        if (longs) {
            slot_base = atomicAdd(&counts->slots, all_slots);
            run_base = atomicAdd(&counts->runs, __popc(longs));
        }
    }
    base = __shfl_sync(0xFFFFFFFFu, base, 0) + inc - np;
    slot_base = __shfl_sync(0xFFFFFFFFu, slot_base, 0) + slots - (np > 1 ? np : 0);
    run_base = __shfl_sync(0xFFFFFFFFu, run_base, 0) + __popc(longs & ((1u << lane) - 1));
    if (np == 1) pieces[base] = Piece{(int)key, i, len, -1};
    if (np > 1) runs[run_base] = Run{(int)key, slot_base, np};
    for (unsigned m = longs; m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int token = __shfl_sync(0xFFFFFFFFu, (int)key, src), start = __shfl_sync(0xFFFFFFFFu, i, src);
        const int n_p = __shfl_sync(0xFFFFFFFFu, np, src), length = __shfl_sync(0xFFFFFFFFu, len, src);
        const int at = __shfl_sync(0xFFFFFFFFu, base, src), slot = __shfl_sync(0xFFFFFFFFu, slot_base, src);
        for (int p = lane; p < n_p; p += 32)
            pieces[at + p] = Piece{token, start + p * kPiece, min(kPiece, length - p * kPiece), slot + p};
    }
}

// n <= kSmall: sort and plan in one CTA of 32 warps, 4 places a thread, warp w
// holding the places [128 w, 128 w + 128) of every pass.
struct SmallShared {
    uint32_t keys[kSmall];
    int idx[kSmall];
    int cnt[32][kDigits];
    int warp_sums[8];
};

__global__ void __launch_bounds__(1024)
embed_sort_small_kernel(const void *tokens, int is64, int n, int V, int passes, uint32_t *keys_out, int *idx_out,
                        Piece *pieces, Run *runs, Counts *counts) {
    extern __shared__ __align__(16) unsigned char raw[];
    SmallShared &sh = *reinterpret_cast<SmallShared *>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) *counts = Counts{0, 0, 0};
    uint32_t key[4];
    int idx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        idx[j] = warp * 128 + j * 32 + lane;
        key[j] = idx[j] < n ? token_key(tokens, is64, idx[j], V) : 0xFFFFFFFFu;  // behind the end: sorts last
    }
    for (int pass = 0; pass < passes; ++pass) {
        for (int d = lane; d < kDigits; d += 32) sh.cnt[warp][d] = 0;
        __syncwarp();
        int rank[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int digit = (key[j] >> (8 * pass)) & 255;
            const unsigned peers = same_digit(0xFFFFFFFFu, digit);
            const int before = __popc(peers & ((1u << lane) - 1));
            const int base = sh.cnt[warp][digit];
            __syncwarp();
            if (before == 0) sh.cnt[warp][digit] = base + __popc(peers);
            __syncwarp();
            rank[j] = base + before;
        }
        __syncthreads();
        // counts of a digit over the warps, then the digits
        int total = 0;
        if (threadIdx.x < kDigits) {
            for (int w = 0; w < 32; ++w) {
                const int c = sh.cnt[w][threadIdx.x];
                sh.cnt[w][threadIdx.x] = total;
                total += c;
            }
        }
        const int first = scan256(total, sh.warp_sums);
        if (threadIdx.x < kDigits)
            for (int w = 0; w < 32; ++w) sh.cnt[w][threadIdx.x] += first;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = sh.cnt[warp][(key[j] >> (8 * pass)) & 255] + rank[j];
            sh.keys[at] = key[j];
            sh.idx[at] = idx[j];
        }
        __syncthreads();
        if (pass + 1 < passes) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                key[j] = sh.keys[warp * 128 + j * 32 + lane];
                idx[j] = sh.idx[warp * 128 + j * 32 + lane];
            }
            __syncthreads();
        }
    }
    for (int i = threadIdx.x; i < n; i += 1024) {
        keys_out[i] = sh.keys[i];
        idx_out[i] = sh.idx[i];
    }
    for (int i0 = 0; i0 < n; i0 += 1024) plan_place(sh.keys, n, V, i0 + threadIdx.x, pieces, runs, counts);
}

// larger n: pass by pass.  CTA b holds the places [b * tile, (b + 1) * tile),
// its warp w an eighth of them; hist [tiles][256].
struct SortArgs {
    const void *tokens;  // the first pass reads the tokens themselves
    int is64;
    const uint32_t *keys_in;
    const int *idx_in;
    uint32_t *keys_out;
    int *idx_out;
    int *hist;
    Counts *counts;
    int n, V, tile, tiles, shift;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs &a, int i) {
    return a.keys_in ? a.keys_in[i] : token_key(a.tokens, a.is64, i, a.V);
}

__global__ void __launch_bounds__(256) embed_hist_kernel(const SortArgs a) {
    __shared__ int cnt[kDigits];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counts = Counts{0, 0, 0};
    const int i1 = min(a.n, (int)(blockIdx.x + 1) * a.tile);
    for (int i = blockIdx.x * a.tile + threadIdx.x; i < i1; i += 256)
        atomicAdd(&cnt[(sort_key(a, i) >> a.shift) & 255], 1);
    __syncthreads();
    a.hist[blockIdx.x * kDigits + threadIdx.x] = cnt[threadIdx.x];
}

__global__ void __launch_bounds__(256) embed_scatter_kernel(const SortArgs a) {
    __shared__ int cnt[8][kDigits];  // next place of a digit, per warp
    __shared__ int warp_sums[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = threadIdx.x;
    for (int w = 0; w < 8; ++w) cnt[w][d] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int part = a.tile / 8;
    const int i0 = blockIdx.x * a.tile + warp * part, i1 = min(a.n, i0 + part);
    for (int i = i0 + lane; i < i1; i += 32) atomicAdd(&cnt[warp][(sort_key(a, i) >> a.shift) & 255], 1);
    int before = 0, total = 0;  // of digit d: in the CTAs before this one, and in all
#pragma unroll 8
    for (int b = 0; b < a.tiles; ++b) {
        const int c = __ldcg(a.hist + b * kDigits + d);
        total += c;
        before += b < (int)blockIdx.x ? c : 0;
    }
    const int first = scan256(total, warp_sums) + before;  // its barriers also close the counting
    int next = first;
    for (int w = 0; w < 8; ++w) {
        const int c = cnt[w][d];
        cnt[w][d] = next;
        next += c;
    }
    __syncthreads();
    for (int i = i0; i < i1; i += 32) {
        const unsigned active = __ballot_sync(0xFFFFFFFFu, i + lane < i1);
        if (i + lane < i1) {
            const uint32_t key = sort_key(a, i + lane);
            const int digit = (key >> a.shift) & 255;
            const unsigned peers = same_digit(active, digit);
            const int rank = __popc(peers & ((1u << lane) - 1));
            const int at = cnt[warp][digit] + rank;
            __syncwarp(active);
            if (rank == 0) cnt[warp][digit] += __popc(peers);
            __syncwarp(active);
            a.keys_out[at] = key;
            a.idx_out[at] = a.idx_in ? a.idx_in[i + lane] : i + lane;
        }
    }
}

__global__ void __launch_bounds__(256) embed_plan_kernel(const uint32_t *keys, int n, int V, Piece *pieces, Run *runs,
                                                         Counts *counts) {
    pdl_wait();
    pdl_trigger();
    plan_place(keys, n, V, blockIdx.x * 256 + threadIdx.x, pieces, runs, counts);
}

// --------------------------------------------------------------------------
// sums
// --------------------------------------------------------------------------
struct SumArgs {
    const void *d_out;
    const uint32_t *keys;
    const int *idx;
    const Piece *pieces;
    const Run *runs;
    const Counts *counts;
    float *partial;  // [slots][D]
    float *acc;      // [V][D] fp32, or
    uint16_t *bf16;  // [V][D]
    float scale;
    int accumulate, n, V, D;
};

// 8 channels of a lane
__device__ __forceinline__ void load_row8(float (&v)[8], const uint16_t *p) {
    const uint4 t = ldg16(p);
    v[0] = bf16lo(t.x), v[1] = bf16hi(t.x), v[2] = bf16lo(t.y), v[3] = bf16hi(t.y);
    v[4] = bf16lo(t.z), v[5] = bf16hi(t.z), v[6] = bf16lo(t.w), v[7] = bf16hi(t.w);
}
__device__ __forceinline__ void load_row8(float (&v)[8], const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// N columns (4 or 8) of row v of the gradient
template <int N>
__device__ __forceinline__ void put_row(const SumArgs &a, int token, int col, const float (&s)[N]) {
    const long long at = (long long)token * a.D + col;
    float r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __fmul_rn(s[i], a.scale);
    if (a.bf16) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<uint2 *>(a.bf16 + at + i) =
                make_uint2(pack_bf16x2(r[i], r[i + 1]), pack_bf16x2(r[i + 2], r[i + 3]));
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float4 *p = reinterpret_cast<float4 *>(a.acc + at + i);
        float4 o = make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        if (a.accumulate) {
            const float4 c = *p;
            o = make_float4(__fadd_rn(c.x, o.x), __fadd_rn(c.y, o.y), __fadd_rn(c.z, o.z), __fadd_rn(c.w, o.w));
        }
        *p = o;
    }
}

// A warp per (piece, 256 columns); then, without accumulate, a warp per (32
// rows of the table, 256 columns), which writes the rows without a token.
template <typename T>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs a) {
    constexpr int U = 8;  // rows in flight
    const int lane = threadIdx.x & 31;
    const int groups = (a.D + 255) / 256;
    const T *d_out = static_cast<const T *>(a.d_out);
    pdl_wait();
    pdl_trigger();
    const long long piece_tasks = (long long)__ldcg(&a.counts->pieces) * groups;
    const long long total = piece_tasks + (a.accumulate ? 0 : (long long)((a.V + 31) / 32) * groups);
    for (long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); task < total;
         task += (long long)gridDim.x * 8) {
        if (task < piece_tasks) {
            const int4 pc = __ldcg(reinterpret_cast<const int4 *>(a.pieces + task / groups));
            const Piece p{pc.x, pc.y, pc.z, pc.w};
            const int col = (int)(task % groups) * 256 + lane * 8;
            const bool live = col < a.D;
            const int mine = lane < p.len ? __ldcg(a.idx + p.start + lane) : 0;
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = 0.0f;
            for (int r0 = 0; r0 < p.len; r0 += U) {
                float v[U][8];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int row = __shfl_sync(0xFFFFFFFFu, mine, (r0 + u) & 31);
                    if (live && r0 + u < p.len) load_row8(v[u], d_out + (long long)row * a.D + col);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r0 + u < p.len) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[i] = __fadd_rn(s[i], v[u][i]);
                    }
            }
            if (live && p.slot < 0) {
                put_row(a, p.token, col, s);
            } else if (live) {
                float *q = a.partial + (long long)p.slot * a.D + col;
                *reinterpret_cast<float4 *>(q) = make_float4(s[0], s[1], s[2], s[3]);
                *reinterpret_cast<float4 *>(q + 4) = make_float4(s[4], s[5], s[6], s[7]);
            }
        } else {
            const long long zt = task - piece_tasks;
            const int v0 = (int)(zt / groups) * 32, col = (int)(zt % groups) * 256 + lane * 8;
            const int v = v0 + lane;
            bool absent = false;
            if (v < a.V) {
                const int at = lower_bound(a.keys, a.n, (uint32_t)v);
                absent = at == a.n || a.keys[at] != (uint32_t)v;
            }
            unsigned m = __ballot_sync(0xFFFFFFFFu, absent);
            if (col >= a.D) m = 0;
            for (; m; m &= m - 1) {
                const long long o = (long long)(v0 + __ffs(m) - 1) * a.D + col;
                if (a.bf16) {
                    stg16(a.bf16 + o, make_uint4(0, 0, 0, 0));
                } else {
                    stg16(a.acc + o, make_uint4(0, 0, 0, 0));
                    stg16(a.acc + o + 4, make_uint4(0, 0, 0, 0));
                }
            }
        }
    }
}

// Runs of several pieces: a CTA per (run, 128 columns).  Warp w adds an eighth
// of the partial sums in order, then the warps are added in order.
__global__ void __launch_bounds__(256) embed_runs_kernel(const SumArgs a) {
    __shared__ float red[8][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (a.D + 127) / 128;
    pdl_wait();
    pdl_trigger();
    const long long total = (long long)__ldcg(&a.counts->runs) * groups;
    for (long long task = blockIdx.x; task < total; task += gridDim.x) {
        const int *rp = reinterpret_cast<const int *>(a.runs + task / groups);
        const Run r{__ldcg(rp), __ldcg(rp + 1), __ldcg(rp + 2)};
        const int col = (int)(task % groups) * 128 + lane * 4;
        const int per = (r.pieces + 7) / 8, p0 = warp * per, p1 = min(r.pieces, p0 + per);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (col < a.D) {
            const float4 *q = reinterpret_cast<const float4 *>(a.partial + (long long)(r.slot + p0) * a.D + col);
#pragma unroll 8
            for (int p = p0; p < p1; ++p, q += a.D / 4) {
                const float4 v = __ldcg(q);
                s[0] = __fadd_rn(s[0], v.x), s[1] = __fadd_rn(s[1], v.y);
                s[2] = __fadd_rn(s[2], v.z), s[3] = __fadd_rn(s[3], v.w);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][lane * 4 + i] = s[i];
        __syncthreads();
        if (warp == 0 && col < a.D) {
#pragma unroll
            for (int w = 1; w < 8; ++w) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = __fadd_rn(s[i], red[w][lane * 4 + i]);
            }
            put_row(a, r.token, col, s);
        }
        __syncthreads();
    }
}

// Workspace: [counts | pieces n | runs | keys 2n | idx 2n | hist | partial].
struct Layout {
    size_t counts, pieces, runs, keys, idx, hist, partial, bytes;
};
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
Layout layout(int n, int D) {
    Layout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    l.counts = take(sizeof(Counts));
    l.pieces = take((size_t)n * sizeof(Piece));
    l.runs = take(((size_t)n / kPiece + 1) * sizeof(Run));
    l.keys = take((size_t)n * 2 * sizeof(uint32_t));
    l.idx = take((size_t)n * 2 * sizeof(int));
    l.hist = take((size_t)kMaxTiles * kDigits * sizeof(int));
    // a run of several pieces has at least 33 places and at most 2 pieces for
    // every 33 of them
    l.partial = take(((size_t)n / 16 + 1) * D * sizeof(float));
    l.bytes = at;
    return l;
}

}  // namespace

size_t embed_bwd_ws_bytes(int n, int V, int D) {
    (void)V;
    return n > 0 ? layout(n, D).bytes : 0;
}

template <typename T>
cudaError_t launch_embed_fwd(const void *tokens, int tokens_are_64, const T *table, float scale, T *out, int n, int V,
                             int D, cudaStream_t stream, const DeviceInfo &) {
    const int vecs = D * (int)sizeof(T) / 16;
    const long long ctas = ((long long)n * ((vecs + 127) / 128) + 7) / 8;
    return launch_pdl(embed_fwd_kernel<T>, dim3((unsigned)(ctas < (1 << 30) ? ctas : (1 << 30))), dim3(256), 0, stream,
                      tokens, tokens_are_64, table, scale, out, n, V, D);
}

template <typename T>
cudaError_t launch_embed_bwd(const T *d_out, const void *tokens, int tokens_are_64, float scale, float *d_table_acc,
                             uint16_t *d_table, int accumulate, void *ws, int n, int V, int D, cudaStream_t stream,
                             const DeviceInfo &dev) {
    char *base = static_cast<char *>(ws);
    const Layout l = layout(n, D);
    Counts *counts = reinterpret_cast<Counts *>(base + l.counts);
    Piece *pieces = reinterpret_cast<Piece *>(base + l.pieces);
    Run *runs = reinterpret_cast<Run *>(base + l.runs);
    uint32_t *keys = reinterpret_cast<uint32_t *>(base + l.keys);
    int *idx = reinterpret_cast<int *>(base + l.idx);
    int passes = 1;  // keys are 0 .. V
    while (passes < 4 && ((uint32_t)V >> (8 * passes)) != 0) ++passes;
    cudaError_t e = cudaSuccess;
    if (n <= kSmall) {
        // keys behind the end are all ones in the bytes sorted: with V also all
        // ones they tie with padding, which comes first by its place
        e = ensure_smem_attr((const void *)embed_sort_small_kernel, sizeof(SmallShared), dev);
        if (e != cudaSuccess) return e;
        e = launch_pdl(embed_sort_small_kernel, dim3(1), dim3(1024), sizeof(SmallShared), stream, tokens, tokens_are_64,
                       n, V, passes, keys, idx, pieces, runs, counts);
        if (e != cudaSuccess) return e;
    } else {
        SortArgs s = {};
        s.tokens = tokens;
        s.is64 = tokens_are_64;
        s.hist = reinterpret_cast<int *>(base + l.hist);
        s.counts = counts;
        s.n = n;
        s.V = V;
        // at most kMaxTiles CTAs, a multiple of 256 places each
        s.tile = (n + kMaxTiles - 1) / kMaxTiles;
        s.tile = s.tile <= kTileMin ? kTileMin : (s.tile + 255) / 256 * 256;
        s.tiles = (n + s.tile - 1) / s.tile;
        for (int pass = 0; pass < passes; ++pass) {
            const int half = pass & 1;
            s.keys_in = pass == 0 ? nullptr : keys + (size_t)(1 - half) * n;
            s.idx_in = pass == 0 ? nullptr : idx + (size_t)(1 - half) * n;
            s.keys_out = keys + (size_t)half * n;
            s.idx_out = idx + (size_t)half * n;
            s.shift = 8 * pass;
            e = launch_pdl(embed_hist_kernel, dim3(s.tiles), dim3(256), 0, stream, s);
            if (e != cudaSuccess) return e;
            e = launch_pdl(embed_scatter_kernel, dim3(s.tiles), dim3(256), 0, stream, s);
            if (e != cudaSuccess) return e;
        }
        keys = s.keys_out;
        idx = s.idx_out;
        e = launch_pdl(embed_plan_kernel, dim3((n + 255) / 256), dim3(256), 0, stream, (const uint32_t *)keys, n, V,
                       pieces, runs, counts);
        if (e != cudaSuccess) return e;
    }
    SumArgs a = {};
    a.d_out = d_out;
    a.keys = keys;
    a.idx = idx;
    a.pieces = pieces;
    a.runs = runs;
    a.counts = counts;
    a.partial = reinterpret_cast<float *>(base + l.partial);
    a.acc = d_table_acc;
    a.bf16 = d_table;
    a.scale = scale;
    a.accumulate = accumulate;
    a.n = n;
    a.V = V;
    a.D = D;
    e = launch_pdl(embed_sum_kernel<T>, dim3(dev.sm_count * 4), dim3(256), 0, stream, a);
    if (e != cudaSuccess || n <= kPiece) return e;
    return launch_pdl(embed_runs_kernel, dim3(dev.sm_count * 2), dim3(256), 0, stream, a);
}

template cudaError_t launch_embed_fwd<uint16_t>(const void *, int, const uint16_t *, float, uint16_t *, int, int, int,
                                                cudaStream_t, const DeviceInfo &);
template cudaError_t launch_embed_fwd<float>(const void *, int, const float *, float, float *, int, int, int,
                                             cudaStream_t, const DeviceInfo &);
template cudaError_t launch_embed_bwd<uint16_t>(const uint16_t *, const void *, int, float, float *, uint16_t *, int,
                                                void *, int, int, int, cudaStream_t, const DeviceInfo &);
template cudaError_t launch_embed_bwd<float>(const float *, const void *, int, float, float *, uint16_t *, int, void *,
                                             int, int, int, cudaStream_t, const DeviceInfo &);

}  // namespace adaln
