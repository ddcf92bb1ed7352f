// Embedding lookup with scaling, and the table's gradient (contract:
// include/adaln_ops.h).
//
//   out[i] = scale * table[t_i];   dT[v] = scale * sum over i, t_i = v, of d_out[i]
//
// Both are bound by HBM: rows read and rows written.  The gradient groups the
// tokens first, so that every row of d_out is read once, every row of dT has
// one owner, and no floating-point atomic decides an order:
//   1. a stable radix sort of (token, place), at most 8 bits a pass: in the
//      shared memory of one CTA where a token and a place fit 32 bits together
//      and n <= kCtaTokens, otherwise by a histogram and a scatter kernel a pass;
//   2. the runs of equal tokens cut into pieces of 32 places.  Which list entry
//      a piece gets is left to an integer atomic: it decides who computes
//      the piece, not what;
//   3. a warp per (piece, 256 columns) adds the piece's rows in ascending order.
//      A token with one piece is written at once.  The pieces of longer runs
//      are the leaves of a 32-way tree: whoever brings the last child of a node
//      adds the children in order (a ticket per node; nobody waits).
// Sorting is a chain of latencies that leaves the memory idle, so the table is
// zeroed meanwhile, by the other CTAs of the sorting launches; step 3 then
// writes the rows of tokens that occur.
#include "common.cuh"
#include "ops.h"

namespace adaln {

namespace {

constexpr int kCtaThreads = 1024;
// Tokens that one CTA sorts, four a thread (11 us at 4096, most of it latency).
// With 32 a thread one CTA took 67 us for 32768 tokens; the kernels that share
// them among CTAs take about 25 us at any such size.
constexpr int kCtaTokens = 4 * kCtaThreads;
constexpr int kPiece = 32;        // places of a piece
constexpr int kFan = 32;          // children of a node
constexpr int kDigits = 256;      // at most 8 bits a pass
constexpr int kTileMin = 1024;    // tokens of a sorting CTA
constexpr int kMaxTiles = 256;    // ... and the number of such CTAs

// One piece of a token's run.  A run of several pieces has a partial sum for
// every piece and every node below the root, level by level from `slot`, and a
// ticket (per column group) for every node, level by level from `node`.
struct __align__(16) Piece {
    int token, start, len, index;  // index: which piece of the run; -1: the only one
    int pieces, slot, node, unused;
};
struct Counts {
    int singles, pieces, slots, nodes;  // runs of one piece; pieces, partial sums and nodes of the longer runs
};

// partial sums and nodes of a run of np > 1 pieces
__host__ __device__ inline void tree_size(int np, int &slots, int &nodes) {
    slots = nodes = 0;
    for (int n = np; n > 1;) {
        slots += n;
        n = (n + kFan - 1) / kFan;
        nodes += n;
    }
}

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

// The lanes whose digit equals this lane's, by one ballot a bit.  (With
// match.any the one-CTA sort of 4096 tokens took 13.5 us instead of 10.5.)
__device__ __forceinline__ unsigned same_digit(int digit, int digit_bits) {
    unsigned peers = 0xFFFFFFFFu;
    for (int k = 0; k < digit_bits; ++k) {
        const bool one = (digit >> k) & 1;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, one);
        peers &= one ? m : ~m;
    }
    return peers;
}

// --------------------------------------------------------------------------
// zeroing: CTAs [first, gridDim.x) of a sorting launch write their share
// --------------------------------------------------------------------------
struct Fill {
    uint4 *p;
    long long vecs;  // of 16 bytes; 0: nothing to zero
};
__device__ void fill_zero(const Fill &f, int cta, int ctas) {
    const long long step = (long long)ctas * blockDim.x;
    for (long long i = (long long)cta * blockDim.x + threadIdx.x; i < f.vecs; i += step)
        f.p[i] = make_uint4(0, 0, 0, 0);
}

// --------------------------------------------------------------------------
// pieces of the sorted tokens
// --------------------------------------------------------------------------
struct PackedKeys {  // token << bits | place
    const uint32_t *items;
    int bits;
    __device__ uint32_t operator()(int i) const { return items[i] >> bits; }
};
struct PlainKeys {
    const uint32_t *keys;
    __device__ uint32_t operator()(int i) const { return keys[i]; }
};

// The first place >= from whose key is not `key` (or n), by all lanes: the next
// 32 places, then a search by 32nds.
template <typename Keys>
__device__ int run_end(const Keys &keys, int n, int from, uint32_t key) {
    const int lane = threadIdx.x & 31;
    int lo = from, hi = min(n, from + 32);
    int c = __popc(__ballot_sync(0xFFFFFFFFu, lo + lane < hi && keys(lo + lane) == key));
    if (lo + c < hi || hi == n) return lo + c;
    lo = hi;
    hi = n;
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) / 32, p = lo + lane * step;
        c = __popc(__ballot_sync(0xFFFFFFFFu, p < hi && keys(p) == key));
        if (c == 0) return lo;
        hi = min(hi, lo + c * step);
        lo += (c - 1) * step + 1;
    }
    return lo + __popc(__ballot_sync(0xFFFFFFFFu, lo + lane < hi && keys(lo + lane) == key));
}

// The pieces of the runs that begin at the warp's 32 places base + lane.
template <typename Keys>
__device__ void plan_places(const Keys &keys, int n, int V, int base, int groups, Piece *pieces, int *tickets,
                            Counts *counts) {
    if (base >= n) return;
    const int lane = threadIdx.x & 31, i = base + lane;
    const uint32_t key = i < n ? keys(i) : 0xFFFFFFFFu;
    uint32_t prev = __shfl_up_sync(0xFFFFFFFFu, key, 1);
    if (lane == 0 && i > 0) prev = keys(i - 1);
    const bool edge = i >= n || i == 0 || key != prev;
    const bool head = edge && i < n && key < (uint32_t)V;
    const unsigned edges = __ballot_sync(0xFFFFFFFFu, edge);
    int len = 0;
    if (edges != 0) {
        // the last run may go on behind the warp's places
        const int last = 31 - __clz(edges);
        const int last_head = __shfl_sync(0xFFFFFFFFu, (int)head, last);
        int behind = base + 32;
        if (last_head) behind = run_end(keys, n, base + 32, __shfl_sync(0xFFFFFFFFu, key, last));
        const unsigned next = lane < 31 ? edges & (0xFFFFFFFEu << lane) : 0u;
        if (head) len = (next ? base + __ffs(next) - 1 : behind) - i;
    }
    const int np = (len + kPiece - 1) / kPiece;
    int slots = 0, nodes = 0;
    if (np > 1) tree_size(np, slots, nodes);
    // one atomic per warp and counter.  Long runs fill the list from the front,
    // so that their trees are begun first; the others from the back.
    const unsigned longs = __ballot_sync(0xFFFFFFFFu, np > 1), ones = __ballot_sync(0xFFFFFFFFu, np == 1);
    int4 *out = reinterpret_cast<int4 *>(pieces);
    if (ones) {
        int at = 0;
        if (lane == 0) at = atomicAdd(&counts->singles, __popc(ones));
        at = n - 1 - __shfl_sync(0xFFFFFFFFu, at, 0) - __popc(ones & ((1u << lane) - 1));
        if (np == 1) out[2 * at] = make_int4((int)key, i, len, -1);
    }
    if (longs == 0) return;
    const int mine = np > 1 ? np : 0;
    int at = mine, slot = slots, node = nodes;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, at, off), y = __shfl_up_sync(0xFFFFFFFFu, slot, off),
                  z = __shfl_up_sync(0xFFFFFFFFu, node, off);
        if (lane >= off) at += x, slot += y, node += z;
    }
    int at0 = 0, slot0 = 0, node0 = 0;
    if (lane == 31) {
        at0 = atomicAdd(&counts->pieces, at);
        slot0 = atomicAdd(&counts->slots, slot);
        node0 = atomicAdd(&counts->nodes, node);
    }
    at += __shfl_sync(0xFFFFFFFFu, at0, 31) - mine;
    slot += __shfl_sync(0xFFFFFFFFu, slot0, 31) - slots;
    node += __shfl_sync(0xFFFFFFFFu, node0, 31) - nodes;
    for (unsigned m = longs; m; m &= m - 1) {  // long runs: by all lanes
        const int src = __ffs(m) - 1;
        const int l_token = __shfl_sync(0xFFFFFFFFu, (int)key, src), l_start = __shfl_sync(0xFFFFFFFFu, i, src);
        const int l_len = __shfl_sync(0xFFFFFFFFu, len, src), l_np = __shfl_sync(0xFFFFFFFFu, np, src);
        const int l_at = __shfl_sync(0xFFFFFFFFu, at, src), l_slot = __shfl_sync(0xFFFFFFFFu, slot, src);
        const int l_node = __shfl_sync(0xFFFFFFFFu, node, src), l_nodes = __shfl_sync(0xFFFFFFFFu, nodes, src);
        for (int p = lane; p < l_np; p += 32) {
            out[2 * (l_at + p)] = make_int4(l_token, l_start + p * kPiece, min(kPiece, l_len - p * kPiece), p);
            out[2 * (l_at + p) + 1] = make_int4(l_np, l_slot, l_node, 0);
        }
        for (long long k = lane; k < (long long)l_nodes * groups; k += 32) tickets[(long long)l_node * groups + k] = 0;
    }
}

// --------------------------------------------------------------------------
// sorting in one CTA: 32 warps, IPT items a thread; warp w holds the places
// [32 IPT w, 32 IPT (w + 1)) of every pass.  An item is token << bits | place.
// --------------------------------------------------------------------------
constexpr int kCntStride = kDigits + 1;  // keeps the scan's reads in different banks
struct CtaShared {
    int cnt[32][kCntStride];  // per warp and digit: the count, then the next place
    int sums[32];
    Counts counts;
    uint32_t items[1];  // [IPT * 1024]
};

template <int IPT>
__global__ void __launch_bounds__(kCtaThreads)
embed_sort_cta_kernel(const void *tokens, int is64, int n, int V, int bits, int digit_bits, int passes, int groups,
                      int *idx_out, Piece *pieces, int *tickets, Counts *counts, Fill fill) {
    extern __shared__ __align__(16) unsigned char raw[];
    CtaShared &sh = *reinterpret_cast<CtaShared *>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x > 0) {
        fill_zero(fill, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    const int base = warp * (32 * IPT) + lane;
    const int nd = 1 << digit_bits;
    uint32_t item[IPT];
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const int i = base + 32 * j;
        item[j] = i < n ? token_key(tokens, is64, i, V) << bits | i : 0xFFFFFFFFu;  // behind the end: last
    }
    if (threadIdx.x == 0) sh.counts = Counts{0, 0, 0, 0};
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = bits + pass * digit_bits;
        for (int d = lane; d < nd; d += 32) sh.cnt[warp][d] = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < IPT; ++j) atomicAdd(&sh.cnt[warp][(item[j] >> shift) & (nd - 1)], 1);
        __syncthreads();
        // exclusive scan over (digit, warp): thread 4 d + q has the warps 8 q ..
        const int d = threadIdx.x >> 2, q = threadIdx.x & 3;
        int c[8], sum = 0;
        if (d < nd) {
#pragma unroll
            for (int k = 0; k < 8; ++k) c[k] = sh.cnt[8 * q + k][d];
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += c[k];
        }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) sh.sums[warp] = inc;
        __syncthreads();
        int before = lane < warp ? sh.sums[lane] : 0;
        before = __reduce_add_sync(0xFFFFFFFFu, before) + inc - sum;
        if (d < nd) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sh.cnt[8 * q + k][d] = before;
                before += c[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            const int digit = (item[j] >> shift) & (nd - 1);
            const unsigned peers = same_digit(digit, digit_bits);
            const int rank = __popc(peers & ((1u << lane) - 1));
            const int at = sh.cnt[warp][digit];
            __syncwarp();
            if (rank == 0) sh.cnt[warp][digit] = at + __popc(peers);
            __syncwarp();
            sh.items[at + rank] = item[j];
        }
        __syncthreads();
        if (pass + 1 < passes) {
#pragma unroll
            for (int j = 0; j < IPT; ++j) item[j] = sh.items[base + 32 * j];
            __syncthreads();
        }
    }
    const uint32_t mask = (1u << bits) - 1u;
    for (int i = threadIdx.x; i < n; i += kCtaThreads) idx_out[i] = (int)(sh.items[i] & mask);
    const PackedKeys keys{sh.items, bits};
    for (int i0 = warp * 32; i0 < n; i0 += kCtaThreads)
        plan_places(keys, n, V, i0, groups, pieces, tickets, &sh.counts);
    __syncthreads();
    if (threadIdx.x == 0) *counts = sh.counts;
}

// --------------------------------------------------------------------------
// larger sorts: pass by pass.  CTA b holds the places [b * tile, (b + 1) *
// tile), its warp w an eighth of them; hist [tiles][256].  The CTAs from
// `tiles` on zero their share of the table.
// --------------------------------------------------------------------------
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
    return a.keys_in ? __ldcg(a.keys_in + i) : token_key(a.tokens, a.is64, i, a.V);
}

__global__ void __launch_bounds__(256) embed_hist_kernel(const SortArgs a, const Fill fill) {
    __shared__ int cnt[kDigits];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= a.tiles) {
        fill_zero(fill, blockIdx.x - a.tiles, gridDim.x - a.tiles);
        return;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counts = Counts{0, 0, 0, 0};
    const int i1 = min(a.n, (int)(blockIdx.x + 1) * a.tile);
#pragma unroll 4
    for (int i = blockIdx.x * a.tile + threadIdx.x; i < i1; i += 256)
        atomicAdd(&cnt[(sort_key(a, i) >> a.shift) & 255], 1);
    __syncthreads();
    a.hist[blockIdx.x * kDigits + threadIdx.x] = cnt[threadIdx.x];
}

__global__ void __launch_bounds__(256) embed_scatter_kernel(const SortArgs a, const Fill fill) {
    constexpr int J = 4;             // places of a lane in flight
    __shared__ int cnt[8][kDigits];  // per warp and digit: the count, then the next place
    __shared__ int sums[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = threadIdx.x;
    for (int w = 0; w < 8; ++w) cnt[w][d] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= a.tiles) {
        fill_zero(fill, blockIdx.x - a.tiles, gridDim.x - a.tiles);
        return;
    }
    const int part = a.tile / 8;
    const int i0 = blockIdx.x * a.tile + warp * part, i1 = min(a.n, i0 + part);
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) atomicAdd(&cnt[warp][(sort_key(a, i) >> a.shift) & 255], 1);
    int before = 0, total = 0;  // of digit d: in the CTAs before this one, and in all
#pragma unroll 16
    for (int b = 0; b < a.tiles; ++b) {
        const int c = __ldcg(a.hist + b * kDigits + d);
        total += c;
        before += b < (int)blockIdx.x ? c : 0;
    }
    int inc = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
        if (lane >= off) inc += o;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();  // also closes the counting
    int next = before + inc - total;
    for (int w = 0; w < warp; ++w) next += sums[w];
    for (int w = 0; w < 8; ++w) {
        const int c = cnt[w][d];
        cnt[w][d] = next;
        next += c;
    }
    __syncthreads();
    for (int i = i0; i < i1; i += 32 * J) {
        uint32_t key[J];
        int idx[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = i + 32 * j + lane;
            key[j] = at < i1 ? sort_key(a, at) : 0u;
            idx[j] = at < i1 && a.idx_in ? __ldcg(a.idx_in + at) : at;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = i + 32 * j + lane < i1;
            const unsigned active = __ballot_sync(0xFFFFFFFFu, in);
            const int digit = (key[j] >> a.shift) & 255;
            const unsigned peers = same_digit(digit, 8) & active;
            const int rank = __popc(peers & ((1u << lane) - 1));
            const int at = cnt[warp][digit] + rank;
            __syncwarp();
            if (in && rank == 0) cnt[warp][digit] += __popc(peers);
            __syncwarp();
            if (in) {
                a.keys_out[at] = key[j];
                a.idx_out[at] = idx[j];
            }
        }
    }
}

__global__ void __launch_bounds__(256) embed_plan_kernel(const uint32_t *keys, int n, int V, int groups,
                                                         Piece *pieces, int *tickets, Counts *counts, int ctas,
                                                         const Fill fill) {
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= ctas) {
        fill_zero(fill, blockIdx.x - ctas, gridDim.x - ctas);
        return;
    }
    plan_places(PlainKeys{keys}, n, V, (int)(blockIdx.x * 256 + (threadIdx.x & ~31u)), groups, pieces, tickets, counts);
}

// --------------------------------------------------------------------------
// sums
// --------------------------------------------------------------------------
struct SumArgs {
    const void *d_out;
    const int *idx;
    const Piece *pieces;
    const Counts *counts;
    int *tickets;    // [nodes][groups]
    float *partial;  // [slots][D]
    float *acc;      // [V][D] fp32, or
    uint16_t *bf16;  // [V][D]
    float scale;
    int accumulate, n, D;
};

// 8 columns of a row as they lie in memory, and added to a sum
__device__ __forceinline__ void load8(uint4 &v, const uint16_t *p) { v = ldg16(p); }
struct Floats8 {
    float4 a, b;
};
__device__ __forceinline__ void load8(Floats8 &v, const float *p) {
    v.a = __ldcg(reinterpret_cast<const float4 *>(p));
    v.b = __ldcg(reinterpret_cast<const float4 *>(p + 4));
}
__device__ __forceinline__ void add8(float (&s)[8], const uint4 &v) {
    s[0] = __fadd_rn(s[0], bf16lo(v.x)), s[1] = __fadd_rn(s[1], bf16hi(v.x));
    s[2] = __fadd_rn(s[2], bf16lo(v.y)), s[3] = __fadd_rn(s[3], bf16hi(v.y));
    s[4] = __fadd_rn(s[4], bf16lo(v.z)), s[5] = __fadd_rn(s[5], bf16hi(v.z));
    s[6] = __fadd_rn(s[6], bf16lo(v.w)), s[7] = __fadd_rn(s[7], bf16hi(v.w));
}
__device__ __forceinline__ void add8(float (&s)[8], const Floats8 &v) {
    s[0] = __fadd_rn(s[0], v.a.x), s[1] = __fadd_rn(s[1], v.a.y);
    s[2] = __fadd_rn(s[2], v.a.z), s[3] = __fadd_rn(s[3], v.a.w);
    s[4] = __fadd_rn(s[4], v.b.x), s[5] = __fadd_rn(s[5], v.b.y);
    s[6] = __fadd_rn(s[6], v.b.z), s[7] = __fadd_rn(s[7], v.b.w);
}

// 8 columns of row `token` of the gradient
__device__ __forceinline__ void put_row(const SumArgs &a, int token, int col, const float (&s)[8]) {
    const long long at = (long long)token * a.D + col;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __fmul_rn(s[i], a.scale);
    if (a.bf16) {
        stg16(a.bf16 + at, make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]),
                                      pack_bf16x2(r[6], r[7])));
        return;
    }
    float4 *p = reinterpret_cast<float4 *>(a.acc + at);
    float4 lo = make_float4(r[0], r[1], r[2], r[3]), hi = make_float4(r[4], r[5], r[6], r[7]);
    if (a.accumulate) {
        const float4 x = p[0], y = p[1];
        lo = make_float4(__fadd_rn(x.x, lo.x), __fadd_rn(x.y, lo.y), __fadd_rn(x.z, lo.z), __fadd_rn(x.w, lo.w));
        hi = make_float4(__fadd_rn(y.x, hi.x), __fadd_rn(y.y, hi.y), __fadd_rn(y.z, hi.z), __fadd_rn(y.w, hi.w));
    }
    p[0] = lo;
    p[1] = hi;
}

// A piece of a longer run: leave its sum, and climb the run's tree while this
// warp brings the last child of the node.  A call of its own: inlined, its
// registers made the sums spill.
__device__ __noinline__ void climb(const SumArgs &a, const int4 *tree, int token, int index, int col, float4 lo,
                                   float4 hi) {
    const int4 t = __ldcg(tree);
    const int pieces = t.x;
    int slot = t.y, node = t.z;
    const bool live = col < a.D;
    float s[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int lane = threadIdx.x & 31, groups = gridDim.y, group = blockIdx.y;
    int count = pieces;  // of the level
    for (;;) {
        float *q = a.partial + (long long)(slot + index) * a.D + col;
        if (live) {
            __stcg(reinterpret_cast<float4 *>(q), make_float4(s[0], s[1], s[2], s[3]));
            __stcg(reinterpret_cast<float4 *>(q + 4), make_float4(s[4], s[5], s[6], s[7]));
        }
        const int parent = index / kFan, children = min(kFan, count - parent * kFan);
        __threadfence();
        __syncwarp();
        int seen = 0;
        if (lane == 0) seen = atomicAdd(a.tickets + (long long)(node + parent) * groups + group, 1);
        if (__shfl_sync(0xFFFFFFFFu, seen, 0) + 1 < children) return;
        __threadfence();
        // the node's children in order, from +0
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = 0.0f;
        if (live) {
            const float *c = a.partial + (long long)(slot + parent * kFan) * a.D + col;
            for (int k0 = 0; k0 < children; k0 += 4) {
                Floats8 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = Floats8();
                    if (k0 + k < children) load8(v[k], c + (long long)(k0 + k) * a.D);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) add8(s, v[k]);
            }
        }
        slot += count;
        count = (count + kFan - 1) / kFan;
        node += count;
        index = parent;
        if (count == 1) break;  // the root
    }
    if (live) put_row(a, token, col, s);
}

// A warp per (piece, 256 columns); blockIdx.y is the column group.
template <typename T, typename Vec, int U>
__global__ void __launch_bounds__(256, 4) embed_sum_kernel(const __grid_constant__ SumArgs a) {
    const int lane = threadIdx.x & 31;
    const int col = blockIdx.y * 256 + lane * 8;
    const bool live = col < a.D;
    // lanes behind the last column read along with the first and write nothing
    const T *d_out = static_cast<const T *>(a.d_out) + (live ? col : 0);
    pdl_wait();
    pdl_trigger();
    const int4 counts = __ldcg(reinterpret_cast<const int4 *>(a.counts));
    const int longs = counts.y, total = counts.x + longs;
    // the next piece's entry and places are loaded while this one's rows are
    const auto entry = [&](int i) {
        return reinterpret_cast<const int4 *>(a.pieces + (i < longs ? i : a.n - 1 - (i - longs)));
    };
    int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int step = gridDim.x * 8;
    if (i >= total) return;
    int4 p = __ldcg(entry(i));
    int mine = lane < p.z ? __ldcg(a.idx + p.y + lane) : 0;
#pragma unroll 1
    for (; i < total; i += step) {
        const int len = p.z;
        int4 p_next = p;
        if (i + step < total) p_next = __ldcg(entry(i + step));
        float s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = 0.0f;
#pragma unroll 1
        for (int r0 = 0; r0 < len; r0 += U) {
            Vec v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = __shfl_sync(0xFFFFFFFFu, mine, (r0 + u) & 31);
                v[u] = Vec();  // +0 behind the end: adding it changes no sum begun from +0
                if (r0 + u < len) load8(v[u], d_out + (long long)row * a.D);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) add8(s, v[u]);
        }
        mine = lane < p_next.z ? __ldcg(a.idx + p_next.y + lane) : 0;
        if (p.w >= 0)
            climb(a, entry(i) + 1, p.x, p.w, col, make_float4(s[0], s[1], s[2], s[3]),
                  make_float4(s[4], s[5], s[6], s[7]));
        else if (live)
            put_row(a, p.x, col, s);
        p = p_next;
    }
}

// Workspace.  A run of several pieces has at least 33 places, so all such runs
// together have at most 2 n / 33 pieces; each run's partial sums are at most
// 9/8 of its pieces, its nodes at most 1 + pieces / 8 (tree_size).
struct Layout {
    size_t counts, pieces, keys, idx, hist, tickets, partial, bytes;
};
Layout layout(int n, int D) {
    Layout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    };
    const size_t groups = (size_t)(D + 255) / 256, N = (size_t)n;
    l.counts = take(sizeof(Counts));
    l.pieces = take(N * sizeof(Piece));
    l.keys = take(N * 2 * sizeof(uint32_t));
    l.idx = take(N * 2 * sizeof(int));
    l.hist = take((size_t)kMaxTiles * kDigits * sizeof(int));
    l.tickets = take((N / 16 + 1) * groups * sizeof(int));
    l.partial = take((N * 9 / 128 + 2) * D * sizeof(float));
    l.bytes = at;
    return l;
}

int bit_length(unsigned v) {
    int b = 0;
    while (v >> b) ++b;
    return b;
}

// CTAs that zero `vecs` 16-byte vectors: 32 KB each, at most two an SM
int fill_ctas(long long vecs, int threads, const DeviceInfo &dev) {
    const long long c = (vecs + 2047) / 2048, most = 2ll * dev.sm_count * (1024 / threads);
    return (int)(c < most ? c : most);
}

template <int IPT>
cudaError_t sort_cta(const void *tokens, int is64, int n, int V, int bits, int digit_bits, int passes, int groups,
                     int *idx, Piece *pieces, int *tickets, Counts *counts, const Fill &fill, cudaStream_t stream,
                     const DeviceInfo &dev) {
    const size_t smem = sizeof(CtaShared) + (size_t)IPT * kCtaThreads * sizeof(uint32_t);
    const cudaError_t e = ensure_smem_attr((const void *)embed_sort_cta_kernel<IPT>, smem, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(embed_sort_cta_kernel<IPT>, dim3(1 + fill_ctas(fill.vecs, kCtaThreads, dev)), dim3(kCtaThreads),
                      smem, stream, tokens, is64, n, V, bits, digit_bits, passes, groups, idx, pieces, tickets, counts,
                      fill);
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
    uint32_t *keys = reinterpret_cast<uint32_t *>(base + l.keys);
    int *idx = reinterpret_cast<int *>(base + l.idx);
    int *tickets = reinterpret_cast<int *>(base + l.tickets);
    const int groups = (D + 255) / 256;
    const int key_bits = bit_length((unsigned)V), bits = n > 1 ? bit_length((unsigned)(n - 1)) : 1;  // keys are 0 .. V
    Fill fill = {d_table ? reinterpret_cast<uint4 *>(d_table) : reinterpret_cast<uint4 *>(d_table_acc),
                 accumulate ? 0 : (long long)V * D * (d_table ? 2 : 4) / 16};
    cudaError_t e = cudaSuccess;
    if (n <= kCtaTokens && key_bits + bits <= 32) {
        const int passes = (key_bits + 7) / 8, digit_bits = (key_bits + passes - 1) / passes;
        e = sort_cta<kCtaTokens / kCtaThreads>(tokens, tokens_are_64, n, V, bits, digit_bits, passes, groups,
                                               idx, pieces, tickets, counts, fill, stream, dev);
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
        // every launch zeroes an equal share
        const int passes = (key_bits + 7) / 8, launches = 2 * passes + 1;
        const long long share = (fill.vecs + launches - 1) / launches, end = fill.vecs;
        long long from = 0;
        auto next = [&]() {
            const Fill f = {fill.p + from, end - from < share ? end - from : share};
            from += f.vecs;
            return f;
        };
        for (int pass = 0; pass < passes; ++pass) {
            const int half = pass & 1;
            s.keys_in = pass == 0 ? nullptr : keys + (size_t)(1 - half) * n;
            s.idx_in = pass == 0 ? nullptr : idx + (size_t)(1 - half) * n;
            s.keys_out = keys + (size_t)half * n;
            s.idx_out = idx + (size_t)half * n;
            s.shift = 8 * pass;
            Fill f = next();
            e = launch_pdl(embed_hist_kernel, dim3(s.tiles + fill_ctas(f.vecs, 256, dev)), dim3(256), 0, stream, s, f);
            if (e != cudaSuccess) return e;
            f = next();
            e = launch_pdl(embed_scatter_kernel, dim3(s.tiles + fill_ctas(f.vecs, 256, dev)), dim3(256), 0, stream, s,
                           f);
            if (e != cudaSuccess) return e;
        }
        idx = s.idx_out;
        const Fill f = next();
        const int ctas = (n + 255) / 256;
        e = launch_pdl(embed_plan_kernel, dim3(ctas + fill_ctas(f.vecs, 256, dev)), dim3(256), 0, stream,
                       (const uint32_t *)s.keys_out, n, V, groups, pieces, tickets, counts, ctas, f);
        if (e != cudaSuccess) return e;
    }
    SumArgs a = {};
    a.d_out = d_out;
    a.idx = idx;
    a.pieces = pieces;
    a.counts = counts;
    a.tickets = tickets;
    a.partial = reinterpret_cast<float *>(base + l.partial);
    a.acc = d_table_acc;
    a.bf16 = d_table;
    a.scale = scale;
    a.accumulate = accumulate;
    a.n = n;
    a.D = D;
    // as many CTAs as the device holds, no more than pieces can be
    const int most = (n + 7) / 8, want = (4 * dev.sm_count + groups - 1) / groups;
    const dim3 grid(most < want ? most : want, groups);
    if (sizeof(T) == 2) return launch_pdl(embed_sum_kernel<uint16_t, uint4, 8>, grid, dim3(256), 0, stream, a);
    return launch_pdl(embed_sum_kernel<float, Floats8, 4>, grid, dim3(256), 0, stream, a);
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
