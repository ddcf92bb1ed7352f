// Embedding lookup with scaling, and the table's gradient (contract:
// include/adaln_ops.h).
//
//   out[i] = scale * table[t_i];   dT[v] = scale * sum over i, t_i = v, of d_out[i]
//
// Both are bound by HBM: rows read and rows written.  The gradient groups the
// tokens first, so that every row of d_out is read once, every row of dT has
// one owner, and no floating-point atomic decides an order:
//   1. a stable radix sort of (token, place), at most 8 bits a pass: in the
//      shared memory of one CTA or of a cluster where a token and a place fit 32
//      bits together, otherwise by a histogram and a scatter kernel a pass;
//   2. runs of more than 32 equal tokens are listed in pieces of 32 places.
//      Which list entry a piece gets is left to an integer atomic: it decides
//      who computes the piece, not what;
//   3. a warp takes a piece, or the shorter runs that begin among some
//      consecutive places, at 256 columns, and adds each run's rows in ascending
//      order, up to 15 rows (bf16; 7 of fp32) in flight whatever the runs' lengths.
//      A short run's row is written at once.  The pieces of a long run are the leaves of a 32-way
//      tree: whoever brings the last child of a node adds the children in order
//      (a ticket per node; nobody waits).
// Sorting is a chain of latencies that leaves the memory idle, so the table is
// zeroed meanwhile, by the other CTAs of the sorting launches; step 3 then
// writes the rows of tokens that occur.
#include "common.cuh"
#include "ops.h"

namespace adaln {

namespace {

constexpr int kTeamThreads = 1024;
constexpr int kPiece = 32;        // places of a piece
constexpr int kFan = 32;          // children of a node
constexpr int kDigits = 256;      // at most 8 bits a pass
constexpr int kTileMin = 1024;    // tokens of a CTA in the sort by kernels
constexpr int kMaxTiles = 256;    // ... and the number of such CTAs

// One piece of a long run.  The run has a partial sum for every piece and every
// node below the root, level by level from `slot`, and a ticket (per column
// group) for every node, level by level from `node`.
struct __align__(16) Piece {
    int token, start, len, index;  // index: which piece of the run
    int pieces, slot, node, unused;
};
struct Counts {
    int pieces, slots, nodes;
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
// lookup: a warp takes 4 vectors of 16 bytes a lane of one row.  Past L1, and out
// of L2 first: 16383 rows of 2048 fp32 take 30.1 us (182 MB, 6.1 TB/s), 31.9
// without.
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
            if (real && v0 + 32 * j < vecs) v[j] = __ldcg(src + v0 + 32 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v0 + 32 * j < vecs) __stcs(dst + v0 + 32 * j, real ? scale16(v[j], scale, T()) : v[j]);
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
// long runs of the sorted tokens
// --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t cluster_load(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Items token << bits | place in the shared memory of the C CTAs of a team,
// 1 << shift in each.
template <int C>
struct TeamKeys {
    const uint32_t *items;
    int bits, shift;
    __device__ uint32_t operator()(int i) const {
        if (C == 1) return items[i] >> bits;
        return cluster_load(cluster_addr(smem_u32(items + (i & ((1 << shift) - 1))), i >> shift)) >> bits;
    }
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

// The pieces of the long run that begins among the warp's 32 places base +
// lane, if one does (it covers every place behind its first, so there is one at
// most).
template <typename Keys>
__device__ void plan_places(const Keys &keys, int n, int V, int base, int groups, Piece *pieces, int *tickets,
                            Counts *counts) {
    const int lane = threadIdx.x & 31, i = base + lane;
    const uint32_t key = i < n ? keys(i) : 0xFFFFFFFFu;
    const uint32_t ahead = i + kPiece < n ? keys(i + kPiece) : 0xFFFFFFFFu;
    uint32_t prev = __shfl_up_sync(0xFFFFFFFFu, key, 1);
    if (lane == 0 && i > 0 && i < n) prev = keys(i - 1);
    const bool head = i < n && key < (uint32_t)V && (i == 0 || prev != key);
    const unsigned longs = __ballot_sync(0xFFFFFFFFu, head && ahead == key);
    if (longs == 0) return;
    const int src = __ffs(longs) - 1, start = base + src;
    const int token = __shfl_sync(0xFFFFFFFFu, (int)key, src);
    const int len = run_end(keys, n, start + kPiece + 1, (uint32_t)token) - start, np = (len + kPiece - 1) / kPiece;
    int slots, nodes, at = 0, slot = 0, node = 0;
    tree_size(np, slots, nodes);
    if (lane == 0) {
        at = atomicAdd(&counts->pieces, np);
        slot = atomicAdd(&counts->slots, slots);
        node = atomicAdd(&counts->nodes, nodes);
    }
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
    slot = __shfl_sync(0xFFFFFFFFu, slot, 0);
    node = __shfl_sync(0xFFFFFFFFu, node, 0);
    int4 *out = reinterpret_cast<int4 *>(pieces);
    for (int p = lane; p < np; p += 32) {
        out[2 * (at + p)] = make_int4(token, start + p * kPiece, min(kPiece, len - p * kPiece), p);
        out[2 * (at + p) + 1] = make_int4(np, slot, node, 0);
    }
    for (long long k = lane; k < (long long)nodes * groups; k += 32) tickets[(long long)node * groups + k] = 0;
}

// --------------------------------------------------------------------------
// sorting in shared memory: a team of one CTA, or of a cluster of 8, with IPT
// items a thread.  CTA r of the team holds the places [r PER, (r + 1) PER) of
// every pass, PER = 1024 IPT, and its warp w 32 IPT of them.  Each pass counts
// the digits, shares the counts over the team, and sends every item to its
// place in the team's memory.  The other CTAs of the grid zero the table.
// --------------------------------------------------------------------------
constexpr int kCntStride = kDigits + 1;  // keeps the scan's reads in different banks
struct TeamShared {
    int cnt[32][kCntStride];  // per warp and digit: the count, then the next place
    int hist[kDigits];        // the CTA's counts, read by the team
    int sums[32];
    Counts counts;
    uint32_t items[1];  // [IPT * 1024]
};

template <int C>
__device__ __forceinline__ void team_sync() {
    if (C == 1) {
        __syncthreads();
    } else {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

template <int C, int IPT>
__device__ __forceinline__ void
team_sort(const void *tokens, int is64, int n, int V, int bits, int digit_bits, int passes, int groups, uint32_t *keys_out,
          int *idx_out, Piece *pieces, int *tickets, Counts *counts, const Fill &fill) {
    extern __shared__ __align__(16) unsigned char raw[];
    TeamShared &sh = *reinterpret_cast<TeamShared *>(raw);
    constexpr int PER = kTeamThreads * IPT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = C == 1 ? 0 : (int)blockIdx.x % C;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x >= C) {
        fill_zero(fill, blockIdx.x - C, gridDim.x - C);
        return;
    }
    const int local = warp * (32 * IPT) + lane;  // the thread's places: local + 32 j of the CTA's
    const int nd = 1 << digit_bits;
    uint32_t item[IPT];
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const int i = team * PER + local + 32 * j;
        item[j] = i < n ? token_key(tokens, is64, i, V) << bits | i : 0xFFFFFFFFu;  // behind the end: last
    }
    if (threadIdx.x == 0) {
        sh.counts = Counts{0, 0, 0};
        if (C > 1 && team == 0) *counts = Counts{0, 0, 0};
    }
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = bits + pass * digit_bits;
        for (int d = lane; d < nd; d += 32) sh.cnt[warp][d] = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < IPT; ++j) atomicAdd(&sh.cnt[warp][(item[j] >> shift) & (nd - 1)], 1);
        __syncthreads();
        // thread 4 d + q: the counts of digit d in the warps 8 q .. 8 q + 7
        const int d = threadIdx.x >> 2, q = threadIdx.x & 3;
        int c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = d < nd ? sh.cnt[8 * q + k][d] : 0;
            sum += c[k];
        }
        int upto = sum;  // inclusive over the quad
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            if (q >= off) upto += o;
        }
        int total = __shfl_sync(0xFFFFFFFFu, upto, lane | 3), before = 0;  // of the digit: all, and before this CTA
        if (C > 1) {
            if (q == 0 && d < nd) sh.hist[d] = total;
            team_sync<C>();
            total = 0;
            if (d < nd) {
#pragma unroll
                for (int k = 0; k < C / 4; ++k) {
                    const int r = q * (C / 4) + k;
                    const int h = (int)cluster_load(cluster_addr(smem_u32(&sh.hist[d]), r));
                    total += h;
                    before += r < team ? h : 0;
                }
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                total += __shfl_xor_sync(0xFFFFFFFFu, total, off);
                before += __shfl_xor_sync(0xFFFFFFFFu, before, off);
            }
        }
        // exclusive scan over the digits, one value a quad
        int inc = q == 0 ? total : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) sh.sums[warp] = inc;
        __syncthreads();
        int first = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.sums[lane] : 0) + inc - total;
        first = __shfl_sync(0xFFFFFFFFu, first, lane & ~3) + before + upto - sum;
        if (d < nd) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sh.cnt[8 * q + k][d] = first;
                first += c[k];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) {
            const int digit = (item[j] >> shift) & (nd - 1);
            const unsigned peers = same_digit(digit, digit_bits);
            const int rank = __popc(peers & ((1u << lane) - 1));
            const int at = sh.cnt[warp][digit] + rank;
            __syncwarp();
            if (rank == 0) sh.cnt[warp][digit] = at + __popc(peers);
            __syncwarp();
            if (C == 1)
                sh.items[at] = item[j];
            else
                cluster_store(cluster_addr(smem_u32(&sh.items[at % PER]), at / PER), item[j]);
        }
        team_sync<C>();
        if (pass + 1 < passes) {
            // with C > 1 the next pass's first barrier keeps others from writing here before this is read
#pragma unroll
            for (int j = 0; j < IPT; ++j) item[j] = sh.items[local + 32 * j];
            if (C == 1) __syncthreads();
        }
    }
    const uint32_t mask = (1u << bits) - 1u;
    const int mine = min(PER, n - team * PER);  // may be negative
    for (int i = threadIdx.x; i < mine; i += kTeamThreads) {
        keys_out[team * PER + i] = sh.items[i] >> bits;
        idx_out[team * PER + i] = (int)(sh.items[i] & mask);
    }
    __syncwarp();
    const TeamKeys<C> keys{sh.items, bits, 31 - __clz(PER)};
    for (int i0 = warp * 32; i0 < mine; i0 += kTeamThreads)
        plan_places(keys, n, V, team * PER + i0, groups, pieces, tickets, C == 1 ? &sh.counts : counts);
    __syncwarp();
    team_sync<C>();  // nobody leaves while its memory is read
    if (C == 1 && threadIdx.x == 0) *counts = sh.counts;
}

template <int IPT>
__global__ void __launch_bounds__(kTeamThreads)
embed_sort_cta_kernel(const void *tokens, int is64, int n, int V, int bits, int digit_bits, int passes, int groups,
                      uint32_t *keys_out, int *idx_out, Piece *pieces, int *tickets, Counts *counts, const Fill fill) {
    team_sort<1, IPT>(tokens, is64, n, V, bits, digit_bits, passes, groups, keys_out, idx_out, pieces, tickets, counts,
                      fill);
}
template <int IPT>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kTeamThreads)
embed_sort_cluster_kernel(const void *tokens, int is64, int n, int V, int bits, int digit_bits, int passes, int groups,
                          uint32_t *keys_out, int *idx_out, Piece *pieces, int *tickets, Counts *counts,
                          const Fill fill) {
    team_sort<8, IPT>(tokens, is64, n, V, bits, digit_bits, passes, groups, keys_out, idx_out, pieces, tickets, counts,
                      fill);
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
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counts = Counts{0, 0, 0};
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
    __shared__ int joined[16][kDigits];
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
    // Digits 8 lane .. 8 lane + 7 in all CTAs and in those before this one: warp w
    // adds the CTAs w, w + 8, ..., then the warps are joined.
    int all[8] = {}, ahead[8] = {};
#pragma unroll 4
    for (int b = warp; b < a.tiles; b += 8) {
        const int4 *h = reinterpret_cast<const int4 *>(a.hist + b * kDigits + 8 * lane);
        const int4 x = __ldcg(h), y = __ldcg(h + 1);
        const int v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            all[k] += v[k];
            ahead[k] += b < (int)blockIdx.x ? v[k] : 0;
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        joined[warp][8 * lane + k] = all[k];
        joined[8 + warp][8 * lane + k] = ahead[k];
    }
    __syncthreads();
    int total = 0, before = 0;  // of digit d
    for (int w = 0; w < 8; ++w) {
        total += joined[w][d];
        before += joined[8 + w][d];
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
    const uint32_t *keys;
    const int *idx;
    const Piece *pieces;
    const Counts *counts;
    int *tickets;    // [nodes][groups]
    float *partial;  // [slots][D]
    float *acc;      // [V][D] fp32, or
    uint16_t *bf16;  // [V][D]
    float scale;
    int accumulate, n, V, D, groups;
    int places;  // of a task: 16 or 32
};

// 8 columns, added to a sum
struct Floats8 {
    float4 a, b;
};
__device__ __forceinline__ void add8(float (&s)[8], const Floats8 &v) {
    s[0] = __fadd_rn(s[0], v.a.x), s[1] = __fadd_rn(s[1], v.a.y);
    s[2] = __fadd_rn(s[2], v.a.z), s[3] = __fadd_rn(s[3], v.a.w);
    s[4] = __fadd_rn(s[4], v.b.x), s[5] = __fadd_rn(s[5], v.b.y);
    s[6] = __fadd_rn(s[6], v.b.z), s[7] = __fadd_rn(s[7], v.b.w);
}
// ... of a ring's row: one 16-byte word of bf16, or two of fp32, 512 bytes apart
__device__ __forceinline__ Floats8 ring_row(const uint16_t *p) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    return {make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y)),
            make_float4(bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w))};
}
__device__ __forceinline__ Floats8 ring_row(const float *p) {
    return {*reinterpret_cast<const float4 *>(p), *reinterpret_cast<const float4 *>(p + 128)};
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

// A piece of a long run: leave its sum, and climb the run's tree while this
// warp brings the last child of the node.
__device__ __forceinline__ void climb(const SumArgs &a, const int4 *tree, int token, int index, int group,
                                      int col, float (&s)[8]) {
    const int4 t = __ldcg(tree);
    int count = t.x, slot = t.y, node = t.z;  // of the level
    const bool live = col < a.D;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
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
        if (lane == 0) seen = atomicAdd(a.tickets + (long long)(node + parent) * a.groups + group, 1);
        if (__shfl_sync(0xFFFFFFFFu, seen, 0) + 1 < children) return;
        __threadfence();
        // the node's children in order, from +0
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = 0.0f;
        if (live) {
            const float *c = a.partial + (long long)(slot + parent * kFan) * a.D + col;
#pragma unroll 1
            for (int k0 = 0; k0 < children; k0 += 4) {
                Floats8 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = Floats8();  // +0 behind the end: adding it changes no sum begun from +0
                    if (k0 + k < children) {
                        const float4 *f = reinterpret_cast<const float4 *>(c + (long long)(k0 + k) * a.D);
                        v[k] = {__ldcg(f), __ldcg(f + 1)};
                    }
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

// A warp per (piece of a long run | short runs that begin at a.places places,
// 256 columns), the column groups of a task side by side.  A lane copies its 8
// columns of the task's rows asynchronously into a ring of its own, 8 KB a warp:
// all that the SM can have in flight, whatever the lengths of the runs.  (One
// run at a time, its rows in registers, took 40 us instead of 28 for 32768 rows
// of 1024 in runs of mostly one or two.)
constexpr int kSumWarps = 8;
constexpr int kRingBytes = 8192;  // of a warp

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(32 * kSumWarps, 3) embed_sum_kernel(const __grid_constant__ SumArgs a) {
    constexpr int R = kRingBytes / (256 * (int)sizeof(T));  // rows of the ring
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // row r at ring + (r % R) * 256: the lane's 8 columns in 16-byte words, fp32
    // two of them, 512 bytes apart
    T *ring = reinterpret_cast<T *>(ring_bytes + warp * kRingBytes);
    pdl_wait();
    pdl_trigger();
    const int longs = __ldcg(&a.counts->pieces), total = longs + (a.n + a.places - 1) / a.places;
#pragma unroll 1
    for (int id = blockIdx.x * kSumWarps + warp; id < total * a.groups; id += gridDim.x * kSumWarps) {
        const int task = id / a.groups, group = id - task * a.groups;
        const int col = group * 256 + lane * 8;
        const bool live = col < a.D;
        // lanes behind the last column read along with the first and write nothing
        const T *d_out = static_cast<const T *>(a.d_out) + (live ? col : 0);
        // the task's places: [begin, end) of the 64 from `base`, two a lane;
        // bit i of `heads`: a run begins at place base + i
        int base, begin = 0, end;
        unsigned long long heads = 1;
        int4 piece = make_int4(0, 0, 0, 0);
        uint32_t key = 0, key2 = 0;
        if (task < longs) {
            piece = __ldcg(reinterpret_cast<const int4 *>(a.pieces + task));
            base = piece.y;
            end = piece.z;
        } else {
            base = (task - longs) * a.places;
            key = base + lane < a.n ? __ldcg(a.keys + base + lane) : 0xFFFFFFFFu;
            key2 = base + 32 + lane < a.n ? __ldcg(a.keys + base + 32 + lane) : 0xFFFFFFFFu;
        }
        const int at = base + lane < a.n ? __ldcg(a.idx + base + lane) : 0;
        const int at2 = base + 32 + lane < a.n ? __ldcg(a.idx + base + 32 + lane) : 0;
        if (task >= longs) {
            uint32_t prev = __shfl_up_sync(0xFFFFFFFFu, key, 1), prev2 = __shfl_up_sync(0xFFFFFFFFu, key2, 1);
            const uint32_t key31 = __shfl_sync(0xFFFFFFFFu, key, 31);
            if (lane == 0) prev = base > 0 ? __ldcg(a.keys + base - 1) : 0xFFFFFFFFu, prev2 = key31;
            heads = __ballot_sync(0xFFFFFFFFu, key != prev) |
                    (unsigned long long)__ballot_sync(0xFFFFFFFFu, key2 != prev2) << 32;
            const unsigned long long mine = heads & ((1ull << a.places) - 1);
            if (mine == 0) continue;
            begin = __ffsll((long long)mine) - 1;
            const int last = 63 - __clzll((long long)mine);  // the last run begins here
            const unsigned long long behind = heads >> (last + 1);  // last < 32
            end = behind ? last + __ffsll((long long)behind) : 64;
            // a long last run, and padding (which sorts last), are left out
            if (end - last > kPiece) end = last;
            const int tokens = __popc(__ballot_sync(0xFFFFFFFFu, key < (uint32_t)a.V)) +
                               __popc(__ballot_sync(0xFFFFFFFFu, key2 < (uint32_t)a.V));
            end = min(end, tokens);
        }
        const auto copy = [&](int r) {  // place r of the task
            if (r < end) {
                const int row = __shfl_sync(0xFFFFFFFFu, r < 32 ? at : at2, r & 31);
                const T *src = d_out + (long long)row * a.D;
                T *dst = ring + (r % R) * 256 + lane * (16 / (int)sizeof(T));
#pragma unroll
                for (int j = 0; j < (int)sizeof(T) / 2; ++j)
                    cp_async16(dst + j * 128, src + j * (16 / (int)sizeof(T)));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int r = begin; r < begin + R - 1; ++r) copy(r);
        float s[8];
        int first = begin;  // of the current run
#pragma unroll 1
        for (int r = begin; begin < end; ++r) {
            if (r == end || ((heads >> r) & 1)) {
                if (r > begin) {
                    if (task < longs) {
                        climb(a, reinterpret_cast<const int4 *>(a.pieces + task) + 1, piece.x, piece.w, group, col, s);
                    } else {
                        const int token = (int)__shfl_sync(0xFFFFFFFFu, first < 32 ? key : key2, first & 31);
                        if (live) put_row(a, token, col, s);
                    }
                }
                if (r == end) break;
                first = r;
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = 0.0f;
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(R - 2) : "memory");
            const T *p = ring + (r % R) * 256 + lane * (16 / (int)sizeof(T));
            add8(s, ring_row(p));
            copy(r + R - 1);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}

// Workspace.  A long run has at least 33 places, so all long runs together have
// at most 2 n / 33 pieces; each run's partial sums are at most 9/8 of its pieces,
// its nodes at most 1 + pieces / 8 (tree_size).
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
    l.pieces = take((N * 2 / 33 + 1) * sizeof(Piece));
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

// C CTAs sort (C = 1 or 8), the others zero
template <int C, int IPT>
cudaError_t sort_team(const void *tokens, int is64, int n, int V, int bits, int digit_bits, int passes, int groups,
                      uint32_t *keys, int *idx, Piece *pieces, int *tickets, Counts *counts, const Fill &fill, cudaStream_t stream,
                      const DeviceInfo &dev) {
    const auto kernel = []() {
        if constexpr (C == 1)
            return embed_sort_cta_kernel<IPT>;
        else
            return embed_sort_cluster_kernel<IPT>;
    }();
    const size_t smem = sizeof(TeamShared) + (size_t)IPT * kTeamThreads * sizeof(uint32_t);
    const cudaError_t e = ensure_smem_attr((const void *)kernel, smem, dev);
    if (e != cudaSuccess) return e;
    const int zeroing = (fill_ctas(fill.vecs, kTeamThreads, dev) + C - 1) / C * C;
    return launch_pdl(kernel, dim3(C + zeroing), dim3(kTeamThreads), smem, stream, tokens, is64, n, V, bits,
                      digit_bits, passes, groups, keys, idx, pieces, tickets, counts, fill);
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
    // In shared memory where a token and a place fit 32 bits: 4 tokens a thread, by
    // one CTA (9.5 us at 4096; with 32 a thread 67 us at 32768) or by a cluster of 8.
    // Beyond, the kernels: with 16 a thread the cluster's call takes 49 us at 33000
    // and 64 at 75351, theirs 32 and 46.  Between, the cluster's call against theirs
    // in us from graphs, text of 1001 tokens x 64 columns: 20.6 / 22.7 at 4097, 23.8
    // / 25.5 at 8192, 27.6 / 30.2 at 20000, 30.0 / 30.9 at 32768; of 50021 tokens x
    // 1024: 30.0 / 37.6, 29.8 / 39.9, 40.8 / 50.7, 47.5 / 58.1.  Of 50021 x 64 they
    // are within 1.2 us of one another from 8192 to 24576.  A cluster's CTA holds 4096
    // places whatever n is, so at 5000 tokens two of its eight sort.
    if (n <= 8 * 4 * kTeamThreads && key_bits + bits <= 32) {
        const int passes = (key_bits + 7) / 8, digit_bits = (key_bits + passes - 1) / passes;
        auto sort = n <= 4 * kTeamThreads ? sort_team<1, 4> : sort_team<8, 4>;
        e = sort(tokens, tokens_are_64, n, V, bits, digit_bits, passes, groups, keys, idx, pieces, tickets, counts,
                 fill, stream, dev);
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
        keys = s.keys_out;
        idx = s.idx_out;
        const Fill f = next();
        const int ctas = (n + 255) / 256;
        e = launch_pdl(embed_plan_kernel, dim3(ctas + fill_ctas(f.vecs, 256, dev)), dim3(256), 0, stream,
                       (const uint32_t *)keys, n, V, groups, pieces, tickets, counts, ctas, f);
        if (e != cudaSuccess) return e;
    }
    SumArgs a = {};
    a.d_out = d_out;
    a.keys = keys;
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
    a.V = V;
    a.D = D;
    a.groups = groups;
    // as many CTAs as the device holds; 16 places a task (4096 labels of 3072
    // columns: 20 us against 23 with 8), or 32 where that still gives every warp
    // two tasks
    const long long want = 3 * dev.sm_count;
    a.places = (long long)n * groups >= 2 * 32 * want * kSumWarps ? 32 : 16;
    const long long most = (((long long)n / a.places + n / kPiece + 2) * groups + kSumWarps - 1) / kSumWarps;
    const dim3 grid((unsigned)(most < want ? most : want));
    const size_t smem = kSumWarps * kRingBytes;
    e = ensure_smem_attr((const void *)embed_sum_kernel<T>, smem, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(embed_sum_kernel<T>, grid, dim3(32 * kSumWarps), smem, stream, a);
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
