// The adapters' products on the tensor cores (lora.cuh says which calls).
//
// Each operand row is read once from memory and R is small, so all three are
// bound by memory; what matters is that the bytes flow without passing through
// registers where they need not.  shrink and grad read their rows by TMA into
// shared memory, from where tcgen05.mma takes them; only their small results
// leave tensor memory.  expand's rows come and leave by TMA as well; a thread adds
// to 64 bytes of a row at a time.  (With mma.sync, rows in registers: 37 instead of
// 31.5 us for 4222 rows of 9216 channels at rank 32, bound by issue.)
//
// h and e are held as three bf16 parts, whose sum is the fp32 number itself (below 2^-109
// it is within 2^-134, half of bf16's smallest number).  The
// gradients, which are fp32, take all three (two would leave 2.5e-6 of error, more
// than all the sums); out and dx are rounded to bf16 once more and take two (2^-17).
#include <algorithm>

#include "lora.cuh"
#include "tc.cuh"

namespace adaln {

static __device__ unsigned g_err_lora;

namespace {

__device__ __forceinline__ void report_error_lora(unsigned code) {
    if (code == kErrDrainFailed)
        atomicOr(&g_err_lora, code);
    else
        atomicCAS(&g_err_lora, 0u, code);
}

constexpr int kM = 128;        // MMA M: tokens (shrink), channels (grad)
constexpr int kBlk = 64;       // channels (shrink) or tokens (grad) of a block: 128 bytes of bf16
constexpr int kRowTile = kM * kBlk * 2;
constexpr int kMaxStages = 6;
constexpr uint64_t kDrainNs = 100000000ull;

struct TcBars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t done;
    uint64_t kept_full, kept_empty;
    uint32_t tmem;
    int abort;
#ifdef ADALN_TEST_WAIT_NEVER_NS
    uint64_t never;  // test builds: a barrier nothing arrives on
#endif
};
constexpr int kBarBytes = 256;
static_assert(sizeof(TcBars) <= kBarBytes, "barrier block");

// Shared-memory matrix descriptor in the 128-byte swizzled layout (version 1, mode
// 2).  K-major: rows of 128 bytes, groups of 8 rows `sbo` bytes apart, `lbo` not
// used.  M- or N-major: `lbo` from 64 rows of the operand to the next 64, `sbo`
// from 8 steps of k to the next 8.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16 with fp32 accumulators, bf16 operands, M = 128; a_mn: A is M-major
__host__ __device__ constexpr uint32_t f16_idesc(int n, bool a_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kM >> 4) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// `bar` gets an arrival once every MMA issued by this thread so far is done
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Waits until the SM has the columns.  A kernel lets the next one start
// (pdl_trigger) only after all its CTAs have theirs: a CTA of the next kernel holds
// its columns while it waits for this kernel's end, so one that came first could
// keep this kernel from ever getting them.
__device__ __forceinline__ void tmem_alloc(uint32_t *at, int cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, int cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
// 8 accumulator columns of this warp's 32 lanes (tmem_ld_done before they are used)
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}
// barrier `id` of `count` threads; is `flag` set in all of them?
__device__ __forceinline__ bool named_bar_and(int id, int count, bool flag) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
        "selp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)flag), "r"(id), "r"(count)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void bars_init(TcBars &sm, int acc_arrivals, int empty_arrivals = 1) {
    for (int s = 0; s < kMaxStages; ++s) {
        mbar_init(&sm.full[s], 1);
        mbar_init(&sm.empty[s], empty_arrivals);
    }
    for (int p = 0; p < 2; ++p) {
        mbar_init(&sm.acc_full[p], 1);
        mbar_init(&sm.acc_empty[p], acc_arrivals);
    }
    mbar_init(&sm.done, 1);
    mbar_init(&sm.kept_full, 1);
    mbar_init(&sm.kept_empty, 1);
    sm.abort = 0;
#ifdef ADALN_TEST_WAIT_NEVER_NS
    mbar_init(&sm.never, 1);
#endif
    fence_barrier_init();
}

// the first wait of the MMA warp, in test builds: it runs out of time
__device__ __forceinline__ bool first_wait(TcBars &sm) {
#ifdef ADALN_TEST_WAIT_NEVER_NS
    return mbar_wait_bounded(&sm.never, 0u, (uint64_t)(ADALN_TEST_WAIT_NEVER_NS));
#else
    (void)sm;
    return true;
#endif
}

// A pair as three bf16x2 words, whose halves' sums are a and b (an infinity or a NaN
// is the first part)
__device__ __forceinline__ void three_parts(float a, float b, uint32_t (&p)[3]) {
    auto rest = [](float v, float part) {
        const float r = __fsub_rn(v, part);
        return fabsf(r) <= 3.4e38f ? r : 0.0f;
    };
    p[0] = pack_bf16x2(a, b);
    a = rest(a, bf16lo(p[0])), b = rest(b, bf16hi(p[0]));
    p[1] = pack_bf16x2(a, b);
    p[2] = pack_bf16x2(__fsub_rn(a, bf16lo(p[1])), __fsub_rn(b, bf16hi(p[1])));
}

// --------------------------------------------------------------------------
// shrink.  A tile is 128 tokens of a sample (MMA M, K-major as they lie in
// memory) by the R ranks (MMA N), the channels in blocks of 64 through a ring of
// stages.  The channels are cut into ks contiguous ranges, fixed by their number
// alone, one for each CTA of a cluster; CTA q joins the ranks of slice q: the
// others write their accumulators of it into its shared memory, and it adds them
// in range order.  About 12 blocks a range give two CTAs an SM, with 90 KB in
// flight each, at 8192 tokens of 3072 channels.  At 4096 a CTA has 0.5 us to its sample's
// id, 2.7 to the first block, 4.2 at 5.6 TB/s, 0.7 to the last MMA's end, 1.8 for the join.
// (24 or 48 blocks a range, and rings of 225 KB: slower.  The blocks that the ring has no
// room for asked of memory at once: 1.6 us more, since the first ones come no sooner than
// the last.)
//
// The tensor core cuts off what it adds, so an accumulator takes kChain blocks, the
// next ones go to another beside it, and they are added with proper rounding: with one
// accumulator for a whole range the relative error of h grew with the channels, 7e-7 at
// 6144 (12 blocks), 2.1e-6 at 16384, 9.1e-6 at 65536 (3.5e-5 where all terms have one
// sign).  Accumulators that do not fit a CTA's share of the SM's tensor memory (all that
// share an SM find room for theirs: one that waits for columns holds up its cluster) are
// taken in passes (LONG), whose sums a thread keeps in registers.  (Forward of 4096 rows of
// 16384 channels at rank 128, three accumulators: 86.8 us, 84.7 with one; of 2048 rows of
// 65536 in three passes: 139 and 111, at rank 16 without passes 58.7 and 57.9.  The next
// pass's first blocks requested before this one's sums are taken: 144.)
//
// Roles (128 threads): warp 0 lane 0 the copies, warp 1 lane 0 the MMAs, then
// thread t holds token t.
// --------------------------------------------------------------------------
constexpr int kPartPitch = kM + 4;  // floats of a rank's tokens
constexpr int kChain = 12;          // blocks of channels that an accumulator takes

struct ShrinkArgs {
    const float *scale;
    const void *ids;
    int is64;
    const int *lens;
    uint16_t *h;
    int S, C, R, NA, Sp;
    int Rp;      // R rounded up to the MMA's multiple of 16
    int ks;      // channel ranges: cluster size, 1, 2, 4 or 8, a divisor of Rp
    int accs;    // accumulators of a pass
    int stages, tmem_cols;
};

template <bool LONG>
__global__ void __launch_bounds__(128)
lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                      const ShrinkArgs g) {
    extern __shared__ unsigned char tc_smem_raw[];
    const uint32_t raw = smem_u32(tc_smem_raw);
    unsigned char *ring = tc_smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int w_tile = g.Rp * kBlk * 2, stage_bytes = kRowTile + w_tile;
    float *part = reinterpret_cast<float *>(ring + (size_t)g.stages * stage_bytes);  // [ks][Rp / ks][kPartPitch]
    TcBars &sm = *reinterpret_cast<TcBars *>(part + (size_t)g.Rp * kPartPitch);
    volatile int *abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.y * kM, b = blockIdx.z;
    const uint32_t rank = g.ks > 1 ? cluster_rank() : 0u;
    const int KB = (g.C + kBlk - 1) / kBlk;
    const int kb0 = kb_begin(KB, g.ks, (int)rank), nkb = kb_begin(KB, g.ks, (int)rank + 1) - kb0;
    if (threadIdx.x == 0) {
        prefetch_map(&map_x), prefetch_map(&map_w);
        bars_init(sm, 1);
    }
    if (warp == 1) tmem_alloc(&sm.tmem, g.tmem_cols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    if (g.ks > 1) cluster_arrive();  // waited for where the others' shared memory is first written
    pdl_wait();
    pdl_trigger();  // not before every CTA holds its tensor memory (tmem_alloc)
    const int a = adapter_of(g.ids, g.is64, b, g.NA);
    const int n = rows_of(g.lens, b, g.S);
    // no adapter, or no row of this tile: nothing reads its state (the whole cluster leaves)
    if (a < 0 || t0 >= n) {
        if (g.ks > 1) cluster_wait();
        if (warp == 1) tmem_free(tmem, g.tmem_cols);
        return;
    }
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    // the accumulators of n blocks added up, ranks c .. c + 15 of this thread's token
    auto chains = [&](int n, int c, float (&f)[16], bool from_zero) {
        for (int q = 0; q * kChain < n; ++q) {
            uint32_t v[16];
            tmem_ld16(trow + (uint32_t)(q * g.Rp + c), v);
            tmem_ld_done();
#pragma unroll
            for (int k = 0; k < 16; ++k)
                f[k] = from_zero && q == 0 ? __uint_as_float(v[k]) : __fadd_rn(f[k], __uint_as_float(v[k]));
        }
    };
    float total[LONG ? kLoraMaxRank / 16 : 1][16];
    const int span = LONG ? g.accs * kChain : nkb;  // blocks of a pass
    bool ok = true;
    for (int pass = 0, i0 = 0; i0 < nkb; ++pass, i0 += span) {
        const int i1 = min(nkb, i0 + span);
        if (warp == 0 && lane == 0) {
            int issued = i0;
            for (int i = i0; i < i1; ++i) {
                const int s = i % g.stages;
                if (i >= g.stages && !mbar_wait_or_abort(&sm.empty[s], (uint32_t)(i / g.stages - 1) & 1u, abort_flag)) {
                    *abort_flag = 1;
                    break;
                }
                unsigned char *st = ring + (size_t)s * stage_bytes;
                mbar_arrive_expect_tx(&sm.full[s], (uint32_t)stage_bytes);
                tma_load_3d(st, &map_x, (kb0 + i) * kBlk, t0, b, &sm.full[s]);
                tma_load_3d(st + kRowTile, &map_w, (kb0 + i) * kBlk, 0, a, &sm.full[s]);
                issued = i + 1;
            }
            // every copy issued has landed before the CTA may leave
            for (int s = 0; s < g.stages && s < issued; ++s) {
                const int last = s + g.stages * ((issued - 1 - s) / g.stages);
                if (!mbar_wait_bounded(&sm.full[s], (uint32_t)(last / g.stages) & 1u, kDrainNs))
                    report_error_lora(kErrDrainFailed);
            }
        } else if (warp == 1 && lane == 0) {
            const uint32_t idesc = f16_idesc(g.Rp, false);
            if (LONG) tc_after_sync();  // the last pass's accumulators have been taken
            for (int i = i0; i < i1; ++i) {
                const int s = i % g.stages, q = (i - i0) / kChain;
                if ((i == 0 && !first_wait(sm)) ||
                    !mbar_wait_or_abort(&sm.full[s], (uint32_t)(i / g.stages) & 1u, abort_flag)) {
                    *abort_flag = 1;
                    break;
                }
                tc_after_sync();
                const uint32_t st = smem_u32(ring + (size_t)s * stage_bytes);
                const uint64_t ad = sw128_desc(st, 16, 1024), wd = sw128_desc(st + kRowTile, 16, 1024);
                const uint32_t acc = tmem + (uint32_t)(q * g.Rp);
#pragma unroll
                for (int k = 0; k < kBlk / 16; ++k)
                    mma_f16(acc, ad + 2u * k, wd + 2u * k, idesc, i - i0 > q * kChain || k > 0);
                mma_commit(&sm.empty[s]);
            }
            mma_commit(&sm.done);  // also after giving up: completes when every issued MMA has
        }

        ok = mbar_wait_or_abort(&sm.done, (uint32_t)pass & 1u, abort_flag) && !*abort_flag;
        if (!ok && threadIdx.x == 0) {
            report_error_lora(kErrLoraShrinkWait);
            if (!mbar_wait_bounded(&sm.done, (uint32_t)pass & 1u, kDrainNs)) report_error_lora(kErrDrainFailed);
        }
        ok = __syncthreads_and(ok);
        tc_after_sync();
        if (!ok) break;
        if (LONG) {
#pragma unroll
            for (int c = 0; c < kLoraMaxRank / 16; ++c)
                if (c * 16 < g.Rp) chains(i1 - i0, c * 16, total[c], pass == 0);
            tc_before_sync();
            __syncthreads();
        }
    }
    if (g.ks > 1) cluster_wait();  // the cluster's CTAs run: their shared memory may be written
    const int slice = g.Rp / g.ks;  // ranks of a CTA
    uint32_t at = g.ks > 1 ? map_to_rank(part + (int)rank * slice * kPartPitch + threadIdx.x, 0u)
                           : smem_u32(part + threadIdx.x);  // place of the next rank
    int q = 0, i = 0;
#pragma unroll(LONG ? kLoraMaxRank / 16 : 1)
    for (int c = 0; c < (LONG ? kLoraMaxRank : g.Rp); c += 16) {
        if (LONG && c >= g.Rp) break;
        float v[16];
        if constexpr (LONG) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = total[c / 16][k];
        } else {
            chains(nkb, c, v, true);
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2) {  // a slice is even
            st_cluster_f32(at, v[k]);
            st_cluster_f32(at + kPartPitch * 4, v[k + 1]);
            at += 2 * kPartPitch * 4;
            if ((i += 2) == slice && ++q < g.ks) {
                i = 0;
                at = map_to_rank(part + (int)rank * slice * kPartPitch + threadIdx.x, (uint32_t)q);
            }
        }
    }
    tc_before_sync();
    if (g.ks > 1)
        cluster_sync();
    else
        __syncthreads();
    // a thread joins 8 tokens of a rank: 16 bytes of each part of the state
    const float scale = g.scale[a];
    uint16_t *h = g.h + (size_t)b * 3 * g.R * g.Sp + t0;
    for (int k = threadIdx.x; ok && k < slice * (kM / 8); k += 128) {
        const int i = k / (kM / 8), t = k % (kM / 8) * 8, r = (int)rank * slice + i;
        if (r >= g.R || t0 + t >= g.Sp) continue;
        float s[8];
        for (int q = 0; q < g.ks; ++q) {
            const float4 *p = reinterpret_cast<const float4 *>(part + (q * slice + i) * kPartPitch + t);
            const float4 x = p[0], y = p[1];
            const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = q == 0 ? f[j] : __fadd_rn(s[j], f[j]);
        }
        if (t0 + t + 8 > n)  // rows past the sample's end: zero, which grad relies on
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (t0 + t + j >= n) s[j] = 0.0f;
        uint32_t w[4][3];
#pragma unroll
        for (int j = 0; j < 4; ++j) three_parts(__fmul_rn(scale, s[2 * j]), __fmul_rn(scale, s[2 * j + 1]), w[j]);
        uint16_t *dst = h + (size_t)r * g.Sp + t;
#pragma unroll
        for (int m = 0; m < 3; ++m)
            stg16(dst + (size_t)m * g.R * g.Sp, make_uint4(w[0][m], w[1][m], w[2][m], w[3][m]));
    }
    if (warp == 1) {
        tc_after_sync();
        tmem_free(tmem, g.tmem_cols);
    }
}

// --------------------------------------------------------------------------
// expand.  A tile is 128 tokens (MMA M) by 64 channels (MMA N).  The state
// [k][token] is A, M-major, the adapter [k][channel] B, N-major, both as they lie
// in memory; k runs over the 2 R rows of the state's first two parts, each part
// against the same R rows of the adapter.  (Where R is an odd multiple of 8, an
// instruction of k = 16 would wrap around them: they are copied twice.)
//
// As many CTAs as the device holds take every gridDim.x-th of the tiles that have
// rows, in the order of the channels, then the tokens: all end at the same time,
// whatever the samples' lengths, and those that run side by side move along the
// same rows.  A tile's base, state and adapter come by TMA into a stage of a ring;
// two accumulators; a thread adds row t's accumulators to the base in shared memory,
// from where the tile leaves by TMA.  A tile that the sample's end crosses leaves by
// row.  Above rank 64, where the state is the most of a stage, a CTA takes a run of
// tiles instead, and keeps the state of its tokens beside the ring (a forward call of
// 4593 rows, 64 and 2560 channels, with the state in the stages and so: 20.7 and 22.5 us
// at rank 64, 27.8 and 24.0 at 96, 30.1 and 26.8 at 128).  4222 rows of 9216 channels at
// rank 32 take 31.5 us, 5.0 TB/s.  (One tile a CTA, of 128 channels, four CTAs an SM,
// each waiting for its own copies: 36.5.  Each CTA a run of one row of tiles: 45, the last
// CTAs alone on the device.)
//
// Roles (320 threads): warp 0 finds the tiles and lane 0 copies, warp 1 lane 0 the
// MMAs, warps 2 to 5 and 6 to 9 every other tile, a token a thread.
// --------------------------------------------------------------------------
constexpr int kExThreads = 320;
constexpr int kExTile = kM * kBlk * 2;  // 16 KB: 64 channels of the base
constexpr int kExStages = 4;   // most; 2 or 4, so that a stage is always the same group's
constexpr int kExCtas = 3;     // most on an SM
static_assert(kExStages <= kMaxStages, "barriers");

enum BaseKind { kNoBase, kBaseByTma, kBaseByRow };

struct ExpandArgs {
    const void *ids;
    int is64;
    const int *lens;
    const uint16_t *base;
    long long base_batch, base_token;
    uint16_t *out;
    long long batch, token;
    int S, C, R, NA;
    int B;
    int copies;  // of the adapter's rows
    int kind;    // of the base
    int stages;
    int keep;    // the state lies beside the stages, for a run of tiles
};

struct ExpandTile {  // what a stage holds
    int b, t0, c0;
    int n;  // rows of the sample from t0 on; 0: there are no more tiles
    int a;  // adapter, -1: none
    int m;  // products before this one among the tiles of its group of warps
    int fresh;  // keep: the state of these tokens is to be loaded
};

// The tiles x, x + gridDim.x, ... of a call, or (keep) the x-th of gridDim.x runs of
// them, for a warp.  Without lens every sample has
// the same number of token tiles; with them the warp goes through the samples, 32 at
// a time.
struct ExpandTiles {
    const ExpandArgs &g;
    long long u, step, end;  // tile number
    int ct;             // channel tiles
    int w0;             // first sample of the window
    long long before;   // token tiles of the samples before it
    int rows, upto;     // this lane's sample: its rows, and the token tiles up to its end
    int next_rows;      // the next window's, on their way
    bool over;
    __device__ __forceinline__ ExpandTiles(const ExpandArgs &args, int lane)
        : g(args), u(blockIdx.x), step(gridDim.x), end(0x7FFFFFFFFFFFFFFFll), ct((args.C + kBlk - 1) / kBlk), w0(0),
          before(0), rows(0), upto(0), next_rows(0), over(false) {
        if (g.lens) first(lane);
        if (!g.keep) return;
        long long all = (long long)g.B * ((g.S + kM - 1) / kM);
        if (g.lens) {
            all = __shfl_sync(0xFFFFFFFFu, upto, 31);
            while (w0 + 32 < g.B) {
                w0 += 32;
                window(lane);
                all += __shfl_sync(0xFFFFFFFFu, upto, 31);
            }
            if (w0 > 0) w0 = 0, first(lane);
        }
        all *= ct;
        u = all * blockIdx.x / gridDim.x, end = all * (blockIdx.x + 1) / gridDim.x, step = 1;
    }
    __device__ __forceinline__ int rows_at(int b) const { return b < g.B ? rows_of(g.lens, b, g.S) : 0; }
    __device__ __forceinline__ void first(int lane) {
        next_rows = rows_at(lane);
        window(lane);
    }
    __device__ __forceinline__ void window(int lane) {
        rows = next_rows;
        next_rows = rows_at(w0 + 32 + lane);
        upto = (rows + kM - 1) / kM;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += v;
        }
    }
    // the next tile; after the last n == 0, as often as it is asked; the same in every lane
    __device__ __forceinline__ ExpandTile next(int lane) {
        ExpandTile t = {0, 0, 0, 0, -1, 0, 0};
        for (; !over; u += step) {
            if (u >= end) {
                over = true;
                break;
            }
            const long long tt = u / ct;  // token tile
            t.c0 = (int)(u - tt * ct) * kBlk;
            if (!g.lens) {
                const int per = (g.S + kM - 1) / kM;
                if (tt >= (long long)g.B * per) {
                    over = true;
                    break;
                }
                t.b = (int)(tt / per), t.t0 = (int)(tt - (long long)t.b * per) * kM, t.n = g.S - t.t0;
            } else {
                unsigned past;
                for (;;) {  // the first sample whose end lies beyond tt
                    past = __ballot_sync(0xFFFFFFFFu, before + upto > tt);
                    if (past || w0 + 32 >= g.B) break;
                    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
                    w0 += 32;
                    window(lane);
                }
                if (!past) {
                    over = true;
                    break;
                }
                const int i = __ffs(past) - 1, n = __shfl_sync(0xFFFFFFFFu, rows, i);
                const int end = __shfl_sync(0xFFFFFFFFu, upto, i);
                t.b = w0 + i, t.t0 = (int)(tt - before - (end - (n + kM - 1) / kM)) * kM, t.n = n - t.t0;
            }
            t.a = adapter_of(g.ids, g.is64, t.b, g.NA);
            if (t.a >= 0 || g.base != g.out) break;
            t.n = 0;  // in place without an adapter: nothing to do
        }
        u += step;
        return t;
    }
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// this thread's stores have read their shared memory
__device__ __forceinline__ void tma_store_read() {
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__global__ void __launch_bounds__(kExThreads, kExCtas)
lora_expand_tc_kernel(const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_o,
                      const ExpandArgs g) {
    extern __shared__ unsigned char tc_smem_raw[];
    __shared__ ExpandTile info[kExStages];
    const uint32_t raw = smem_u32(tc_smem_raw);
    unsigned char *ring = tc_smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int R = g.R, h_box = 2 * R * 128, w_rows = R * 128, w_tile = g.copies * w_rows;
    const int w_at = kExTile + (g.keep ? 0 : 2 * h_box), stage_bytes = w_at + w_tile;  // base, state, adapter
    unsigned char *kept = ring + (size_t)g.stages * stage_bytes;
    TcBars &sm = *reinterpret_cast<TcBars *>(kept + (g.keep ? 2 * h_box : 0));
    volatile int *abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_map(&map_h), prefetch_map(&map_w), prefetch_map(&map_y), prefetch_map(&map_o);
        bars_init(sm, 128, 2);
    }
    if (warp == 1) tmem_alloc(&sm.tmem, 2 * kBlk);
    pdl_wait();
    const bool by_tma = g.kind == kBaseByTma;
    tc_before_sync();
    __syncthreads();
    pdl_trigger();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    bool ok = true;
    if (warp == 0) {
        ExpandTiles tiles(g, lane);
        int issued = 0, products[2] = {0, 0}, b = -1, t0 = -1, loads = 0;  // keep: tokens of the state, loads of it
        for (int i = 0, ends = 0; ends < 2; ++i) {  // the end is told twice, once to each group of warps
            ExpandTile t = tiles.next(lane);
            t.m = i & 1 ? products[1] : products[0];
            if (t.n > 0 && t.a >= 0) (i & 1 ? products[1] : products[0]) += 1;
            ends += t.n == 0;
            t.fresh = t.n > 0 && t.a >= 0 && (t.b != b || t.t0 != t0);
            if (t.fresh) b = t.b, t0 = t.t0;
            const int s = i % g.stages;
            // free: the tile's MMAs are done, and its store has read it
            if (i >= g.stages)
                ok = ok && mbar_wait_or_abort(&sm.empty[s], (uint32_t)(i / g.stages - 1) & 1u, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                *abort_flag = 1;
                ok = false;
                break;
            }
            if (lane == 0) {
                unsigned char *p = ring + (size_t)s * stage_bytes;
                info[s] = t;
                const int bytes = t.n == 0 ? 0 : (by_tma ? kExTile : 0) + (t.a >= 0 ? stage_bytes - kExTile : 0);
                mbar_arrive_expect_tx(&sm.full[s], (uint32_t)bytes);
                if (t.n > 0 && by_tma) tma_load_3d(p, &map_y, t.c0, t.t0, t.b, &sm.full[s]);
                if (t.n > 0 && t.a >= 0) {
                    for (int k = 0; k < g.copies; ++k)
                        tma_load_3d(p + w_at + k * w_rows, &map_w, t.c0, 0, t.a, &sm.full[s]);
                    if (!g.keep)
                        for (int k = 0; k < 2; ++k)
                            tma_load_3d(p + kExTile + k * h_box, &map_h, t.t0 + k * kBlk, 0, t.b, &sm.full[s]);
                }
                if (g.keep && t.fresh) {
                    // once the MMAs that read the last tokens' state are done
                    if (loads > 0) ok = mbar_wait_or_abort(&sm.kept_empty, (uint32_t)(loads - 1) & 1u, abort_flag);
                    if (ok) {
                        mbar_arrive_expect_tx(&sm.kept_full, (uint32_t)(2 * h_box));
                        for (int k = 0; k < 2; ++k)
                            tma_load_3d(kept + k * h_box, &map_h, t.t0 + k * kBlk, 0, t.b, &sm.kept_full);
                        ++loads;
                    }
                }
            }
            issued = i + 1;
        }
        // every copy issued lands before the CTA leaves
        if (lane == 0 && loads > 0 && !mbar_wait_bounded(&sm.kept_full, (uint32_t)(loads - 1) & 1u, kDrainNs))
            report_error_lora(kErrDrainFailed);
        if (lane == 0)
            for (int s = 0; s < g.stages && s < issued; ++s) {
                const int last = s + g.stages * ((issued - 1 - s) / g.stages);
                if (!mbar_wait_bounded(&sm.full[s], (uint32_t)(last / g.stages) & 1u, kDrainNs))
                    report_error_lora(kErrDrainFailed);
            }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = f16_idesc(kBlk, true) | (1u << 16);  // B N-major
            bool go = first_wait(sm);
            for (int i = 0, loads = 0; go; ++i) {
                const int s = i % g.stages;
                go = mbar_wait_or_abort(&sm.full[s], (uint32_t)(i / g.stages) & 1u, abort_flag);
                if (!go || info[s].n == 0) break;
                const bool add = info[s].a >= 0;
                const int m = info[s].m, p = i & 1;  // an accumulator for each group
                const bool fresh = info[s].fresh;
                mbar_arrive(&sm.empty[s]);  // one of two; the other comes after the tile's accumulators were taken
                if (!add) continue;
                if (m > 0) go = mbar_wait_or_abort(&sm.acc_empty[p], (uint32_t)(m - 1) & 1u, abort_flag);
                if (go && g.keep && fresh) {
                    if (loads > 0) mma_commit(&sm.kept_empty);  // arrives when the MMAs so far are done
                    go = mbar_wait_or_abort(&sm.kept_full, (uint32_t)loads & 1u, abort_flag);
                    ++loads;
                }
                if (!go) break;
                tc_after_sync();
                const uint32_t at = smem_u32(ring + (size_t)s * stage_bytes);
                const uint64_t hd = sw128_desc(g.keep ? smem_u32(kept) : at + kExTile, (uint32_t)h_box, 1024),
                               wd = sw128_desc(at + (uint32_t)w_at, 0, 1024);
                for (int k = 0, r = 0; k < R / 8; ++k) {  // rows 16 k .. of the state, r .. of the adapter
                    mma_f16(tmem + (uint32_t)(p * kBlk), hd + (2048u >> 4) * k, wd + (uint32_t)(r * 128 >> 4), idesc,
                            k > 0);
                    r += 16;
                    if (r >= g.copies * R) r -= g.copies * R;
                }
                mma_commit(&sm.acc_full[p]);
            }
            if (!go) {
                *abort_flag = 1;
                // MMAs issued before may still be writing the accumulators
                mma_commit(&sm.done);
                if (!mbar_wait_bounded(&sm.done, 0u, kDrainNs)) report_error_lora(kErrDrainFailed);
            }
        }
    } else {
        const int t = (warp & 3) * 32 + lane;  // a warp reads the tensor memory of lanes 32 (warp mod 4) ..
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int group = (warp - 2) >> 2;
        const bool leads = (threadIdx.x - 64) % 128 == 0;
        for (int i = group;; i += 2) {
            const int s = i % g.stages;
            // the stages are even in number: this one's phases are all this group's
            ok = mbar_wait_or_abort(&sm.full[s], (uint32_t)(i / g.stages) & 1u, abort_flag);
            const ExpandTile e = info[s];
            const int p = group;
            if (ok && e.n > 0 && e.a >= 0)
                ok = mbar_wait_or_abort(&sm.acc_full[p], (uint32_t)e.m & 1u, abort_flag);
            // the group's warps go on, or give up, together
            if (!named_bar_and(1 + group, 128, ok)) {
                ok = false;
                *abort_flag = 1;
                break;
            }
            if (e.n == 0) break;
            const bool whole = e.n >= kM || e.t0 + e.n == g.S;  // no row of the tile is to be left alone
            unsigned char *tile = ring + (size_t)s * stage_bytes;
            const long long row = e.t0 + t;
            const uint16_t *y_row = g.base + e.b * g.base_batch + row * g.base_token + e.c0;
            uint16_t *o_row = g.out + e.b * g.batch + row * g.token + e.c0;
            tc_after_sync();
#pragma unroll
            for (int c = 0; c < kBlk; c += 32) {
                uint32_t v[32];
                if (e.a >= 0) {
                    tmem_ld32(trow + (uint32_t)(p * kBlk + c), v);
                    tmem_ld_done();
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    unsigned char *at = tile + t * 128 + (((c / 8 + q) ^ (t & 7)) << 4);  // the row's 128 bytes, swizzled
                    uint4 y = make_uint4(0u, 0u, 0u, 0u);
                    if (by_tma)
                        y = *reinterpret_cast<const uint4 *>(at);
                    else if (g.kind == kBaseByRow && t < e.n && e.c0 + c + q * 8 < g.C)
                        y = *reinterpret_cast<const uint4 *>(y_row + c + q * 8);
                    if (e.a >= 0) {
                        uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            yw[j] = px_to_bf16x2(px_add(px_bf16(yw[j]), px_make(__uint_as_float(v[q * 8 + 2 * j]),
                                                                               __uint_as_float(v[q * 8 + 2 * j + 1]))));
                        y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
                    }
                    if (whole)
                        *reinterpret_cast<uint4 *>(at) = y;
                    else if (t < e.n && e.c0 + c + q * 8 < g.C)
                        stg16(o_row + c + q * 8, y);
                }
            }
            if (e.a >= 0) {
                tc_before_sync();
                mbar_arrive(&sm.acc_empty[p]);
            }
            if (whole) fence_proxy_async_smem();
            named_bar(1 + group, 128);
            if (leads) {
                if (whole) {
                    tma_store_3d(&map_o, tile, e.c0, e.t0, e.b);
                    tma_store_read();
                }
                mbar_arrive(&sm.empty[s]);
            }
        }
        if (leads) tma_store_done();
    }
    tc_before_sync();
    ok = __syncthreads_and(ok && !*abort_flag);
    if (!ok && threadIdx.x == 0) report_error_lora(kErrLoraExpandWait);
    if (warp == 1) {
        tc_after_sync();
        tmem_free(tmem, 2 * kBlk);
    }
}

// --------------------------------------------------------------------------
// grad.  A tile is 128 channels (MMA M, read M-major as the rows lie in memory)
// by the 3 R rows of the state (MMA N, rounded up to 16, in two MMAs above 256); the
// tokens of a piece in blocks of 64 (the MMA's k) through a ring of stages.  The
// three parts' columns are added when they leave tensor memory.
//
// Schedules and order as on the CUDA cores: OWNER, every piece of an adapter in
// order by one CTA, with two accumulators (where they fit), so that one piece's
// leave while the next one's MMAs run, and the total in shared memory; otherwise as
// many CTAs as the device holds take every gridDim.x-th piece of every tile.  (A call for
// dA and dU alone on 4096 of 8192 rows of 3072 and 3072 channels at rank 16: 30 us with a
// CTA a piece or two, a quarter of it the last CTAs, 24.7 so; this kernel by itself reads
// 3.1 TB/s there.)  At rank 128 the state is three quarters of what a tile
// reads, from L2: 18 us for 3700 rows of 2048 and 2560 channels, 150 MB into shared memory.
// (Two tiles a CTA beside one state, 90 MB, two stages: 7 us more; 4 less only from 8192
// rows of 3072 channels on.)
//
// Roles (192 threads): warp 0 lane 0 the copies, warp 1 the MMAs (and zeros for
// the rows of a block past the sample's end, which may hold anything), warps 2
// to 5 a channel a thread.
// --------------------------------------------------------------------------
constexpr int kGradThreads = 192;

struct GradArgs {
    GradOperand o[2];
    const void *ids;
    int is64;
    const int *lens;
    int accumulate;
    int B, S, R, NA, pieces;
    int early; // what this kernel reads is there before the kernel it follows ends
    int Np;    // 3 R rounded up to 16
    int bufs;  // accumulators
    int stages, tmem_cols;
};

// The pieces x, x + step, ... among those that are (samples with an adapter, rows),
// for a warp: it goes through the samples 32 at a time, the next ones' ids and lengths
// on their way.
struct GradPieces {
    const GradArgs &g;
    int w0;           // first sample of the window
    long long before; // pieces of the samples before it
    int rows, upto;   // this lane's sample: its rows (0 without an adapter), and the pieces up to its end
    int next_rows;    // the same of the next window's
    __device__ __forceinline__ GradPieces(const GradArgs &args, int lane) : g(args), w0(0), before(0) {
        next_rows = rows_at(lane);
        window(lane);
    }
    __device__ __forceinline__ int rows_at(int b) const {
        return b < g.B && adapter_of<true>(g.ids, g.is64, b, g.NA) >= 0 ? rows_of<true>(g.lens, b, g.S) : 0;
    }
    __device__ __forceinline__ void window(int lane) {
        rows = next_rows;
        next_rows = rows_at(w0 + 32 + lane);
        upto = (rows + kLoraTcPiece - 1) / kLoraTcPiece;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += v;
        }
    }
    // piece u (u ascending from call to call): rows [s0, s1) of sample b; false: there are not that many
    __device__ __forceinline__ bool find(long long u, int lane, int &b, int &s0, int &s1) {
        unsigned past;
        for (;;) {  // the first sample whose end lies beyond u
            past = __ballot_sync(0xFFFFFFFFu, before + upto > u);
            if (past || w0 + 32 >= g.B) break;
            before += __shfl_sync(0xFFFFFFFFu, upto, 31);
            w0 += 32;
            window(lane);
        }
        if (!past) return false;
        const int i = __ffs(past) - 1, n = __shfl_sync(0xFFFFFFFFu, rows, i), end = __shfl_sync(0xFFFFFFFFu, upto, i);
        b = w0 + i;
        s0 = (int)(u - before - (end - (n + kLoraTcPiece - 1) / kLoraTcPiece)) * kLoraTcPiece;
        s1 = min(n, s0 + kLoraTcPiece);
        return true;
    }
};

template <bool OWNER>
__global__ void __launch_bounds__(kGradThreads)
lora_grad_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_e,
                    const __grid_constant__ CUtensorMap map_d, const __grid_constant__ CUtensorMap map_h,
                    const GradArgs g) {
    extern __shared__ unsigned char tc_smem_raw[];
    const uint32_t raw = smem_u32(tc_smem_raw);
    unsigned char *ring = tc_smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int R = g.R, Np = g.Np, h_tile = Np * kBlk * 2, stage_bytes = kRowTile + h_tile;
    float *total = reinterpret_cast<float *>(ring + (size_t)g.stages * stage_bytes);  // OWNER: [R][128]
    TcBars &sm = *reinterpret_cast<TcBars *>(reinterpret_cast<unsigned char *>(total) + (OWNER ? (size_t)R * kM * 4 : 0));
    __shared__ int found[kGradThreads];
    __shared__ int count[kGradThreads / 32];
    volatile int *abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = g.o[0].blocks + g.o[1].blocks;
    if (threadIdx.x == 0) {
        prefetch_map(&map_x), prefetch_map(&map_e), prefetch_map(&map_d), prefetch_map(&map_h);
        bars_init(sm, 128);
    }
    if (warp == 1) tmem_alloc(&sm.tmem, g.tmem_cols);
    if (!g.early) pdl_wait();
    tc_before_sync();
    __syncthreads();
    pdl_trigger();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;

    // warps 2 to 5: this thread's channel of a tile (a warp reads the tensor memory of lanes 32 (warp mod 4) ..)
    const int lane_row = (warp & 3) * 32 + lane;
    int blk = 0, unit = 0, issued = 0;  // blocks and pieces taken so far, by each role
    bool ok = true;
    const int Na = Np <= 256 ? Np : 256;  // columns of the first MMA; the second's, if any: Np - Na
    const uint32_t idesc = f16_idesc(Na, true), idesc_b = f16_idesc(Np - Na, true);

    // One piece: rows [s0, s1) of sample b, channels from c0 of operand o.  Each role does its part.
    auto piece = [&](const GradOperand &o, bool x_side, int c0, int b, int s0, int s1) {
        const int nblk = (s1 - s0 + kBlk - 1) / kBlk;
        const int p = unit % g.bufs, use = unit / g.bufs;  // accumulator
        if (warp == 0) {
            const CUtensorMap *map_src = x_side ? &map_x : &map_d, *map_state = x_side ? &map_e : &map_h;
            if (lane == 0)
                for (int k = 0; k < nblk; ++k, ++blk) {
                    const int st = blk % g.stages;
                    if (blk >= g.stages &&
                        !mbar_wait_or_abort(&sm.empty[st], (uint32_t)(blk / g.stages - 1) & 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    unsigned char *q = ring + (size_t)st * stage_bytes;
                    const int s = s0 + k * kBlk;
                    mbar_arrive_expect_tx(&sm.full[st], (uint32_t)stage_bytes);
                    tma_load_3d(q, map_src, c0, s, b, &sm.full[st]);
                    tma_load_3d(q + kRowTile / 2, map_src, c0 + kBlk, s, b, &sm.full[st]);
                    tma_load_3d(q + kRowTile, map_state, s, 0, b, &sm.full[st]);
                    if (Np > 256) tma_load_3d(q + kRowTile + h_tile / 2, map_state, s, Np / 2, b, &sm.full[st]);
                    issued = blk + 1;
                }
        } else if (warp == 1) {
            const uint32_t acc = tmem + (uint32_t)(p * Np);
            bool go = unit > 0 || first_wait(sm);
            if (use > 0) go = go && mbar_wait_or_abort(&sm.acc_empty[p], (uint32_t)(use - 1) & 1u, abort_flag);
            go = __all_sync(0xFFFFFFFFu, go);
            for (int k = 0; k < nblk && go; ++k, ++blk) {
                const int st = blk % g.stages;
                go = mbar_wait_or_abort(&sm.full[st], (uint32_t)(blk / g.stages) & 1u, abort_flag);
                go = __all_sync(0xFFFFFFFFu, go);
                if (!go) break;
                unsigned char *tile = ring + (size_t)st * stage_bytes;
                const int left = s1 - s0 - k * kBlk;
                if (left < kBlk && s1 < g.S) {
                    // rows past the sample's end: their state is zero, and zero times NaN is not
                    for (int z = left * 8 + lane; z < kBlk * 8; z += 32) {
                        stg16(tile + z * 16, make_uint4(0u, 0u, 0u, 0u));
                        stg16(tile + kRowTile / 2 + z * 16, make_uint4(0u, 0u, 0u, 0u));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    tc_after_sync();
                    const uint32_t at = smem_u32(tile);
                    // 16 tokens further: two groups of 8 rows of A, 32 bytes of B
                    const uint64_t ad = sw128_desc(at, kRowTile / 2, 1024), hd = sw128_desc(at + kRowTile, 16, 1024);
#pragma unroll
                    for (int q = 0; q < kBlk / 16; ++q) {
                        mma_f16(acc, ad + (2048u >> 4) * q, hd + 2u * q, idesc, k > 0 || q > 0);
                        if (Np > Na)
                            mma_f16(acc + (uint32_t)Na, ad + (2048u >> 4) * q,
                                    hd + (uint32_t)(Na * kBlk * 2 >> 4) + 2u * q, idesc_b, k > 0 || q > 0);
                    }
                    mma_commit(&sm.empty[st]);
                }
                __syncwarp();
            }
            if (!go) {
                *abort_flag = 1;
                ok = false;
            } else if (lane == 0) {
                mma_commit(&sm.acc_full[p]);
            }
        } else {
            ok = mbar_wait_or_abort(&sm.acc_full[p], (uint32_t)use & 1u, abort_flag) && !*abort_flag;
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                *abort_flag = 1;
            } else {
                tc_after_sync();
                if (!OWNER) pdl_wait();  // before the first store
                const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(p * Np);
                const int c = c0 + lane_row;
                float *dst = o.part + (b * (long long)g.pieces + s0 / kLoraTcPiece) * R * o.C + c;
                for (int r = 0; r < R; r += 8) {
                    uint32_t hi[8], mid[8], lo[8];
                    tmem_ld8(at + (uint32_t)r, hi);
                    tmem_ld8(at + (uint32_t)(R + r), mid);
                    tmem_ld8(at + (uint32_t)(2 * R + r), lo);
                    tmem_ld_done();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float v = __fadd_rn(__uint_as_float(hi[j]),
                                                  __fadd_rn(__uint_as_float(mid[j]), __uint_as_float(lo[j])));
                        if (OWNER) {
                            float *t = total + (r + j) * kM + lane_row;
                            *t = __fadd_rn(*t, v);
                        } else if (c < o.C) {
                            dst[(long long)(r + j) * o.C] = v;
                        }
                    }
                }
                tc_before_sync();
                mbar_arrive(&sm.acc_empty[p]);
            }
        }
        ++unit;
    };

    if constexpr (!OWNER) {
        GradPieces pieces(g, lane);
        for (long long u = blockIdx.x; __all_sync(0xFFFFFFFFu, ok); u += gridDim.x) {
            const long long v = u / tiles;
            const int tile = (int)(u - v * tiles);
            int b, s0, s1;
            if (!pieces.find(v, lane, b, s0, s1)) break;
            const bool x_side = tile < g.o[0].blocks;
            piece(g.o[x_side ? 0 : 1], x_side, (tile - (x_side ? 0 : g.o[0].blocks)) * kM, b, s0, s1);
        }
    } else {
        const bool x_side = (int)blockIdx.x < g.o[0].blocks;
        const GradOperand &o = g.o[x_side ? 0 : 1];
        const int c0 = ((int)blockIdx.x - (x_side ? 0 : g.o[0].blocks)) * kM, c = c0 + lane_row, a = blockIdx.y;
        bool any = false;
        for (int b0 = 0; b0 < g.B; b0 += kGradThreads) {
            // the samples of adapter a among the next ones, in order
            const int b = b0 + threadIdx.x;
            const bool mine = b < g.B && adapter_of<true>(g.ids, g.is64, b, g.NA) == a;
            const unsigned vote = __ballot_sync(0xFFFFFFFFu, mine);
            if (lane == 0) count[warp] = __popc(vote);
            __syncthreads();
            int before = 0, samples = 0;
            for (int w = 0; w < kGradThreads / 32; ++w) {
                if (w < warp) before += count[w];
                samples += count[w];
            }
            if (mine) found[before + __popc(vote & ((1u << lane) - 1u))] = b;
            __syncthreads();
            if (samples > 0 && !any) {
                any = true;
                if (warp >= 2)
                    for (int r = 0; r < R; ++r)
                        total[r * kM + lane_row] =
                            g.accumulate && c < o.C ? __ldcg(o.acc + ((long long)a * R + r) * o.C + c) : 0.0f;
            }
            for (int i = 0; i < samples && ok; ++i) {
                const int n = rows_of<true>(g.lens, found[i], g.S);
                for (int s0 = 0; s0 < n && ok; s0 += kLoraTcPiece)
                    piece(o, x_side, c0, found[i], s0, min(n, s0 + kLoraTcPiece));
            }
            // found[] is written again; a role that gave up takes the others with it
            ok = __syncthreads_and(ok && !*abort_flag);
            if (!ok) break;
        }
        pdl_wait();
        if (ok && warp >= 2 && c < o.C && (any || !g.accumulate))
            for (int r = 0; r < R; ++r)
                o.acc[((long long)a * R + r) * o.C + c] = any ? total[r * kM + lane_row] : 0.0f;
    }
    // every copy issued lands and every MMA ends before the CTA leaves
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < g.stages && s < issued; ++s) {
            const int last = s + g.stages * ((issued - 1 - s) / g.stages);
            if (!mbar_wait_bounded(&sm.full[s], (uint32_t)(last / g.stages) & 1u, kDrainNs))
                report_error_lora(kErrDrainFailed);
        }
    } else if (warp == 1 && lane == 0) {
        mma_commit(&sm.done);
        if (!mbar_wait_bounded(&sm.done, 0u, kDrainNs)) report_error_lora(kErrDrainFailed);
    }
    __syncwarp();
    pdl_wait();  // in every CTA: the next kernel takes this one's end for that of all before it
    tc_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) report_error_lora(kErrLoraGradWait);
    if (warp == 1) {
        tc_after_sync();
        tmem_free(tmem, g.tmem_cols);
    }
}

// --------------------------------------------------------------------------
// host side
// --------------------------------------------------------------------------
// A bf16 tensor [n2, n1, n0] with strides in elements (of dimensions of more than
// one index) as a TMA map of boxes box1 x 64, 128-byte swizzled; outside: zeros.
bool make_map_3d(CUtensorMap *m, const void *ptr, int64_t n0, int64_t n1, int64_t n2, int64_t st1, int64_t st2,
                 int box1) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    const int64_t dense = (n0 + 7) / 8 * 8;
    const cuuint64_t dims[3] = {(cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)(n1 > 1 ? st1 : dense) * 2, (cuuint64_t)(n2 > 1 ? st2 : dense) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kBlk, (cuuint32_t)box1, 1}, estr[3] = {1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int padded_tokens(int S) { return (S + 7) / 8 * 8; }

int tmem_columns(int need) {
    int cols = 32;
    while (cols < need) cols *= 2;
    return cols;
}

// CTAs of `smem` bytes that share an SM (228 KB, 1 KB of it taken by each, and up to
// 1 KB of static shared memory), at most 3
constexpr int kSmOfOne = 225 * 1024, kSmOfTwo = 112 * 1024, kSmOfThree = 74 * 1024;
int ctas_of(size_t smem) { return smem <= kSmOfThree ? 3 : smem <= kSmOfTwo ? 2 : 1; }

// stages of `bytes` beside `extra` bytes: as many as let `ctas` CTAs share an SM, or
// where that leaves fewer than three, one CTA less.  (Gradients of 4096 of 8192 rows,
// 3072 and 3072 channels, rank 16: 28.5 us with two CTAs, 24.7 with three, whose
// pieces are dealt more evenly; shrink's tiles are too few for three.)
int stages_for(int bytes, int extra, int ctas) {
    const int fixed = extra + kBarBytes + 1024;
    int n = ctas > 2 ? (kSmOfThree - fixed) / bytes : 0;
    if (n < 3) n = (kSmOfTwo - fixed) / bytes;
    if (n < 3) n = (kSmOfOne - fixed) / bytes;
    return n < kMaxStages ? n : kMaxStages;
}
static_assert(kRowTile + 3 * kLoraMaxRank * kBlk * 2 <= (225 * 1024 - kLoraMaxRank * kM * 4 - kBarBytes - 1024) / 2,
              "two stages at the largest rank");

}  // namespace

cudaError_t lora_tc_shrink(const adaln_rows &src, const void *W, const LoraCall &c, int C, void *h,
                           cudaStream_t stream, const DeviceInfo &dev) {
    ShrinkArgs g = {};
    g.scale = c.scale, g.ids = c.ids, g.is64 = c.ids_are_64, g.lens = c.lens, g.h = static_cast<uint16_t *>(h);
    g.S = c.S, g.C = C, g.R = c.R, g.NA = c.NA, g.Sp = padded_tokens(c.S);
    g.Rp = (c.R + 15) / 16 * 16;
    const int KB = (C + kBlk - 1) / kBlk;
    g.ks = KB <= 12 ? 1 : KB <= 24 ? 2 : KB <= 48 ? 4 : 8;
    const int stage = kRowTile + g.Rp * kBlk * 2, part = g.Rp * kPartPitch * 4;
    g.stages = stages_for(stage, part, 2);
    CUtensorMap map_x, map_w;
    if (!make_map_3d(&map_x, src.data, C, c.S, c.B, src.token, src.batch, kM) ||
        !make_map_3d(&map_w, W, C, c.R, c.NA, C, (int64_t)c.R * C, g.Rp))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)g.stages * stage + part + kBarBytes + 1024;
    // one CTA an SM (above rank 64: 195 KB and more, beside which no other kernel with
    // tensor memory fits), or two (no more: 92 KB and more each)
    const int cols = ctas_of(smem) == 1 ? 512 : 256;
    const int most = (KB + g.ks - 1) / g.ks, chains = (most + kChain - 1) / kChain;  // of a range
    const bool in_passes = chains * g.Rp > cols;
    g.accs = in_passes ? cols / g.Rp : chains;
    g.tmem_cols = tmem_columns(g.accs * g.Rp);
    auto kern = in_passes ? lora_shrink_tc_kernel<true> : lora_shrink_tc_kernel<false>;
    cudaError_t err = ensure_smem_attr((const void *)kern, smem, dev);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.ks, (unsigned)((c.S + kM - 1) / kM), (unsigned)c.B);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[3];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[1].val.sharedMemCarveout = (unsigned)cudaSharedmemCarveoutMaxShared;
    attr[2].id = cudaLaunchAttributeClusterDimension;
    attr[2].val.clusterDim.x = (unsigned)g.ks;
    attr[2].val.clusterDim.y = 1;
    attr[2].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 3;
    return cudaLaunchKernelEx(&cfg, kern, map_x, map_w, g);
}

cudaError_t lora_tc_expand(const void *h, const void *W, const LoraCall &c, int C, cudaStream_t stream,
                           const DeviceInfo &dev) {
    ExpandArgs g = {};
    g.ids = c.ids, g.is64 = c.ids_are_64, g.lens = c.lens;
    g.base = static_cast<const uint16_t *>(c.base.data), g.base_batch = c.base.batch, g.base_token = c.base.token;
    g.out = static_cast<uint16_t *>(c.out.data), g.batch = c.out.batch, g.token = c.out.token;
    g.S = c.S, g.C = C, g.R = c.R, g.NA = c.NA;
    g.copies = c.R % 16 == 0 ? 1 : 2;
    // a broadcast base has strides that no tensor map takes
    const bool broadcast = (c.B > 1 && c.base.batch == 0) || (c.S > 1 && c.base.token == 0);
    g.kind = !g.base ? kNoBase : broadcast ? kBaseByRow : kBaseByTma;
    const int Sp = padded_tokens(c.S);
    CUtensorMap map_h, map_w, map_y, map_o;
    // the first two parts of the state: 2 R of its 3 R rows; without adapters nothing reads it or them
    const void *any = c.out.data;
    if (!make_map_3d(&map_h, c.NA > 0 ? h : any, Sp, 2 * c.R, c.B, Sp, (int64_t)3 * c.R * Sp, 2 * c.R) ||
        !make_map_3d(&map_w, c.NA > 0 ? W : any, C, c.R, c.NA > 0 ? c.NA : 1, C, (int64_t)c.R * C, c.R) ||
        !make_map_3d(&map_o, c.out.data, C, c.S, c.B, c.out.token, c.out.batch, kM) ||
        !(g.kind == kBaseByTma ? make_map_3d(&map_y, c.base.data, C, c.S, c.B, c.base.token, c.base.batch, kM)
                               : make_map_3d(&map_y, c.out.data, C, c.S, c.B, c.out.token, c.out.batch, kM)))
        return cudaErrorInvalidValue;
    g.B = c.B;
    g.keep = c.R > 64;
    const int state = 4 * c.R * 128, stage = kExTile + g.copies * c.R * 128 + (g.keep ? 0 : state);
    const int beside = (g.keep ? state : 0) + kBarBytes + 1024;
    // 2 or 4 stages, whichever gives an SM more of them in all: 8 up to rank 16, 6 up
    // to 32, 4 beyond, but 2 at ranks 56 and 120, whose adapter rows are there twice
    // (4608 rows of 3072 and 3072 channels, forward: rank 48 28.9 us, 56 34.9, 64 30.1,
    // 112 34.2, 120 40.9, 128 36.0)
    int per_sm = 0;
    for (int n = 2; n <= kExStages; n += 2) {
        const int ctas = std::min(kExCtas, 228 * 1024 / (n * stage + beside + 1024));
        if (n * ctas > g.stages * per_sm) g.stages = n, per_sm = ctas;
    }
    const size_t smem = (size_t)g.stages * stage + beside;
    const long long most = (long long)((C + kBlk - 1) / kBlk) * ((c.S + kM - 1) / kM) * c.B,
                    room = (long long)per_sm * dev.sm_count;
    cudaError_t err = ensure_smem_attr((const void *)lora_expand_tc_kernel, smem, dev);
    if (err != cudaSuccess) return err;
    return launch_pdl(lora_expand_tc_kernel, dim3((unsigned)std::min(most, room)), dim3(kExThreads), smem, stream,
                      map_h, map_w, map_y, map_o, g);
}

cudaError_t lora_tc_grads(const GradOperand &o0, const GradOperand &o1, const LoraCall &c, bool in_parts,
                          cudaStream_t stream, const DeviceInfo &dev) {
    GradArgs g = {};
    g.o[0] = o0, g.o[1] = o1;
    g.o[0].blocks = o0.acc ? (o0.C + kM - 1) / kM : 0;
    g.o[1].blocks = o1.acc ? (o1.C + kM - 1) / kM : 0;
    g.ids = c.ids, g.is64 = c.ids_are_64, g.lens = c.lens, g.accumulate = c.accumulate;
    g.B = c.B, g.S = c.S, g.R = c.R, g.NA = c.NA, g.pieces = (c.S + kLoraTcPiece - 1) / kLoraTcPiece;
    g.early = c.grads_early;
    g.Np = (3 * c.R + 15) / 16 * 16;
    const int stage = kRowTile + g.Np * kBlk * 2, extra = in_parts ? 0 : c.R * kM * 4;
    g.stages = stages_for(stage, extra, 3);
    const size_t smem = (size_t)g.stages * stage + extra + kBarBytes + 1024;
    const int per_sm = ctas_of(smem);
    // two accumulators where the SM's CTAs all find room for them: one that did not would wait for another's end
    g.bufs = 2 * g.Np <= 512 && tmem_columns(2 * g.Np) * per_sm <= 512 ? 2 : 1;
    g.tmem_cols = tmem_columns(g.bufs * g.Np);
    const int h_box = g.Np <= 256 ? g.Np : g.Np / 2;  // a box has at most 256 rows
    const int Sp = padded_tokens(c.S);
    CUtensorMap map_x, map_e, map_d, map_h;
    if (!make_map_3d(&map_x, o0.src, o0.C, c.S, c.B, o0.token, o0.batch, kBlk) ||
        !make_map_3d(&map_e, o0.h, Sp, 3 * c.R, c.B, Sp, (int64_t)3 * c.R * Sp, h_box) ||
        !make_map_3d(&map_d, o1.src, o1.C, c.S, c.B, o1.token, o1.batch, kBlk) ||
        !make_map_3d(&map_h, o1.h, Sp, 3 * c.R, c.B, Sp, (int64_t)3 * c.R * Sp, h_box))
        return cudaErrorInvalidValue;
    auto kern = in_parts ? lora_grad_tc_kernel<false> : lora_grad_tc_kernel<true>;
    cudaError_t err = ensure_smem_attr((const void *)kern, smem, dev);
    if (err != cudaSuccess) return err;
    const int tiles = g.o[0].blocks + g.o[1].blocks;
    const long long units = (long long)tiles * g.pieces * c.B, room = (long long)per_sm * dev.sm_count;
    const dim3 grid = in_parts ? dim3((unsigned)std::min(units, room)) : dim3((unsigned)tiles, (unsigned)c.NA);
    return launch_pdl(kern, grid, dim3(kGradThreads), smem, stream, map_x, map_e, map_d, map_h, g);
}

int read_and_clear_lora_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_err_lora, sizeof(v)) != cudaSuccess) return -1;
    if (v != 0 && cudaMemcpyToSymbol(g_err_lora, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return (int)v;
}

}  // namespace adaln
