// The adapters' products on the tensor cores (lora.cuh says which calls): bf16
// rows, more than 16 tokens a sample.
//
// Each operand row is read once from memory and R is small, so all three are
// bound by memory; what matters is that the bytes flow without passing through
// registers where they need not.  shrink and grad read their rows by TMA into
// shared memory, from where tcgen05.mma takes them; only their small results
// leave tensor memory.  expand adds a product of depth 2 R to rows that every
// element of must be touched anyway: its rows go through registers, as the
// accumulators of mma.sync in an order that makes each thread's eight columns
// contiguous.
//
// h and e are held as three bf16 parts, whose sum is the fp32 number itself.  The
// gradients, which are fp32, take all three (two would leave 2.5e-6 of error, more
// than all the sums); out and dx are rounded to bf16 once more and take two (2^-17).
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
__device__ __forceinline__ void tmem_ld4(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
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
__device__ __forceinline__ void bars_init(TcBars &sm, int acc_arrivals) {
    for (int s = 0; s < kMaxStages; ++s) {
        mbar_init(&sm.full[s], 1);
        mbar_init(&sm.empty[s], 1);
    }
    for (int p = 0; p < 2; ++p) {
        mbar_init(&sm.acc_full[p], 1);
        mbar_init(&sm.acc_empty[p], acc_arrivals);
    }
    mbar_init(&sm.done, 1);
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

// v as three bf16 parts (an infinity is the first)
__device__ __forceinline__ void three_parts(float v, uint16_t (&p)[3]) {
    p[0] = bf16_bits(v);
    p[1] = p[2] = 0;
    if ((p[0] & 0x7FFFu) == 0x7F80u) return;
    const float rest = __fsub_rn(v, bf16f(p[0]));
    p[1] = bf16_bits(rest);
    p[2] = bf16_bits(__fsub_rn(rest, bf16f(p[1])));
}

// --------------------------------------------------------------------------
// shrink.  A tile is 128 tokens of a sample (MMA M, K-major as they lie in
// memory) by the R ranks (MMA N), the channels in blocks of 64 through a ring of
// stages.  The channels are cut into ks contiguous ranges, fixed by their number
// alone, one for each CTA of a cluster; CTA q joins the ranks of slice q: the
// others write their accumulators of it into its shared memory, and it adds them
// in range order.  About 12 blocks a range give two CTAs an SM, with 90 KB in
// flight each, at 8192 tokens of 3072 channels.
//
// Roles (128 threads): warp 0 lane 0 the copies, warp 1 lane 0 the MMAs, then
// thread t holds token t.
// --------------------------------------------------------------------------
struct ShrinkArgs {
    const float *scale;
    const void *ids;
    int is64;
    const int *lens;
    uint16_t *h;
    int S, C, R, NA, Sp;
    int Rp;      // R rounded up to the MMA's multiple of 16
    int ks;      // channel ranges: cluster size, 1, 2, 4 or 8, a divisor of Rp / 4
    int stages, tmem_cols;
};

__global__ void __launch_bounds__(128)
lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                      const ShrinkArgs g) {
    extern __shared__ unsigned char tc_smem_raw[];
    const uint32_t raw = smem_u32(tc_smem_raw);
    unsigned char *ring = tc_smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int w_tile = g.Rp * kBlk * 2, stage_bytes = kRowTile + w_tile;
    float4 *part = reinterpret_cast<float4 *>(ring + (size_t)g.stages * stage_bytes);  // [ks][Rp / 4 / ks][128]
    TcBars &sm = *reinterpret_cast<TcBars *>(reinterpret_cast<unsigned char *>(part) + (size_t)g.Rp * kM * 4);
    volatile int *abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.y * kM, b = blockIdx.z;
    pdl_wait();
    pdl_trigger();
    const int a = adapter_of(g.ids, g.is64, b, g.NA);
    const int n = rows_of(g.lens, b, g.S);
    // no adapter, or no row of this tile: nothing reads its state (the whole cluster leaves)
    if (a < 0 || t0 >= n) return;
    const float scale = g.scale[a];
    const uint32_t rank = g.ks > 1 ? cluster_rank() : 0u;
    const int KB = (g.C + kBlk - 1) / kBlk;
    const int kb0 = kb_begin(KB, g.ks, (int)rank), nkb = kb_begin(KB, g.ks, (int)rank + 1) - kb0;
    if (threadIdx.x == 0) bars_init(sm, 1);
    if (warp == 1) tmem_alloc(&sm.tmem, g.tmem_cols);
    tc_before_sync();
    if (g.ks > 1)
        cluster_sync();  // also: the cluster's CTAs run, so their shared memory may be written
    else
        __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;

    if (warp == 0 && lane == 0) {
        int issued = 0;
        for (int i = 0; i < nkb; ++i) {
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
        for (int i = 0; i < nkb; ++i) {
            const int s = i % g.stages;
            if ((i == 0 && !first_wait(sm)) ||
                !mbar_wait_or_abort(&sm.full[s], (uint32_t)(i / g.stages) & 1u, abort_flag)) {
                *abort_flag = 1;
                break;
            }
            tc_after_sync();
            const uint32_t st = smem_u32(ring + (size_t)s * stage_bytes);
            const uint64_t ad = sw128_desc(st, 16, 1024), wd = sw128_desc(st + kRowTile, 16, 1024);
#pragma unroll
            for (int k = 0; k < kBlk / 16; ++k) mma_f16(tmem, ad + 2u * k, wd + 2u * k, idesc, i > 0 || k > 0);
            mma_commit(&sm.empty[s]);
        }
        mma_commit(&sm.done);  // also after giving up: completes when every issued MMA has
    }

    bool ok = mbar_wait_or_abort(&sm.done, 0u, abort_flag) && !*abort_flag;
    if (!ok && threadIdx.x == 0) {
        report_error_lora(kErrLoraShrinkWait);
        if (!mbar_wait_bounded(&sm.done, 0u, kDrainNs)) report_error_lora(kErrDrainFailed);
    }
    ok = __syncthreads_and(ok);
    tc_after_sync();
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const int slice = g.Rp / 4 / g.ks;  // ranks of a CTA, by four
    float4 *mine = part + (int)rank * slice * kM + threadIdx.x;
    for (int q = 0, c = 0; q < g.ks; ++q) {
        const uint32_t at = g.ks > 1 ? map_to_rank(mine, (uint32_t)q) : smem_u32(mine);
        for (int i = 0; i < slice; ++i, c += 4) {
            uint32_t v[4];
            tmem_ld4(trow + (uint32_t)c, v);
            tmem_ld_done();
            st_cluster_v4(at + (uint32_t)(i * kM * 16), make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]),
                                                                   __uint_as_float(v[2]), __uint_as_float(v[3])));
        }
    }
    tc_before_sync();
    if (g.ks > 1)
        cluster_sync();
    else
        __syncthreads();
    const int t = t0 + (int)threadIdx.x;
    if (ok && t < g.Sp) {
        uint16_t *h = g.h + (size_t)b * 3 * g.R * g.Sp + t;
        for (int i = 0; i < slice; ++i) {
            const int r = ((int)rank * slice + i) * 4;
            if (r >= g.R) break;
            float4 s = part[i * kM + threadIdx.x];
            for (int q = 1; q < g.ks; ++q) {
                const float4 v = part[(q * slice + i) * kM + threadIdx.x];
                s = make_float4(__fadd_rn(s.x, v.x), __fadd_rn(s.y, v.y), __fadd_rn(s.z, v.z), __fadd_rn(s.w, v.w));
            }
            const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint16_t p[3] = {0, 0, 0};  // rows past the sample's end: zero, which grad relies on
                if (t < n) three_parts(__fmul_rn(scale, f[j]), p);
#pragma unroll
                for (int k = 0; k < 3; ++k) h[(size_t)(k * g.R + r + j) * g.Sp] = p[k];
            }
        }
    }
    if (warp == 1) {
        tc_after_sync();
        tmem_free(tmem, g.tmem_cols);
    }
}

// --------------------------------------------------------------------------
// expand.  A CTA takes 256 channels of a run of tokens, 32 at a time; a warp 32
// channels.  With A the state [k][token] and B the adapter [k][channel], both
// transposed by ldmatrix; k runs over the 2 R rows of the state's first two parts,
// each part against the same R rows of the adapter.  Column n = 2 c + i of the MMA's tile j
// stands for channel 8 c + 2 j + i of the warp's 32, so that the accumulators of
// a thread are 8 consecutive channels of a token: one 16-byte load and store.
// The adapter's tile is permuted accordingly on its way into shared memory.
// --------------------------------------------------------------------------
constexpr int kExTok = 32;                 // tokens a warp multiplies at once, the next 32 requested before
constexpr int kExC = 256;                  // channels of a CTA
constexpr int kExWPitch = kExC * 2 + 16;   // bytes; 16 more, so that 8 rows lie in distinct banks
// tokens of a CTA, whose state stays in shared memory beside the adapter's tile:
// the more, the fewer times the tile is read, the fewer CTAs share an SM
__host__ __device__ constexpr int ex_run(int R) { return R <= 32 ? 256 : R <= 64 ? 128 : 64; }
__host__ __device__ constexpr int ex_h_pitch(int run) { return run * 2 + 16; }

__device__ __forceinline__ void ldsm_trans(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(256, 2)
lora_expand_tc_kernel(const uint16_t *__restrict__ h, const uint16_t *__restrict__ W, const void *ids, int is64,
                      const int *lens, const uint16_t *base, long long base_batch, long long base_token, uint16_t *out,
                      long long batch, long long token, int S, int Sp, int C, int R, int NA, int run) {
    extern __shared__ __align__(16) unsigned char ex_smem[];
    unsigned char *w_s = ex_smem, *h_s = ex_smem + (size_t)R * kExWPitch;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, s0 = blockIdx.y * run, c0 = blockIdx.x * kExC;
    const int h_pitch = ex_h_pitch(run);
    pdl_wait();
    pdl_trigger();
    const int n = min(rows_of(lens, b, S), s0 + run) - s0;
    if (n <= 0) return;
    const int a = adapter_of(ids, is64, b, NA);
    if (a < 0 && base == out) return;
    const int ch = c0 + warp * 32 + (lane & 3) * 8;  // this thread's channels
    const bool live = ch < C;
    const uint16_t *y_at = base + b * base_batch + (s0 + (lane >> 2)) * base_token + ch;
    uint16_t *o_at = out + b * batch + (s0 + (lane >> 2)) * token + ch;
    auto request = [&](int s, uint4 (&y)[2][2]) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                y[m][k] = make_uint4(0u, 0u, 0u, 0u);
                // not the read-only path: base may be out
                if (base && live && s + m * 16 + k * 8 + (lane >> 2) < n)
                    y[m][k] = *reinterpret_cast<const uint4 *>(y_at + (s + m * 16 + k * 8) * base_token);
            }
    };
    uint4 y[2][2], next[2][2];
    request(0, y);
    if (a >= 0) {
        const uint16_t *w = W + (long long)a * R * C;
        for (int i = threadIdx.x; i < R * (kExC / 8); i += 256) {
            const int r = i / (kExC / 8), v = i % (kExC / 8);  // 8 channels: c = v % 4 of strip v / 4
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (c0 + v * 8 < C) x = ldg16(w + (long long)r * C + c0 + v * 8);
            unsigned char *p = w_s + r * kExWPitch + (v >> 2) * 64 + (v & 3) * 4;
            *reinterpret_cast<uint32_t *>(p) = x.x;
            *reinterpret_cast<uint32_t *>(p + 16) = x.y;
            *reinterpret_cast<uint32_t *>(p + 32) = x.z;
            *reinterpret_cast<uint32_t *>(p + 48) = x.w;
        }
        const uint16_t *hp = h + (size_t)b * 3 * R * Sp + s0;
        const int vecs = (min(n, run) + 31) / 32 * 4;  // 8 tokens each, whole steps of 32
        for (int i = threadIdx.x; i < 2 * R * vecs; i += 256) {
            const int k = i / vecs, v = i - k * vecs;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (s0 + v * 8 < Sp) x = *reinterpret_cast<const uint4 *>(hp + (size_t)k * Sp + v * 8);
            *reinterpret_cast<uint4 *>(h_s + k * h_pitch + v * 16) = x;
        }
        __syncthreads();
    }
    if (c0 + warp * 32 >= C) return;
    const int blocks = R >> 3;
    const uint32_t ws = smem_u32(w_s) + (lane & 7) * kExWPitch + warp * 64 + (lane >> 3) * 16;
    const uint32_t hs = smem_u32(h_s) + ((lane >> 4) * 8 + (lane & 7)) * h_pitch + ((lane >> 3) & 1) * 16;
    for (int s = 0; s < n; s += kExTok) {
        request(s + kExTok, next);
        float acc[2][4][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[m][j][k] = 0.0f;
        if (a >= 0) {
            for (int k = 0, w0 = 0; k < blocks; ++k) {  // rows 16 k .. of the state, 8 w0 .. and 8 w1 .. of W
                const int w1 = w0 + 1 == blocks ? 0 : w0 + 1;
                uint32_t wa[4], wb[4];
                ldsm_trans(ws + w0 * 8 * kExWPitch, wa);
                ldsm_trans(ws + w1 * 8 * kExWPitch, wb);
                w0 = w1 + 1 == blocks ? 0 : w1 + 1;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t ha[4];
                    ldsm_trans(hs + k * 16 * h_pitch + (s + m * 16) * 2, ha);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_bf16(acc[m][j], ha, wa[j], wb[j]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (live && s + m * 16 + k * 8 + (lane >> 2) < n) {
                    const uint32_t yw[4] = {y[m][k].x, y[m][k].y, y[m][k].z, y[m][k].w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[j] = px_to_bf16x2(px_add(px_bf16(yw[j]), px_make(acc[m][j][2 * k], acc[m][j][2 * k + 1])));
                    stg16(o_at + (s + m * 16 + k * 8) * token, make_uint4(o[0], o[1], o[2], o[3]));
                }
                y[m][k] = next[m][k];
            }
    }
}

// --------------------------------------------------------------------------
// grad.  A tile is 128 channels (MMA M, read M-major as the rows lie in memory)
// by the 3 R rows of the state (MMA N, rounded up to 16, in two MMAs above 256); the
// tokens of a piece in blocks of 64 (the MMA's k) through a ring of stages.  The
// three parts' columns are added when they leave tensor memory.
//
// Schedules and order as lora_grad_kernel's: OWNER, every piece of an adapter in
// order by one CTA, with two accumulators (where they fit), so that one piece's
// leave while the next one's MMAs run, and the total in shared memory; otherwise a
// CTA a piece.
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
    int Np;    // 3 R rounded up to 16
    int bufs;  // accumulators
    int stages, tmem_cols;
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
    const bool first = (int)blockIdx.x < g.o[0].blocks;
    const GradOperand &o = g.o[first ? 0 : 1];
    const CUtensorMap *map_src = first ? &map_x : &map_d, *map_state = first ? &map_e : &map_h;
    const int c0 = ((int)blockIdx.x - (first ? 0 : g.o[0].blocks)) * kM;
    pdl_wait();
    pdl_trigger();
    int samples = 1, s_begin = 0, s_most = g.S;
    const int a = OWNER ? (int)blockIdx.y : adapter_of(g.ids, g.is64, blockIdx.z, g.NA);
    if (!OWNER) {
        s_begin = blockIdx.y * kLoraTcPiece;
        s_most = s_begin + kLoraTcPiece;
        if (a < 0 || s_begin >= rows_of(g.lens, blockIdx.z, g.S)) return;
    }
    if (threadIdx.x == 0) bars_init(sm, 128);
    if (warp == 1) tmem_alloc(&sm.tmem, g.tmem_cols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;

    // this thread's channel (warps 2 to 5; a warp reads the tensor memory of lanes 32 (warp mod 4) ..)
    const int lane_row = (warp & 3) * 32 + lane;
    const int c = c0 + lane_row;
    const bool holds = warp >= 2 && c < o.C;
    int blk = 0, unit = 0, issued = 0;  // blocks and pieces taken so far, by each role
    bool any = false, ok = true;
    const int Na = Np <= 256 ? Np : 256;  // columns of the first MMA; the second's, if any: Np - Na
    const uint32_t idesc = f16_idesc(Na, true), idesc_b = f16_idesc(Np - Na, true);

    for (int b0 = 0; b0 < (OWNER ? g.B : 1); b0 += kGradThreads) {
        if (OWNER) {
            // the samples of adapter a among the next ones, in order
            const int b = b0 + threadIdx.x;
            const bool mine = b < g.B && adapter_of(g.ids, g.is64, b, g.NA) == a;
            const unsigned vote = __ballot_sync(0xFFFFFFFFu, mine);
            if (lane == 0) count[warp] = __popc(vote);
            __syncthreads();
            int before = 0;
            samples = 0;
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
                            g.accumulate && c < o.C ? o.acc[((long long)a * R + r) * o.C + c] : 0.0f;
            }
        }
        for (int i = 0; i < samples && ok; ++i) {
            const int b = OWNER ? found[i] : (int)blockIdx.z;
            const int n = rows_of(g.lens, b, g.S);
            for (int s0 = s_begin; s0 < min(n, s_most) && ok; s0 += kLoraTcPiece, ++unit) {
                const int s1 = min(n, s0 + kLoraTcPiece), nblk = (s1 - s0 + kBlk - 1) / kBlk;
                if (warp == 0) {
                    if (lane == 0)
                        for (int k = 0; k < nblk; ++k, ++blk) {
                            const int st = blk % g.stages;
                            if (blk >= g.stages &&
                                !mbar_wait_or_abort(&sm.empty[st], (uint32_t)(blk / g.stages - 1) & 1u, abort_flag)) {
                                *abort_flag = 1;
                                ok = false;
                                break;
                            }
                            unsigned char *p = ring + (size_t)st * stage_bytes;
                            const int s = s0 + k * kBlk;
                            mbar_arrive_expect_tx(&sm.full[st], (uint32_t)stage_bytes);
                            tma_load_3d(p, map_src, c0, s, b, &sm.full[st]);
                            tma_load_3d(p + kRowTile / 2, map_src, c0 + kBlk, s, b, &sm.full[st]);
                            tma_load_3d(p + kRowTile, map_state, s, 0, b, &sm.full[st]);
                            if (Np > 256) tma_load_3d(p + kRowTile + h_tile / 2, map_state, s, Np / 2, b, &sm.full[st]);
                            issued = blk + 1;
                        }
                } else if (warp == 1) {
                    const int p = unit % g.bufs, use = unit / g.bufs;
                    const uint32_t acc = tmem + (uint32_t)(p * Np);
                    bool go = unit > 0 || first_wait(sm);
                    if (use > 0)
                        go = go && mbar_wait_or_abort(&sm.acc_empty[p], (uint32_t)(use - 1) & 1u, abort_flag);
                    go = __all_sync(0xFFFFFFFFu, go);
                    for (int k = 0; k < nblk && go; ++k, ++blk) {
                        const int st = blk % g.stages;
                        go = mbar_wait_or_abort(&sm.full[st], (uint32_t)(blk / g.stages) & 1u, abort_flag);
                        go = __all_sync(0xFFFFFFFFu, go);
                        if (!go) break;
                        unsigned char *tile = ring + (size_t)st * stage_bytes;
                        const int left = s1 - s0 - k * kBlk;
                        if (left < kBlk && s0 + k * kBlk + left < g.S) {
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
                            const uint64_t ad = sw128_desc(at, kRowTile / 2, 1024),
                                           hd = sw128_desc(at + kRowTile, 16, 1024);
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
                    const int p = unit % g.bufs;
                    ok = mbar_wait_or_abort(&sm.acc_full[p], (uint32_t)(unit / g.bufs) & 1u, abort_flag) &&
                         !*abort_flag;
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) {
                        *abort_flag = 1;
                    } else {
                        tc_after_sync();
                        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(p * Np);
                        float *dst = o.part + ((long long)(b * (long long)g.pieces + s0 / kLoraTcPiece) * R) * o.C + c;
                        for (int r = 0; r < R; r += 8) {
                            uint32_t hi[8], mid[8], lo[8];
                            tmem_ld8(at + (uint32_t)r, hi);
                            tmem_ld8(at + (uint32_t)(R + r), mid);
                            tmem_ld8(at + (uint32_t)(2 * R + r), lo);
                            tmem_ld_done();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float v = __fadd_rn(__uint_as_float(hi[j]), __fadd_rn(__uint_as_float(mid[j]),
                                                                                           __uint_as_float(lo[j])));
                                if (OWNER) {
                                    float *t = total + (r + j) * kM + lane_row;
                                    *t = __fadd_rn(*t, v);
                                } else if (holds) {
                                    dst[(long long)(r + j) * o.C] = v;
                                }
                            }
                        }
                        if (OWNER) {
                            tc_before_sync();
                            mbar_arrive(&sm.acc_empty[p]);
                        }
                    }
                }
            }
        }
        if (OWNER) {
            // found[] is written again; a role that gave up takes the others with it
            ok = __syncthreads_and(ok && !*abort_flag);
            if (!ok) break;
        }
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
    if (OWNER && ok && holds && (any || !g.accumulate))
        for (int r = 0; r < R; ++r) o.acc[((long long)a * R + r) * o.C + c] = any ? total[r * kM + lane_row] : 0.0f;
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

// stages of `bytes` beside `extra` bytes: as many as let two CTAs share an SM, or
// where that leaves fewer than three, as many as one CTA has room for
int stages_for(int bytes, int extra) {
    const int fixed = extra + kBarBytes + 1024;
    int n = (113 * 1024 - fixed) / bytes;
    if (n < 3) n = (225 * 1024 - fixed) / bytes;
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
    while (g.Rp / 4 % g.ks != 0) g.ks /= 2;
    const int stage = kRowTile + g.Rp * kBlk * 2, part = g.Rp * kM * 4;
    g.stages = stages_for(stage, part);
    g.tmem_cols = tmem_columns(g.Rp);
    CUtensorMap map_x, map_w;
    if (!make_map_3d(&map_x, src.data, C, c.S, c.B, src.token, src.batch, kM) ||
        !make_map_3d(&map_w, W, C, c.R, c.NA, C, (int64_t)c.R * C, g.Rp))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)g.stages * stage + part + kBarBytes + 1024;
    cudaError_t err = ensure_smem_attr((const void *)lora_shrink_tc_kernel, smem, dev);
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
    return cudaLaunchKernelEx(&cfg, lora_shrink_tc_kernel, map_x, map_w, g);
}

cudaError_t lora_tc_expand(const void *h, const void *W, const LoraCall &c, int C, cudaStream_t stream,
                           const DeviceInfo &dev) {
    const int run = ex_run(c.R);
    const size_t smem = (size_t)c.R * kExWPitch + (size_t)2 * c.R * ex_h_pitch(run);
    cudaError_t err = ensure_smem_attr((const void *)lora_expand_tc_kernel, smem, dev);
    if (err != cudaSuccess) return err;
    const dim3 grid((C + kExC - 1) / kExC, (c.S + run - 1) / run, c.B);
    return launch_pdl(lora_expand_tc_kernel, grid, dim3(256), smem, stream, static_cast<const uint16_t *>(h),
                      static_cast<const uint16_t *>(W), c.ids, c.ids_are_64, c.lens,
                      static_cast<const uint16_t *>(c.base.data), (long long)c.base.batch, (long long)c.base.token,
                      static_cast<uint16_t *>(c.out.data), (long long)c.out.batch, (long long)c.out.token, c.S,
                      padded_tokens(c.S), C, c.R, c.NA, run);
}

cudaError_t lora_tc_grads(const GradOperand &o0, const GradOperand &o1, const LoraCall &c, bool in_parts,
                          cudaStream_t stream, const DeviceInfo &dev) {
    GradArgs g = {};
    g.o[0] = o0, g.o[1] = o1;
    g.o[0].blocks = o0.acc ? (o0.C + kM - 1) / kM : 0;
    g.o[1].blocks = o1.acc ? (o1.C + kM - 1) / kM : 0;
    g.ids = c.ids, g.is64 = c.ids_are_64, g.lens = c.lens, g.accumulate = c.accumulate;
    g.B = c.B, g.S = c.S, g.R = c.R, g.NA = c.NA, g.pieces = (c.S + kLoraTcPiece - 1) / kLoraTcPiece;
    g.Np = (3 * c.R + 15) / 16 * 16;
    g.bufs = !in_parts && g.Np <= 256 ? 2 : 1;
    const int stage = kRowTile + g.Np * kBlk * 2, extra = in_parts ? 0 : c.R * kM * 4;
    g.stages = stages_for(stage, extra);
    g.tmem_cols = tmem_columns(g.bufs * g.Np);
    const int h_box = g.Np <= 256 ? g.Np : g.Np / 2;  // a box has at most 256 rows
    const int Sp = padded_tokens(c.S);
    CUtensorMap map_x, map_e, map_d, map_h;
    if (!make_map_3d(&map_x, o0.src, o0.C, c.S, c.B, o0.token, o0.batch, kBlk) ||
        !make_map_3d(&map_e, o0.h, Sp, 3 * c.R, c.B, Sp, (int64_t)3 * c.R * Sp, h_box) ||
        !make_map_3d(&map_d, o1.src, o1.C, c.S, c.B, o1.token, o1.batch, kBlk) ||
        !make_map_3d(&map_h, o1.h, Sp, 3 * c.R, c.B, Sp, (int64_t)3 * c.R * Sp, h_box))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)g.stages * stage + extra + kBarBytes + 1024;
    auto kern = in_parts ? lora_grad_tc_kernel<false> : lora_grad_tc_kernel<true>;
    cudaError_t err = ensure_smem_attr((const void *)kern, smem, dev);
    if (err != cudaSuccess) return err;
    const unsigned x = (unsigned)(g.o[0].blocks + g.o[1].blocks);
    const dim3 grid = in_parts ? dim3(x, (unsigned)g.pieces, (unsigned)c.B) : dim3(x, (unsigned)c.NA);
    return launch_pdl(kern, grid, dim3(kGradThreads), smem, stream, map_x, map_e, map_d, map_h, g);
}

int read_and_clear_lora_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_err_lora, sizeof(v)) != cudaSuccess) return -1;
    if (v != 0 && cudaMemcpyToSymbol(g_err_lora, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return (int)v;
}

}  // namespace adaln
