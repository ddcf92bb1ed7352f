// C ABI of libadaln.so, second part (declared in include/adaln_ops.h): the
// host-side argument checks, in the order of api.cu, then the launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "checks.h"
#include "common.cuh"
#include "ops.h"

using namespace adaln;

namespace {

constexpr double kMaxElements = 1099511627776.0;  // 2^40
constexpr int kMaxHeads = 1024;
constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxTensors = 65536;

bool valid_eps(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }

// ---- head rows -------------------------------------------------------------

// The stride of a dimension of size 1 is not used, so it may hold anything: 0 from
// here on, also for the kernels, whose lanes without a row form addresses with it.
adaln_heads used(const adaln_heads &t, int B, int S, int H) {
    return {t.data, B > 1 ? t.batch : 0, S > 1 ? t.token : 0, H > 1 ? t.head : 0};
}

// Head rows as a lattice of dense byte runs: the dimensions of more than one
// index, innermost first, those that continue the run below them merged into it.
struct Lattice {
    uintptr_t base;
    int64_t run;  // bytes
    int nd;
    int64_t size[3], stride[3];  // strides in bytes, ascending
    int64_t extent;              // bytes from base to the end
    bool nested;                 // no two runs share a byte: each stride covers what lies inside it
};

Lattice lattice(const adaln_heads &rows, int B, int S, int H, int Dh, int es) {
    const adaln_heads t = used(rows, B, S, H);
    Lattice l = {};
    l.base = (uintptr_t)t.data;
    l.run = (int64_t)Dh * es;
    const int64_t size[3] = {H, S, B}, stride[3] = {t.head * es, t.token * es, t.batch * es};
    int64_t sz[3], st[3];
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (size[i] <= 1) continue;
        int j = n++;
        for (; j > 0 && st[j - 1] > stride[i]; --j) st[j] = st[j - 1], sz[j] = sz[j - 1];
        st[j] = stride[i], sz[j] = size[i];
    }
    l.extent = l.run;
    l.nested = true;
    for (int i = 0; i < n; ++i) {
        if (st[i] < l.extent) l.nested = false;
        l.extent += (sz[i] - 1) * st[i];
        if (l.nd == 0 && st[i] == l.run) {
            l.run *= sz[i];
        } else if (l.nd > 0 && st[i] == l.size[l.nd - 1] * l.stride[l.nd - 1]) {
            l.size[l.nd - 1] *= sz[i];
        } else {
            l.size[l.nd] = sz[i];
            l.stride[l.nd++] = st[i];
        }
    }
    return l;
}

// Do runs of x and y overlap?  Exact where the two have the same strides (two
// slices of one buffer); otherwise their whole extents are compared.
bool lattices_overlap(const Lattice &x, const Lattice &y) {
    if (!(x.base < y.base + (uint64_t)y.extent && y.base < x.base + (uint64_t)x.extent)) return false;
    // a lattice without a dimension is one run: any stride describes it
    const Lattice &more = x.nd >= y.nd ? x : y;
    int64_t sx[3] = {1, 1, 1}, sy[3] = {1, 1, 1};
    for (int i = 0; i < more.nd; ++i) {
        if ((x.nd > 0 && x.nd != more.nd) || (y.nd > 0 && y.nd != more.nd)) return true;
        if ((x.nd > 0 && x.stride[i] != more.stride[i]) || (y.nd > 0 && y.stride[i] != more.stride[i])) return true;
        if (x.nd > 0) sx[i] = x.size[i];
        if (y.nd > 0) sy[i] = y.size[i];
    }
    const int64_t off = (int64_t)(y.base - x.base);
    if (more.nd == 0) return true;
    // is -y.run < off + sum_i k_i stride_i < x.run for some k_i in (-sx_i, sy_i)?
    // the innermost k by division, the others by trial
    const int64_t st0 = more.stride[0];
    if (st0 == 0) return true;
    const int64_t n1 = more.nd > 1 ? sx[1] + sy[1] - 1 : 1, n2 = more.nd > 2 ? sx[2] + sy[2] - 1 : 1;
    if ((double)n1 * (double)n2 > 1e6) return true;  // too many to try: refused
    for (int64_t i2 = 0; i2 < n2; ++i2) {
        const int64_t o2 = off + (more.nd > 2 ? (i2 - (sx[2] - 1)) * more.stride[2] : 0);
        for (int64_t i1 = 0; i1 < n1; ++i1) {
            const int64_t o = o2 + (more.nd > 1 ? (i1 - (sx[1] - 1)) * more.stride[1] : 0);
            // the least k0 with o + k0 st0 > -y.run
            const int64_t need = -y.run + 1 - o;
            int64_t k0 = need >= 0 ? (need + st0 - 1) / st0 : -((-need) / st0);
            k0 = std::max(k0, -(sx[0] - 1));
            if (k0 <= sy[0] - 1 && o + k0 * st0 < x.run) return true;
        }
    }
    return false;
}

bool same_rows(const adaln_heads &a, const adaln_heads &b, int B, int S, int H) {
    return a.data == b.data && (B <= 1 || a.batch == b.batch) && (S <= 1 || a.token == b.token) &&
           (H <= 1 || a.head == b.head);
}

bool valid_strides(const adaln_heads &t, int B, int S, int H) {
    // below 2^42 elements, so that no offset of a valid size overflows
    const int64_t top = (int64_t)1 << 42, st[3] = {t.batch, t.token, t.head};
    const int sz[3] = {B, S, H};
    for (int i = 0; i < 3; ++i)
        if (sz[i] > 1 && (st[i] < 0 || st[i] > top / sz[i])) return false;
    return true;
}
bool aligned_rows(const adaln_heads &t, int B, int S, int H, int es) {
    const int64_t st[3] = {t.batch, t.token, t.head};
    const int sz[3] = {B, S, H};
    for (int i = 0; i < 3; ++i)
        if (sz[i] > 1 && st[i] * es % 16 != 0) return false;
    return aligned16(t.data);
}

bool valid_heads(int B, int S, int Hq, int Hk, int Dh) {
    return Dh >= 8 && Dh <= 256 && Dh % 8 == 0 && Hq >= 1 && Hq <= kMaxHeads && Hk >= 0 && Hk <= kMaxHeads && B >= 0 &&
           B <= 65535 && S >= 0 && S <= kMaxS && (double)B * S * (Hq + Hk) * Dh < kMaxElements;
}

// The checks that forward and backward share; `ins` are the head rows read (q,
// k and, backward, the output gradients at the same index), `outs` those
// written.  In place: outs[t] may be exactly ins[place + t].
adaln_status check_heads(HeadsCall &c, const adaln_heads *const *ins, int nin, const adaln_heads *const *outs,
                         int place, int es) {
    const int Hq = c.H[0], Hk = c.H[1];
    if (!valid_heads(c.B, c.S, Hq, Hk, c.Dh) || c.Dr < 0 || c.Dr > c.Dh || c.Dr % 8 != 0 || c.P < 0)
        return ADALN_ERR_SHAPE;
    if (c.pos == nullptr && c.Dr > 0 && c.S > c.P) return ADALN_ERR_SHAPE;
    const bool empty = c.B == 0 || c.S == 0;
    for (int i = 0; i < nin + 2; ++i) {
        const adaln_heads *h = i < nin ? ins[i] : outs[i - nin];
        const int H = c.H[i & 1];
        if (!empty && H > 0 && h && !valid_strides(*h, c.B, c.S, H)) return ADALN_ERR_SHAPE;
    }
    if (!valid_eps(c.eps) || (c.pos_is_64 != 0 && c.pos_is_64 != 1) || (c.interleaved != 0 && c.interleaved != 1) ||
        (c.accumulate != 0 && c.accumulate != 1))
        return ADALN_ERR_ARG;
    if (Hk == 0 && (c.w[1] || c.dw[1])) return ADALN_ERR_ARG;
    if (empty) return ADALN_OK;
    for (int i = 0; i < nin + 2; ++i) {
        const adaln_heads *h = i < nin ? ins[i] : outs[i - nin];
        if (c.H[i & 1] > 0 && (!h || !h->data)) return ADALN_ERR_NULL;
    }
    if (c.Dr > 0 && c.P > 0 && (!c.cos || !c.sin)) return ADALN_ERR_NULL;
    for (int i = 0; i < nin + 2; ++i) {
        const adaln_heads *h = i < nin ? ins[i] : outs[i - nin];
        const int H = c.H[i & 1];
        if (H > 0 && !aligned_rows(*h, c.B, c.S, H, es)) return ADALN_ERR_ALIGN;
    }
    if (!aligned16(c.w[0]) || !aligned16(c.w[1]) || !aligned16(c.cos) || !aligned16(c.sin) || !aligned16(c.pos) ||
        !aligned16(c.dw[0]) || !aligned16(c.dw[1]))
        return ADALN_ERR_ALIGN;
    // overlaps: head rows against head rows, and everything else by its extent
    Lattice in[4], out[2];
    for (int i = 0; i < nin; ++i)
        if (c.H[i & 1] > 0) in[i] = lattice(*ins[i], c.B, c.S, c.H[i & 1], c.Dh, es);
    const size_t rows = (size_t)c.B * c.S;
    const Buf flat_in[] = {{c.w[0], (size_t)c.Dh * es}, {c.w[1], (size_t)c.Dh * es},
                           {c.cos, (size_t)c.P * (c.Dr / 2) * 4}, {c.sin, (size_t)c.P * (c.Dr / 2) * 4},
                           {c.pos, rows * (c.pos_is_64 ? 8 : 4)}};
    const Buf flat_out[] = {{c.dw[0], (size_t)c.Dh * 4}, {c.dw[1], (size_t)c.Dh * 4},
                            {c.ws, (c.dw[0] || c.dw[1]) ? adaln_qk_norm_rope_bwd_workspace_bytes(c.B, c.S, Hq, Hk, c.Dh)
                                                        : 0}};
    if (any_alias(flat_out, 3, flat_in, 5)) return ADALN_ERR_ALIAS;
    for (int t = 0; t < 2; ++t) {
        if (c.H[t] == 0) continue;
        out[t] = lattice(*outs[t], c.B, c.S, c.H[t], c.Dh, es);
        if (!out[t].nested) return ADALN_ERR_ALIAS;
        for (int i = 0; i < nin; ++i) {
            if (c.H[i & 1] == 0) continue;
            if (i == place + t && same_rows(*outs[t], *ins[i], c.B, c.S, c.H[t])) continue;
            if (lattices_overlap(out[t], in[i])) return ADALN_ERR_ALIAS;
        }
        const Buf whole = {outs[t]->data, (size_t)out[t].extent};
        for (const Buf &f : flat_in)
            if (overlaps(whole, f)) return ADALN_ERR_ALIAS;
        for (const Buf &f : flat_out)
            if (overlaps(whole, f)) return ADALN_ERR_ALIAS;
    }
    if (Hk > 0 && lattices_overlap(out[0], out[1])) return ADALN_ERR_ALIAS;
    for (int i = 0; i < nin; ++i)
        if (c.H[i & 1] > 0)
            for (const Buf &f : flat_out)
                if (overlaps(Buf{ins[i]->data, (size_t)in[i].extent}, f)) return ADALN_ERR_ALIAS;
    return ADALN_OK;
}

template <typename T>
adaln_status heads_fwd(const adaln_heads *q, const adaln_heads *k, const T *wq, const T *wk, const float *cos,
                       const float *sin, const void *pos, int pos_is_64, const adaln_heads *q_out,
                       const adaln_heads *k_out, int B, int S, int Hq, int Hk, int Dh, int Dr, int P, int interleaved,
                       float eps, void *stream) {
    HeadsCall c = {};
    c.w[0] = wq, c.w[1] = wk;
    c.cos = cos, c.sin = sin, c.pos = pos, c.pos_is_64 = pos_is_64;
    c.B = B, c.S = S, c.H[0] = Hq, c.H[1] = Hk, c.Dh = Dh, c.Dr = Dr, c.P = P;
    c.interleaved = interleaved, c.eps = eps;
    const adaln_heads *ins[] = {q, k}, *outs[] = {q_out, k_out};
    adaln_status st = check_heads(c, ins, 2, outs, 0, sizeof(T));
    if (st != ADALN_OK) return st;
    DeviceInfo dev;
    st = check_current_device(&dev);
    if (st != ADALN_OK) return st;
    if (B == 0 || S == 0) return ADALN_OK;
    for (int t = 0; t < 2; ++t)
        if (c.H[t] > 0) c.x[t] = used(*ins[t], B, S, c.H[t]), c.out[t] = used(*outs[t], B, S, c.H[t]);
    return from_cuda(launch_heads_fwd<T>(c, (cudaStream_t)stream, dev));
}

template <typename T>
adaln_status heads_bwd(const adaln_heads *d_q_out, const adaln_heads *d_k_out, const adaln_heads *q,
                       const adaln_heads *k, const T *wq, const T *wk, const float *cos, const float *sin,
                       const void *pos, int pos_is_64, const adaln_heads *d_q, const adaln_heads *d_k, float *dwq_acc,
                       float *dwk_acc, int accumulate, void *workspace, size_t workspace_bytes, int B, int S, int Hq,
                       int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream) {
    HeadsCall c = {};
    c.w[0] = wq, c.w[1] = wk;
    c.cos = cos, c.sin = sin, c.pos = pos, c.pos_is_64 = pos_is_64;
    c.B = B, c.S = S, c.H[0] = Hq, c.H[1] = Hk, c.Dh = Dh, c.Dr = Dr, c.P = P;
    c.interleaved = interleaved, c.eps = eps;
    c.dw[0] = dwq_acc, c.dw[1] = dwk_acc, c.accumulate = accumulate;
    c.ws = static_cast<float *>(workspace);
    const adaln_heads *ins[] = {d_q_out, d_k_out, q, k}, *outs[] = {d_q, d_k};
    adaln_status st = check_heads(c, ins, 4, outs, 0, sizeof(T));
    if (st != ADALN_OK) return st;
    if (!aligned16(workspace)) return ADALN_ERR_ALIGN;
    const size_t need = (dwq_acc || dwk_acc) ? adaln_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hk, Dh) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return ADALN_ERR_WORKSPACE;
    DeviceInfo dev;
    st = check_current_device(&dev);
    if (st != ADALN_OK) return st;
    if (B == 0 || S == 0) {
        cudaError_t e = cudaSuccess;
        for (int t = 0; t < 2; ++t)
            if (c.dw[t] && !accumulate && e == cudaSuccess)
                e = cudaMemsetAsync(c.dw[t], 0, (size_t)Dh * 4, (cudaStream_t)stream);
        return from_cuda(e);
    }
    for (int t = 0; t < 2; ++t)
        if (c.H[t] > 0) {
            c.dy[t] = used(*ins[t], B, S, c.H[t]);
            c.x[t] = used(*ins[2 + t], B, S, c.H[t]);
            c.out[t] = used(*outs[t], B, S, c.H[t]);
        }
    return from_cuda(launch_heads_bwd<T>(c, (cudaStream_t)stream, dev));
}

// ---- embedding ---------------------------------------------------------------

bool valid_embed(int n, int V, int D) {
    return D >= 8 && D <= kMaxD && D % 8 == 0 && n >= 0 && n <= kMaxTokens && V >= 0 && V <= kMaxTokens;
}

template <typename T>
adaln_status embed_fwd(const void *tokens, int tokens_are_64, const T *table, float scale, T *out, int n, int V, int D,
                       void *stream) {
    if (!valid_embed(n, V, D)) return ADALN_ERR_SHAPE;
    if ((tokens_are_64 != 0 && tokens_are_64 != 1) || !isfinite(scale)) return ADALN_ERR_ARG;
    const Buf ins[] = {{tokens, (size_t)n * (tokens_are_64 ? 8 : 4)}, {table, n > 0 ? (size_t)V * D * sizeof(T) : 0}};
    const Buf outs[] = {{out, (size_t)n * D * sizeof(T)}};
    if (any_missing(ins, 2) || any_missing(outs, 1)) return ADALN_ERR_NULL;
    if (!aligned16(tokens) || !aligned16(table) || !aligned16(out)) return ADALN_ERR_ALIGN;
    if (any_alias(outs, 1, ins, 2)) return ADALN_ERR_ALIAS;
    DeviceInfo dev;
    const adaln_status st = check_current_device(&dev);
    if (st != ADALN_OK) return st;
    if (n == 0) return ADALN_OK;
    return from_cuda(launch_embed_fwd<T>(tokens, tokens_are_64, table, scale, out, n, V, D, (cudaStream_t)stream, dev));
}

template <typename T>
adaln_status embed_bwd(const T *d_out, const void *tokens, int tokens_are_64, float scale, float *d_table_acc,
                       adaln_bf16 *d_table, int accumulate, void *workspace, size_t workspace_bytes, int n, int V,
                       int D, void *stream) {
    if (!valid_embed(n, V, D)) return ADALN_ERR_SHAPE;
    if ((tokens_are_64 != 0 && tokens_are_64 != 1) || !isfinite(scale) || (accumulate != 0 && accumulate != 1))
        return ADALN_ERR_ARG;
    if (V > 0 && ((d_table_acc != nullptr) == (d_table != nullptr) || (accumulate && d_table))) return ADALN_ERR_ARG;
    const size_t need = adaln_embed_bwd_workspace_bytes(n, V, D);
    const Buf ins[] = {{d_out, (size_t)n * D * sizeof(T)}, {tokens, (size_t)n * (tokens_are_64 ? 8 : 4)}};
    const Buf outs[] = {{d_table_acc, d_table_acc ? (size_t)V * D * 4 : 0},
                        {d_table, d_table ? (size_t)V * D * 2 : 0},
                        {workspace, need}};
    if (any_missing(ins, 2)) return ADALN_ERR_NULL;
    if (!aligned16(d_out) || !aligned16(tokens) || !aligned16(d_table_acc) || !aligned16(d_table) ||
        !aligned16(workspace))
        return ADALN_ERR_ALIGN;
    if (any_alias(outs, 3, ins, 2)) return ADALN_ERR_ALIAS;
    if (need > 0 && (!workspace || workspace_bytes < need)) return ADALN_ERR_WORKSPACE;
    DeviceInfo dev;
    const adaln_status st = check_current_device(&dev);
    if (st != ADALN_OK) return st;
    if (V == 0) return ADALN_OK;
    if (n == 0) {
        // no tokens: the gradient is its starting value (+0 unless accumulating)
        if (accumulate) return ADALN_OK;
        return from_cuda(d_table ? cudaMemsetAsync(d_table, 0, outs[1].bytes, (cudaStream_t)stream)
                                 : cudaMemsetAsync(d_table_acc, 0, outs[0].bytes, (cudaStream_t)stream));
    }
    return from_cuda(launch_embed_bwd<T>(d_out, tokens, tokens_are_64, scale, d_table_acc, d_table, accumulate,
                                         workspace, n, V, D, (cudaStream_t)stream, dev));
}

// ---- gradients ---------------------------------------------------------------

adaln_status check_list(const adaln_tensor *t, int count) {
    if (count < 0 || count > kMaxTensors) return ADALN_ERR_SHAPE;
    if (count > 0 && !t) return ADALN_ERR_NULL;
    double total = 0.0;
    for (int i = 0; i < count; ++i) {
        if (t[i].numel < 0 || (double)t[i].numel >= kMaxElements) return ADALN_ERR_SHAPE;
        total += (double)t[i].numel;
    }
    if (total >= kMaxElements) return ADALN_ERR_SHAPE;
    for (int i = 0; i < count; ++i)
        if (t[i].dtype != ADALN_F32 && t[i].dtype != ADALN_BF16) return ADALN_ERR_ARG;
    for (int i = 0; i < count; ++i)
        if (t[i].numel > 0 && !t[i].data) return ADALN_ERR_NULL;
    return ADALN_OK;
}
int elem_bytes(const adaln_tensor &t) { return t.dtype == ADALN_BF16 ? 2 : 4; }
bool list_aligned(const adaln_tensor *t, int count) {
    for (int i = 0; i < count; ++i)
        if (t[i].numel > 0 && (uintptr_t)t[i].data % elem_bytes(t[i]) != 0) return false;
    return true;
}

// The ranges of a call: the gradients not scaled in place (read), the outputs
// and more[] (written).  A gradient scaled in place counts once, as written.
struct Ranges {
    const adaln_tensor *grads, *outs;
    int count;
    const Buf *more;
    int nmore;

    int size() const { return 2 * count + nmore; }
    // range i, if there is one
    bool get(int i, uintptr_t &begin, uintptr_t &end, bool &out) const {
        if (i >= 2 * count) {
            const Buf &b = more[i - 2 * count];
            begin = (uintptr_t)b.p, end = begin + b.bytes, out = true;
            return b.p && b.bytes > 0;
        }
        const int k = i >> 1;
        out = i & 1;
        if (grads[k].numel == 0 || (out ? !outs : outs && outs[k].data == grads[k].data)) return false;
        begin = (uintptr_t)(out ? outs : grads)[k].data;
        end = begin + (uintptr_t)grads[k].numel * elem_bytes(grads[k]);
        return true;
    }
};

struct Place {
    uintptr_t begin;
    int i;
    bool operator<(const Place &o) const { return begin < o.begin || (begin == o.begin && i < o.i); }
};

// Does a written range overlap another range?  A sweep in ascending order.  The
// lists can hold thousands and no call allocates, so the order comes in blocks
// of N places on the stack: each pass over the list keeps the N / 2 least ranges
// behind the block before it, or all that are left where they fit.
template <int N>
__attribute__((noinline)) bool written_overlap(const Ranges &r) {
    Place block[N], last = {0, -1};
    uintptr_t any_end = 0, out_end = 0, begin, end;
    bool out;
    for (bool more = true; more;) {
        int n = 0;
        Place most = {UINTPTR_MAX, 0x7FFFFFFF};  // the least place left out
        more = false;
        for (int i = 0; i < r.size(); ++i) {
            if (!r.get(i, begin, end, out)) continue;
            const Place p = {begin, i};
            if (!(last < p) || !(p < most)) continue;
            block[n++] = p;
            if (n == N) {
                std::nth_element(block, block + N / 2, block + N);
                n = N / 2;
                most = block[n];
                more = true;
            }
        }
        std::sort(block, block + n);
        for (int k = 0; k < n; ++k) {
            r.get(block[k].i, begin, end, out);
            if (begin < (out ? any_end : out_end)) return true;
            any_end = std::max(any_end, end);
            if (out) out_end = std::max(out_end, end);
        }
        if (n > 0) last = block[n - 1];
    }
    return false;
}

adaln_status grad_call(const adaln_tensor *grads, const adaln_tensor *outs, int count, bool clip, double max_norm,
                       float *stats, void *workspace, size_t workspace_bytes, void *stream) {
    adaln_status st = check_list(grads, count);
    if (st == ADALN_ERR_SHAPE) return st;
    if (clip && count > 0 && !outs) return ADALN_ERR_NULL;
    if (clip && !(max_norm >= 0.0)) return ADALN_ERR_ARG;
    if (st != ADALN_OK) return st;
    if (clip) {
        for (int i = 0; i < count; ++i)
            if (outs[i].numel != grads[i].numel) return ADALN_ERR_SHAPE;
        for (int i = 0; i < count; ++i)
            if (outs[i].dtype != grads[i].dtype) return ADALN_ERR_ARG;
        st = check_list(outs, count);
        if (st != ADALN_OK) return st;
    }
    if (!stats) return ADALN_ERR_NULL;
    if (!list_aligned(grads, count) || (clip && !list_aligned(outs, count)) || !aligned16(stats) ||
        !aligned16(workspace))
        return ADALN_ERR_ALIGN;
    const size_t need = adaln_grad_norm_workspace_bytes(grads, count);
    const Buf more[] = {{stats, clip ? 8u : 4u}, {workspace, need}};
    // 60 tensors with outputs, out of order: 4 us on the host; 2000: 0.24 ms; 65536: 29 ms
    const Ranges ranges = {grads, clip ? outs : nullptr, count, more, 2};
    if (ranges.size() < 512 ? written_overlap<512>(ranges) : written_overlap<8192>(ranges)) return ADALN_ERR_ALIAS;
    if (need > 0 && (!workspace || workspace_bytes < need)) return ADALN_ERR_WORKSPACE;
    DeviceInfo dev;
    st = check_current_device(&dev);
    if (st != ADALN_OK) return st;
    cudaError_t e = launch_grad_norm(grads, count, stats, clip, max_norm, workspace, (cudaStream_t)stream, dev);
    if (e == cudaSuccess && clip) e = launch_grad_scale(grads, outs, count, stats, (cudaStream_t)stream, dev);
    return from_cuda(e);
}

}  // namespace

extern "C" {

size_t adaln_qk_norm_rope_bwd_workspace_bytes(int B, int S, int Hq, int Hk, int Dh) {
    if (B == 0 || S == 0 || !valid_heads(B, S, Hq, Hk, Dh)) return 0;
    return round256(heads_bwd_ws_floats(B, S, Hq, Hk, Dh) * sizeof(float));
}

adaln_status adaln_qk_norm_rope_fwd(const adaln_heads *q, const adaln_heads *k, const adaln_bf16 *wq,
                                    const adaln_bf16 *wk, const float *cos, const float *sin, const void *pos,
                                    int pos_is_64, const adaln_heads *q_out, const adaln_heads *k_out, int B, int S,
                                    int Hq, int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream) {
    return heads_fwd(q, k, wq, wk, cos, sin, pos, pos_is_64, q_out, k_out, B, S, Hq, Hk, Dh, Dr, P, interleaved, eps,
                     stream);
}

adaln_status adaln_f32_qk_norm_rope_fwd(const adaln_heads *q, const adaln_heads *k, const float *wq, const float *wk,
                                        const float *cos, const float *sin, const void *pos, int pos_is_64,
                                        const adaln_heads *q_out, const adaln_heads *k_out, int B, int S, int Hq,
                                        int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream) {
    return heads_fwd(q, k, wq, wk, cos, sin, pos, pos_is_64, q_out, k_out, B, S, Hq, Hk, Dh, Dr, P, interleaved, eps,
                     stream);
}

adaln_status adaln_qk_norm_rope_bwd(const adaln_heads *d_q_out, const adaln_heads *d_k_out, const adaln_heads *q,
                                    const adaln_heads *k, const adaln_bf16 *wq, const adaln_bf16 *wk,
                                    const float *cos, const float *sin, const void *pos, int pos_is_64,
                                    const adaln_heads *d_q, const adaln_heads *d_k, float *dwq_acc, float *dwk_acc,
                                    int accumulate, void *workspace, size_t workspace_bytes, int B, int S, int Hq,
                                    int Hk, int Dh, int Dr, int P, int interleaved, float eps, void *stream) {
    return heads_bwd(d_q_out, d_k_out, q, k, wq, wk, cos, sin, pos, pos_is_64, d_q, d_k, dwq_acc, dwk_acc, accumulate,
                     workspace, workspace_bytes, B, S, Hq, Hk, Dh, Dr, P, interleaved, eps, stream);
}

adaln_status adaln_f32_qk_norm_rope_bwd(const adaln_heads *d_q_out, const adaln_heads *d_k_out, const adaln_heads *q,
                                        const adaln_heads *k, const float *wq, const float *wk, const float *cos,
                                        const float *sin, const void *pos, int pos_is_64, const adaln_heads *d_q,
                                        const adaln_heads *d_k, float *dwq_acc, float *dwk_acc, int accumulate,
                                        void *workspace, size_t workspace_bytes, int B, int S, int Hq, int Hk, int Dh,
                                        int Dr, int P, int interleaved, float eps, void *stream) {
    return heads_bwd(d_q_out, d_k_out, q, k, wq, wk, cos, sin, pos, pos_is_64, d_q, d_k, dwq_acc, dwk_acc, accumulate,
                     workspace, workspace_bytes, B, S, Hq, Hk, Dh, Dr, P, interleaved, eps, stream);
}

adaln_status adaln_embed_fwd(const void *tokens, int tokens_are_64, const adaln_bf16 *table, float scale,
                             adaln_bf16 *out, int n, int V, int D, void *stream) {
    return embed_fwd(tokens, tokens_are_64, table, scale, out, n, V, D, stream);
}

adaln_status adaln_f32_embed_fwd(const void *tokens, int tokens_are_64, const float *table, float scale, float *out,
                                 int n, int V, int D, void *stream) {
    return embed_fwd(tokens, tokens_are_64, table, scale, out, n, V, D, stream);
}

size_t adaln_embed_bwd_workspace_bytes(int n, int V, int D) {
    return valid_embed(n, V, D) ? round256(embed_bwd_ws_bytes(n, V, D)) : 0;
}

adaln_status adaln_embed_bwd(const adaln_bf16 *d_out, const void *tokens, int tokens_are_64, float scale,
                             float *d_table_acc, adaln_bf16 *d_table, int accumulate, void *workspace,
                             size_t workspace_bytes, int n, int V, int D, void *stream) {
    return embed_bwd(d_out, tokens, tokens_are_64, scale, d_table_acc, d_table, accumulate, workspace, workspace_bytes,
                     n, V, D, stream);
}

adaln_status adaln_f32_embed_bwd(const float *d_out, const void *tokens, int tokens_are_64, float scale,
                                 float *d_table_acc, int accumulate, void *workspace, size_t workspace_bytes, int n,
                                 int V, int D, void *stream) {
    return embed_bwd(d_out, tokens, tokens_are_64, scale, d_table_acc, (adaln_bf16 *)nullptr, accumulate, workspace,
                     workspace_bytes, n, V, D, stream);
}

size_t adaln_grad_norm_workspace_bytes(const adaln_tensor *grads, int count) {
    if (check_list(grads, count) != ADALN_OK) return 0;
    size_t pieces = 0;
    for (int i = 0; i < count; ++i) pieces += (size_t)grad_pieces(grads[i]);
    return round256(pieces * sizeof(float2));
}

adaln_status adaln_grad_norm(const adaln_tensor *grads, int count, float *norm, void *workspace,
                             size_t workspace_bytes, void *stream) {
    return grad_call(grads, nullptr, count, false, 0.0, norm, workspace, workspace_bytes, stream);
}

adaln_status adaln_grad_clip(const adaln_tensor *grads, const adaln_tensor *outs, int count, double max_norm,
                             float *stats, void *workspace, size_t workspace_bytes, void *stream) {
    return grad_call(grads, outs, count, true, max_norm, stats, workspace, workspace_bytes, stream);
}

}  // extern "C"
