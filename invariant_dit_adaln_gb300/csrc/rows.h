// Host-side checks of strided rows, shared by the C ABI's translation units
// (ops_api.cu, tune_api.cu): which rows overlap, which strides are usable.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "adaln_ops.h"
#include "checks.h"

namespace adaln {

// The stride of a dimension of size 1 is not used, so it may hold anything: 0 from
// here on, also for the kernels, whose lanes without a row form addresses with it.
inline adaln_heads used(const adaln_heads &t, int B, int S, int H) {
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

inline Lattice lattice(const adaln_heads &rows, int B, int S, int H, int Dh, int es) {
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
inline bool lattices_overlap(const Lattice &x, const Lattice &y) {
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

inline bool same_rows(const adaln_heads &a, const adaln_heads &b, int B, int S, int H) {
    return a.data == b.data && (B <= 1 || a.batch == b.batch) && (S <= 1 || a.token == b.token) &&
           (H <= 1 || a.head == b.head);
}

inline bool valid_strides(const adaln_heads &t, int B, int S, int H) {
    // below 2^42 elements, so that no offset of a valid size overflows
    const int64_t top = (int64_t)1 << 42, st[3] = {t.batch, t.token, t.head};
    const int sz[3] = {B, S, H};
    for (int i = 0; i < 3; ++i)
        if (sz[i] > 1 && (st[i] < 0 || st[i] > top / sz[i])) return false;
    return true;
}
inline bool aligned_rows(const adaln_heads &t, int B, int S, int H, int es) {
    const int64_t st[3] = {t.batch, t.token, t.head};
    const int sz[3] = {B, S, H};
    for (int i = 0; i < 3; ++i)
        if (sz[i] > 1 && st[i] * es % 16 != 0) return false;
    return aligned16(t.data);
}

}  // namespace adaln
