"""Plain 64-bit forms of the operators of include/adaln_tune.h, with the error
bounds the GPU results are held to.

U = 2^-24 is the relative error of one fp32 rounding.  A sum of n terms along
a chain of depth k is within k U of the sum of their magnitudes; a tensor-core
instruction may truncate what it adds, so one of its steps counts as 2 U.
"""

from __future__ import annotations

import torch

from ops_ref import HALF, U, f64

GROUP = 32


def groups(x):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def record_of(x):
    """The records of rows x [..., D], byte for byte, from the definition in 64
    bits: the exponent by comparison with 127.5 2^k."""
    D = x.shape[-1]
    g = groups(f64(x))
    top = g.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(top)
    k = torch.full_like(top, -126.0)
    for e in range(-126, 121):  # the least k with top < 127.5 2^k, at most 121
        k = torch.where(top >= 127.5 * 2.0 ** e, e + 1.0, k)
    k = torch.where(bad, 128.0, k)
    q = torch.where(bad, 0.0, torch.round(g * torch.exp2(-k)).clamp(-127, 127))
    q = q.flatten(-2)[..., :D].to(torch.int8)
    s = (k.squeeze(-1) + 127).to(torch.uint8)
    return torch.cat((torch.nn.functional.pad(q, (0, -D % 16)).view(torch.uint8),
                      torch.nn.functional.pad(s, (0, -s.shape[-1] % 16))), -1).contiguous()


def value_of(rec, D):
    """The values of records, in 64 bits."""
    first, n = (D + 15) // 16 * 16, (D + GROUP - 1) // GROUP
    k = rec[..., first:first + n].double() - 127
    k = torch.where(k == 128, torch.inf, torch.exp2(k))
    return (groups(rec[..., :D].contiguous().view(torch.int8).double()) * k[..., None]).flatten(-2)[..., :D]


def again(x8, emb, mean, rstd):
    """The norm's output from values, rounded step by step in fp32 (on the CPU)."""
    D = x8.shape[-1]
    t = emb.dtype
    e = emb.cpu().float()[:, None]
    onep = (1 + e[..., :D]).to(t).float()
    xhat = (x8.cpu().float() - mean.cpu()[..., None]) * rstd.cpu()[..., None]
    return (xhat * onep + e[..., D:]).to(t)


class Lora:
    """out, dx, dA, dU of one call in 64 bits, and a bound on each.

    h: a lane's chain holds K / 64 pairs (CUDA cores), a tensor-core range K / 16
    instructions of 16 products; 2 (K / 16 + 16) + 16 U is more than either, and
    the joins.  Held as two bf16 parts: 2^-17.  out: R products and the base, 2 U
    each.  Gradients: a piece's rows (256 fused multiply-adds and their join: 320 U is
    more; 512 / 16 instructions: 2 (32 + 16) U), the pieces, the samples.
    """

    def __init__(self, x, A, Uw, scale, ids, y, lens, d_out=None, dx_base=None):
        B, S, K = x.shape
        NA, R, _ = A.shape
        N = Uw.shape[-1]
        self.dtype, half = x.dtype, HALF[x.dtype]
        at = ids.cpu().long()
        ok = (at >= 0) & (at < NA)
        n = torch.full((B,), S) if lens is None else lens.cpu().long().clamp(0, S)
        self.rows = (torch.arange(S) < n[:, None])[..., None]
        live = self.rows & ok[:, None, None]
        w = torch.where(ok, f64(scale)[at.clamp(0, max(NA - 1, 0))] if NA else 0.0, 0.0)[:, None, None]
        pick = torch.where(ok, at, 0)
        Ab, Ub = (f64(t)[pick] if NA else torch.zeros((B, R, t.shape[-1])).double() for t in (A, Uw))
        xf = torch.where(live, f64(x), 0.0)
        yf = torch.zeros((B, S, N)).double() if y is None else f64(y)
        split = 2.0 ** -17 if x.dtype == torch.bfloat16 else 0.0

        def shrink(src, W):
            h = w * (src @ W.transpose(1, 2))
            size = w.abs() * (src.abs() @ W.abs().transpose(1, 2))
            C = src.shape[-1]
            return h, (2 * (C // 16 + 17) + 16) * U * size + split * h.abs()

        def expand(h, eh, W, base):
            out = base + h @ W
            err = eh @ W.abs() + (R + 2) * 2 * U * (h.abs() @ W.abs() + base.abs())
            return out, err * (1 + half) + half * out.abs()

        def grad(h, eh, src):
            size = h.abs().transpose(1, 2) @ src.abs()
            err = eh.transpose(1, 2) @ src.abs() + (320 + S // 256 + B) * U * size
            g, e = (torch.zeros((NA, R, src.shape[-1])).double().index_add_(0, at[ok], v[ok])
                    for v in (h.transpose(1, 2) @ src, err))
            return g, e

        self.h, eh = shrink(xf, Ab)
        self.out, self.out_err = expand(self.h, eh, Ub, yf)
        if d_out is not None:
            d = torch.where(live, f64(d_out), 0.0)
            e, ee = shrink(d, Ub)
            self.dx, self.dx_err = expand(e, ee, Ab, torch.zeros((B, S, K)).double() if dx_base is None
                                          else f64(dx_base))
            self.dA, self.dA_err = grad(e, ee, xf)
            self.dU, self.dU_err = grad(self.h, eh, d)

    def check_rows(self, got, want, err, before, what):
        """The rows of the samples within the bound, the others as they were."""
        g, b = f64(got), before if isinstance(before, float) else f64(before)
        d = torch.where(self.rows, (g - want).abs(), 0.0)
        bad = ~(d <= err)
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {d[bad].max():.3g}"
        same = torch.where(self.rows, torch.zeros_like(g), g - b)
        assert (same == 0).all(), f"{what}: rows past the end changed"
