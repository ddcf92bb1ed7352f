"""Plain 64-bit forms of the operators of include/adaln_ops.h, with the error
bounds the GPU results are held to.

U = 2^-24 is the relative error of one fp32 rounding.  A sum of n terms along
a chain of depth k is within k U of the sum of their magnitudes.  Depths
count the kernels' documented orders; what they leave is rounded up.
"""

from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of the type, relative


def f64(t):
    return t.detach().to("cpu", torch.float64)


def pairs(Dr, interleaved):
    i = torch.arange(Dr // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + Dr // 2)


def rotate(n, c, s, interleaved, back=False):
    """The first 2 * c.shape[-1] channels of n turned by (c, s)."""
    Dr = 2 * c.shape[-1]
    a, b = pairs(Dr, interleaved)
    y = n.clone()
    s = -s if back else s
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., a] * s + n[..., b] * c
    return y


def rotate_size(n, c, s, interleaved):
    """The sum of the magnitudes of the terms of each rotated channel."""
    return rotate(n.abs(), c.abs(), -s.abs(), interleaved).abs().maximum(
        rotate(n.abs(), c.abs(), s.abs(), interleaved).abs())


def angles(cos, sin, pos, B, S):
    """(cos, sin) [B,S,1,Dr/2] of the rows, and which rows are real."""
    P = cos.shape[0]
    p = torch.arange(S).expand(B, S) if pos is None else pos.cpu().long()
    real = (p >= 0) & (p < P)
    at = torch.where(real, p, 0)
    return f64(cos)[at][:, :, None], f64(sin)[at][:, :, None], real[:, :, None, None]


def heads_fwd(x, w, cos, sin, pos, eps, interleaved):
    """(y, bound) of head rows x [B,S,H,Dh].

    r: the chain of 5 adds in a lane and at most 5 across lanes, 1/Dh and the
    fused eps give 13 U on the argument, half of that on r, and 4 U for the
    reciprocal root (CUDA bounds rsqrtf by 2 ulp): 11 U.  n = x r w: 2 more.  A
    turned channel: 3 more on its two terms.  16 in all.
    """
    B, S = x.shape[:2]
    c, s, real = angles(cos, sin, pos, B, S)
    xf = torch.where(real, f64(x), 0.0)
    r = 1.0 / (xf.square().mean(-1, keepdim=True) + eps).sqrt()
    n = xf * r * (1.0 if w is None else f64(w))
    y = torch.where(real, rotate(n, c, s, interleaved), 0.0)
    half = HALF[x.dtype]
    err = 16 * U * torch.where(real, rotate_size(n, c, s, interleaved), 0.0)
    return y, err * (1 + half) + (half if x.dtype != torch.float32 else 0.0) * y.abs()


def heads_bwd(dy, x, w, cos, sin, pos, eps, interleaved):
    """(dx, bound, dw, bound) of head rows.

    With G the size of g's terms, M = sum G |w| |x|: g is within 3 U of G, h
    within 4 U, hx within 16 U of M (10 adds, g x, the product), r^2/Dh within 25
    U, r within 11 U.  So dx is within r U (16 G |w| + 64 |x| r^2/Dh M).
    dw: 15 U on g x r and the sum's depth: at most 24 rows a lane or 2 H (a tile
    holds 48 tasks of 2 rows over 4 warps, or one token), 3 shuffles, 4 warps, a
    128th of the tiles (at most S) and 14 in the fold, the samples.
    """
    B, S = x.shape[:2]
    c, s, real = angles(cos, sin, pos, B, S)
    xf, gy = torch.where(real, f64(x), 0.0), torch.where(real, f64(dy), 0.0)
    wf = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else f64(w)
    r = 1.0 / (xf.square().mean(-1, keepdim=True) + eps).sqrt()
    g = rotate(gy, c, s, interleaved, back=True)
    G = rotate_size(gy, c, s, interleaved)
    h = g * wf
    dx = torch.where(real, r * (h - xf * r * r * (h * xf).mean(-1, keepdim=True)), 0.0)
    M = (G * wf.abs() * xf.abs()).mean(-1, keepdim=True)
    err = torch.where(real, U * r * (16 * G * wf.abs() + 64 * xf.abs() * r * r * M), 0.0)
    half = HALF[x.dtype]
    err = err * (1 + half) + (half if x.dtype != torch.float32 else 0.0) * dx.abs()
    dw = torch.where(real, g * xf * r, 0.0).sum((0, 1, 2))
    depth = 15 + max(24, 2 * x.shape[2]) + 3 + 4 + (S + 127) // 128 + 14 + B
    dw_err = depth * U * torch.where(real, G * xf.abs() * r, 0.0).sum((0, 1, 2))
    return dx, err, dw, dw_err


def embed_bwd(d_out, tokens, V, scale):
    """(gradient, sum of magnitudes, occurrences) in 64 bits."""
    t = tokens.cpu().long().reshape(-1)
    g = f64(d_out).reshape(t.numel(), -1)
    ok = (t >= 0) & (t < V)
    acc = torch.zeros((V, g.shape[1]), dtype=torch.float64)
    size = torch.zeros_like(acc)
    acc.index_add_(0, t[ok], g[ok])
    size.index_add_(0, t[ok], g[ok].abs())
    return acc * scale, size * abs(scale), torch.bincount(t[ok], minlength=V)


def embed_bwd_order(d_out, tokens, V, scale):
    """The gradient by the documented order, in fp32 rounded step by step:
    pieces of 32 occurrences from +0, and nodes of 32 children from +0 above
    them."""
    t = tokens.cpu().long().reshape(-1)
    g = d_out.detach().cpu().float().reshape(t.numel(), -1)
    out = torch.zeros((V, g.shape[1]))
    for v in t[(t >= 0) & (t < V)].unique().tolist():
        sums = list(g[t == v])
        while True:
            level = []
            for i in range(0, len(sums), 32):
                s = torch.zeros(g.shape[1])
                for x in sums[i:i + 32]:
                    s = s + x
                level.append(s)
            sums = level
            if len(sums) == 1:
                break
        total = sums[0]
        out[v] = total * torch.tensor(scale, dtype=torch.float32)
    return out


def check(got, want, bound, what):
    """got within bound of want everywhere (and finite there)."""
    d = (f64(got) - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off; worst {d[bad].max():.3g} against "
                           f"{bound.expand_as(d)[bad][d[bad].argmax()]:.3g}")
