"""The plain 64-bit forms that the GPU results are compared with, against
autograd of the definition and against differences."""

from __future__ import annotations

import pytest
import torch

import ops_ref


def tables(P, Dr, seed=0):
    a = torch.rand((P, Dr // 2), generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * 6.28
    return a.cos(), a.sin()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("Dh,Dr", [(8, 8), (16, 8), (24, 0)])
def test_heads_backward_against_differences(Dh, Dr, interleaved):
    g = torch.Generator().manual_seed(Dh + Dr)
    x, dy = (torch.randn((2, 3, 2, Dh), generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.1 * torch.randn(Dh, generator=g, dtype=torch.float64)
    cos, sin = tables(4, Dr)
    pos = torch.tensor([[0, 3, -1], [2, 4, 1]])  # -1 and 4 are padding
    ops_ref.HALF[torch.float64] = 2.0 ** -53

    def loss(x, w):
        return (ops_ref.heads_fwd(x, w, cos, sin, pos, 1e-6, interleaved)[0] * dy).sum()

    dx, _, dw, _ = ops_ref.heads_bwd(dy, x, w, cos, sin, pos, 1e-6, interleaved)
    h = 1e-6
    for _ in range(4):
        d = torch.randn(x.shape, generator=g, dtype=torch.float64)
        num = (loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h)
        # truncation h^2 and rounding 2^-52 |loss| / h are both below 1e-7 here
        assert abs(num - (dx * d).sum()) < 1e-6
        e = torch.randn(w.shape, generator=g, dtype=torch.float64)
        num = (loss(x, w + h * e) - loss(x, w - h * e)) / (2 * h)
        assert abs(num - (dw * e).sum()) < 1e-6


def test_heads_forward_is_a_complex_rotation():
    x = torch.randn((1, 4, 2, 16), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    cos, sin = tables(4, 16)
    ops_ref.HALF[torch.float64] = 2.0 ** -53
    y, _ = ops_ref.heads_fwd(x, None, cos, sin, None, 0.0, True)
    n = x / x.square().mean(-1, keepdim=True).sqrt()
    z = torch.view_as_complex(n.reshape(1, 4, 2, 8, 2)) * torch.complex(cos, sin)[None, :, None]
    assert torch.allclose(y, torch.view_as_real(z).reshape(x.shape), rtol=1e-14, atol=1e-14)


def test_embed_order_is_the_sum():
    g = torch.Generator().manual_seed(2)
    tokens = torch.tensor([3] * 300 + [0] * 33 + [5] + [-1, 7, 3])
    d = torch.randn((len(tokens), 8), generator=g)
    want, size, count = ops_ref.embed_bwd(d, tokens, 7, 0.5)
    got = ops_ref.embed_bwd_order(d, tokens, 7, 0.5)
    assert count.tolist() == [33, 0, 0, 301, 0, 1, 0]
    # 32 in a piece, 10 pieces, the scale
    ops_ref.check(got, want, 43 * ops_ref.U * size, "order")
