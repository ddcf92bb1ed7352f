"""adaln_grad_norm and adaln_grad_clip: what may be handed over as a list, and
the workspace a caller keeps."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def make(sizes):
    g = torch.Generator().manual_seed(len(sizes))
    return [torch.randn(n, generator=g).to(BF16 if i % 2 else F32).cuda() for i, n in enumerate(sizes)]


@pytest.mark.parametrize("sizes", [[], [0], [1], [4096, 4097], [8192 * 7 + 1, 3, 100000, 0, 8193]])
def test_workspace_of_the_size_asked_for(sizes):
    """8 bytes for each 16 KB of each tensor, rounded up to 256; smaller ones are refused."""
    grads = make(sizes)
    need = binding.adaln_grad_norm_workspace_bytes(grads)
    pieces = sum(-(-t.numel() * t.element_size() // 16384) for t in grads)
    assert need == -(-8 * pieces // 256) * 256
    want = binding.adaln_grad_norm(grads)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(binding.adaln_grad_norm(grads, workspace=ws), want)
    assert torch.equal(binding.adaln_grad_clip(grads, 1.0, workspace=ws)[1][:1], want)
    if need:
        with pytest.raises(ValueError):
            binding.adaln_grad_norm(grads, workspace=ws[:-1])


def test_lists_of_any_kind():
    """Lists, tuples and iterators; the outputs come back as they were given, an iterator as a list."""
    grads = make([5000, 7, 300])
    want, stats = binding.adaln_grad_clip(grads, 0.5)
    assert torch.equal(binding.adaln_grad_norm(iter(grads)), stats[:1])
    for kind in (list, tuple, iter, lambda x: (t for t in x)):
        outs = [torch.empty_like(t) for t in grads]
        given = kind(outs)
        back, s2 = binding.adaln_grad_clip(kind(grads), 0.5, outs=given)
        assert torch.equal(s2, stats) and len(list(back)) == 3
        assert back is given or isinstance(back, list)
        assert all(torch.equal(a, w) for a, w in zip(outs, want)) and all(a is b for a, b in zip(back, outs))


def test_coefficient_of_norms_beyond_fp32():
    """coef comes from the norm before its rounding: elements that fp32 holds with
    a norm that it does not are scaled, not lost; only infinite elements give 0."""
    g = [torch.full((20000,), 3e38, device="cuda")]
    norm = float(g[0].double().square().sum().sqrt())
    outs, stats = binding.adaln_grad_clip(g, 1e38)
    assert stats[0] == float("inf")
    # one rounding of coef, as the sums of squares are within 12 U of the norm: 14 U; a product's rounding more
    assert abs(float(stats[1]) - 1e38 / norm) <= 14 * 2.0 ** -24 * (1e38 / norm)
    want = g[0].double() * (1e38 / norm)
    assert ((outs[0].double() - want).abs() <= 15 * 2.0 ** -24 * want).all()
    outs, stats = binding.adaln_grad_clip(g, float("inf"))
    assert stats.tolist() == [float("inf"), 1.0] and torch.equal(outs[0], g[0])
    g[0][5] = float("-inf")
    outs, stats = binding.adaln_grad_clip(g, 1e38)
    assert stats.tolist() == [float("inf"), 0.0] and outs[0][5].isnan() and int(outs[0].count_nonzero()) == 1
