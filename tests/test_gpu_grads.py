"""adaln_grad_norm and adaln_grad_clip against 64 bits, at the ends of the
number range and at every alignment.

The squares of 16 KB are summed in fp32 along a chain of at most 8 fused adds, 2
adds, 5 across lanes and 8 warps: the sum is within 23 U, the root within 12
U, and the result rounds once: 13 U, held to 17.  coef: one rounding more; a clipped value:
one product and the rounding of its type more."""

from __future__ import annotations

import math

import pytest
import torch

import ops_ref
from gpu_util import lib
from invariant_dit_adaln_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = ops_ref.U


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def exact_norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def make(sizes, seed=0, mixed=True):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * 10.0 ** (-(i % 4))).to(BF16 if mixed and i % 2 else F32).cuda()
            for i, n in enumerate(sizes)]


LISTS = [[], [0], [1], [0, 1, 0, 3], [4095, 4096, 4097, 8191, 8192, 8193, 16383, 16384, 16385], [1] * 17, [5] * 129, [3] * 1500, [1, 0, 2] * 2000,
         [1000000, 7, 333333], [40000] * 70]


def check_clip(grads, outs, stats, max_norm):
    norm = exact_norm(grads)
    assert abs(float(stats[0]) - norm) <= 17 * U * norm
    coef = min(1.0, max_norm / (norm + 1e-6))
    for g, o in zip(grads, outs):
        want = g.double().cpu() * coef
        half = ops_ref.HALF[g.dtype]
        # 1e-40: below the normal range of fp32 a rounding is absolute
        ops_ref.check(o, want, want.abs() * (20 * U + (half if g.dtype == BF16 else 0.0)) * (1 + half) + 1e-40, "clip")


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s, default=0)}")
def test_norm_and_clip(sizes):
    grads = make(sizes)
    norm = exact_norm(grads)
    got = binding.adaln_grad_norm(grads)
    assert got.shape == (1,) and abs(float(got) - norm) <= 17 * U * norm
    for max_norm in (0.5 * norm, 2 * norm + 1, 0.0, math.inf):
        outs, stats = binding.adaln_grad_clip(grads, max_norm)
        assert float(stats[0]) == float(got)
        check_clip(grads, outs, stats, max_norm)
        again = [g.clone() for g in grads]
        back, s2 = binding.adaln_grad_clip(again, max_norm, outs=again)
        assert back is again and torch.equal(s2, stats)
        assert all(torch.equal(a, o) for a, o in zip(again, outs))
        if max_norm >= norm + 1:
            assert float(stats[1]) == 1.0 and all(torch.equal(a, g) for a, g in zip(outs, grads))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_alignment(dtype):
    """Every offset of input and output within 16 bytes: the bits of the aligned call, and nothing else written."""
    step = 16 // torch.empty(0, dtype=dtype).element_size()
    for n in (1, 5, 8, 100, 8192 + 3, 40001):
        g = torch.randn(n, device="cuda").to(dtype)
        (want,), stats = binding.adaln_grad_clip([g], 0.5)
        for i in range(step):
            src = torch.full((n + 32,), float("nan"), dtype=dtype, device="cuda")
            src[i:i + n] = g
            assert torch.equal(binding.adaln_grad_norm([src[i:i + n]]), stats[:1])
            for j in (i, 0, 1, step - 1):
                dst = torch.full((n + 32,), 7.0, dtype=dtype, device="cuda")
                _, s2 = binding.adaln_grad_clip([src[i:i + n]], 0.5, outs=[dst[j:j + n]])
                assert torch.equal(s2, stats) and torch.equal(dst[j:j + n], want), (n, i, j)
                assert (dst[:j] == 7).all() and (dst[j + n:] == 7).all()
            view = [src[i:i + n]]
            binding.adaln_grad_clip(view, 0.5, outs=view)
            assert torch.equal(view[0], want) and src[:i].isnan().all() and src[i + n:].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ends_of_the_range(dtype):
    """Squares that fp32 cannot hold; infinities and NaN; zeros."""
    for value in (1e30, 3e38, 1e-30, 1e-38):
        g = [torch.full((20000,), value, device="cuda").to(dtype), torch.zeros(9, device="cuda").to(dtype)]
        norm = exact_norm(g)
        got = float(binding.adaln_grad_norm(g))
        if norm > 3.4028235677973366e38:
            assert got == math.inf
        else:
            assert abs(got - norm) <= 2 * U * norm, value
    # ordinary values beside tiny ones, each in pieces of their own and together
    g = [torch.full((20000,), 1e-25, device="cuda").to(dtype), torch.ones(20000, device="cuda").to(dtype)]
    g.append(torch.cat(g))
    norm = exact_norm(g)
    assert abs(float(binding.adaln_grad_norm(g)) - norm) <= 17 * U * norm
    zero = [torch.zeros(50000, device="cuda").to(dtype)]
    outs, stats = binding.adaln_grad_clip(zero, 1.0)
    assert stats.tolist() == [0.0, 1.0] and not outs[0].any()
    bad = torch.ones(30000, device="cuda").to(dtype)
    bad[29999] = float("inf")
    outs, stats = binding.adaln_grad_clip([bad], 1.0)
    assert stats.tolist() == [math.inf, 0.0] and outs[0][29999].isnan() and not outs[0][:29999].any()
    assert binding.adaln_grad_clip([bad], math.inf)[1].tolist() == [math.inf, 1.0]
    bad[3] = float("nan")
    for max_norm in (1.0, math.inf):
        outs, stats = binding.adaln_grad_clip([bad], max_norm)
        assert stats.isnan().all() and outs[0].isnan().all()


def test_order_is_fixed():
    """The same bits from run to run, for copies elsewhere, and for a tensor listed twice."""
    grads = make([123457, 99, 8192 * 3 + 5], mixed=True)
    want = binding.adaln_grad_norm(grads)
    for _ in range(5):
        assert torch.equal(binding.adaln_grad_norm([g.clone() for g in grads]), want)
    twice = binding.adaln_grad_norm([grads[0], grads[0]])
    one = exact_norm(grads[:1])
    assert abs(float(twice) - math.sqrt(2) * one) <= 17 * U * math.sqrt(2) * one


def test_beyond_2_31_elements():
    n = (1 << 31) + 40000
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[0], g[n - 1], g[(1 << 31) + 17] = 3.0, 4.0, 12.0
    assert float(binding.adaln_grad_norm([g])) == 13.0
    binding.adaln_grad_clip([g], 6.5, outs=[g])
    # coef = 6.5 / (13 + 1e-6), and 3 coef is rounded to bf16
    assert g[0] == 1.5 and g[n - 1] == 2.0 and g[(1 << 31) + 17] == 6.0


def test_graph_and_stream():
    grads = make([30000, 17, 500, 70000] * 40)
    outs = [torch.empty_like(g) for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, stats = binding.adaln_grad_clip(grads, 1.0, outs=outs)
    for _ in range(2):
        want, s2 = binding.adaln_grad_clip(grads, 1.0)
        graph.replay()
        assert torch.equal(stats, s2) and all(torch.equal(a, b) for a, b in zip(outs, want))
        grads[0].mul_(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want, s2 = binding.adaln_grad_clip(grads, 1.0)
    got, s3 = binding.adaln_grad_clip(grads, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s2, s3) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    g = torch.ones(10, device="cuda")
    for bad in (lambda: binding.adaln_grad_norm([g.cpu()]), lambda: binding.adaln_grad_norm([g.half()])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: binding.adaln_grad_norm([g[::2]]), lambda: binding.adaln_grad_clip([g], 1.0, outs=[]),
                lambda: binding.adaln_grad_norm([g], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: binding.adaln_grad_clip([g], -1.0), lambda: binding.adaln_grad_clip([g], float("nan")),
                lambda: binding.adaln_grad_clip([g], 1.0, outs=[g[:5]]),
                lambda: binding.adaln_grad_clip([g, g], 1.0, outs=[g, g]),
                lambda: binding.adaln_grad_clip([g[:8]], 1.0, outs=[g[1:9]])):
        with pytest.raises(binding.AdaLNError):
            bad()
