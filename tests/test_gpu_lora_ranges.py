"""Low-rank adapters over their whole range against 64 bits: drawn sizes, every
rank, many samples, the largest sizes, infinities."""

from __future__ import annotations

import random

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding
from ops_ref import check
from test_gpu_lora import NAME, TYPES, fn, inputs, run, same, verify
from tune_ref import Lora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    torch.cuda.synchronize()
    assert binding.device_error() == 0


def drawn(seed):
    """(B, S, K, N, R, NA, lens or None): at most 2^23 elements of x or y."""
    r = random.Random(seed)

    def spread(lo, hi):
        return round(lo * (hi / lo) ** r.random())

    K, N, R = 8 * spread(1, 512), 8 * spread(1, 512), 8 * r.randint(1, 16)
    S = spread(1, 3000)
    B = max(1, min(spread(1, 200), (1 << 23) // (S * max(K, N))))
    lens = [r.choice((S, r.randint(0, S), r.randint(0, S), 0, 1)) for _ in range(B)] if r.random() < 0.6 else None
    return B, S, K, N, R, r.randint(1, 9), lens


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("seed", range(24))
def test_drawn(t, seed):
    *size, lens = drawn(seed)
    c = inputs(t, *size, seed=seed, lens=lens, is64=seed % 2 == 0)
    verify(t, c, run(t, c), f"{size}: ")


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", range(1, 19))
def test_few_tokens(t, S):
    """Each number of tokens up to the tensor cores' first, alone and with lengths."""
    for B, R, lens in ((5, 24, None), (40, 56, [i * 7 % (S + 1) for i in range(40)])):
        c = inputs(t, B, S, 392, 200, R, 3, lens=lens)
        verify(t, c, run(t, c), f"{B}: ")


@pytest.mark.parametrize("S,R", [(11, 64), (11, 128), (12, 48), (12, 56), (12, 128), (13, 48), (14, 48), (15, 40),
                                 (16, 40), (19, 32), (20, 32), (26, 24), (27, 24), (39, 16), (40, 16), (79, 8),
                                 (80, 8)])
def test_both_sides_of_the_tensor_cores(S, R):
    t = torch.bfloat16
    for B, lens in ((3, None), (37, [i * 5 % (S + 1) for i in range(37)])):
        c = inputs(t, B, S, 200, 392, R, 3, lens=lens)
        verify(t, c, run(t, c), f"{B}: ")
        alone = {k: v if k in ("A", "U", "scale") else v[1:2].contiguous() for k, v in c.items() if v is not None}
        alone.setdefault("lens", None)
        assert all(same(a[0], b[1]) for a, b in zip(run(t, alone)[:2], run(t, c)[:2]))


@pytest.mark.parametrize("R", range(8, 136, 8))
def test_every_rank(R):
    """bf16 above 16 tokens: the stages, accumulators and schedules depend on R."""
    t = torch.bfloat16
    for S, lens in ((150, None), (600, [600, 513, 100])):
        c = inputs(t, 3, S, 328, 264, R, 2, lens=lens)
        verify(t, c, run(t, c), f"{S}: ")


@pytest.mark.parametrize("R", [16, 32, 40, 128])
def test_many_samples(R):
    """More samples than a window of the tile finders, with lengths, some without an
    adapter, in place and not: runs of tiles and dealt tiles."""
    t = torch.bfloat16
    r = random.Random(R)
    B, S, K, N = 150, 140, 136, 200
    lens = [r.choice((0, 1, 17, 127, 128, 129, S)) for _ in range(B)]
    c = inputs(t, B, S, K, N, R, 3, lens=lens)
    c["ids"][32:70] = -1
    want = run(t, c)
    verify(t, c, want)
    y, base = c["y"].clone(), c["dx_base"].clone()
    w = (c["A"], c["U"], c["scale"], c["ids"])
    _, state = fn("lora_fwd", t)(c["x"], *w, y=y, lens=c["lens"], out=y)
    fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, lens=c["lens"], dx_base=base, dx=base)
    for b, n in enumerate(lens):
        assert same(y[b, :n], want[0][b, :n]) and same(y[b, n:], c["y"][b, n:])
        assert same(base[b, :n], want[1][b, :n]) and same(base[b, n:], c["dx_base"][b, n:])
    # all lengths zero; no sample with an adapter
    c["lens"].zero_()
    verify(t, c, run(t, c))
    c["lens"].fill_(S)
    c["ids"].fill_(-1)
    verify(t, c, run(t, c))


@pytest.mark.parametrize("R", [8, 24, 32, 64, 104])
def test_bases(R):
    """No base, a base of one row for all, of a row a sample, of a sample for all."""
    t = torch.bfloat16
    B, S, K, N = 3, 200, 72, 136
    c = inputs(t, B, S, K, N, R, 2, lens=[200, 131, 64])
    w = (c["A"], c["U"], c["scale"], c["ids"])
    for y in (None, c["y"][:1, :1].expand(B, S, N), c["y"][:, :1].expand(B, S, N), c["y"][:1].expand(B, S, N)):
        out = torch.full((B, S, N), 7.0, dtype=t, device="cuda")
        fn("lora_fwd", t)(c["x"], *w, y=y, lens=c["lens"], out=out)
        r = Lora(c["x"], *w, y, c["lens"])
        r.check_rows(out, r.out, r.out_err, 7.0, "out")


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("size", [(1, 1, 65536, 65536, 128, 2), (2, 20, 65536, 8, 16, 1), (2, 33, 8, 65536, 40, 1),
                                  (1, 70001, 8, 16, 8, 1), (1, 20000, 64, 8, 128, 1), (3, 2, 4096, 12288, 64, 3)],
                         ids=lambda s: "x".join(map(str, s)))
def test_largest(t, size):
    c = inputs(t, *size)
    c["ids"].fill_(0)
    verify(t, c, run(t, c))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 12, 150])
def test_infinities(t, S):
    """What an infinity or a NaN enters is not finite, and nothing else changes."""
    B, K, N, R = 3, 136, 72, 16
    for where in ("x", "d_out", "A", "U", "scale", "y", "dx_base"):
        for bad in (float("inf"), float("nan")):
            c = inputs(t, B, S, K, N, R, 2)
            c["ids"] = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
            clean = run(t, c)
            v = c[where]
            v[(1,) if v.dim() == 1 else (1, v.shape[1] // 2, 5)] = bad
            got = run(t, c)
            x, A, U, y, d, base = (c[k].double() for k in ("x", "A", "U", "y", "d_out", "dx_base"))
            at = c["ids"].long()
            s = c["scale"].double()[at][:, None, None]
            h, e = s * (x @ A[at].transpose(1, 2)), s * (d @ U[at].transpose(1, 2))
            dA, dU = (torch.zeros(like.shape, dtype=torch.float64, device="cuda").index_add_(0, at, p.transpose(1, 2) @ q)
                      for like, p, q in ((A, e, x), (U, h, d)))
            for name, g, plain, first in zip(("out", "dx", "dA", "dU"), got,
                                             (y + h @ U[at], base + e @ A[at], dA, dU), clean):
                assert torch.equal(g.isfinite(), plain.isfinite()), (where, bad, name)
                # rows and channels that the value does not reach keep their bytes
                if where in ("x", "y") and name == "out" or where in ("d_out", "dx_base") and name == "dx":
                    keep = plain.isfinite()
                    assert torch.equal(g[keep], first[keep]), (where, bad, name)


def test_large_states():
    """h near the ends of what bf16 and fp32 hold."""
    t = torch.bfloat16
    for size in (2.0 ** 100, 2.0 ** 126, 2.0 ** -100):
        c = inputs(t, 2, 40, 64, 72, 8, 1)
        c["ids"].fill_(0)
        c["scale"].fill_(size)
        c["U"] = (c["U"].float() / size).to(t)
        c["y"].zero_()
        out, state = fn("lora_fwd", t)(c["x"], c["A"], c["U"], c["scale"], c["ids"], y=c["y"])
        r = Lora(c["x"], c["A"], c["U"], c["scale"], c["ids"], c["y"], None)
        check(out, r.out, r.out_err, f"{size}")
