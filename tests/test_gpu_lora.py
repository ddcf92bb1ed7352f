"""Low-rank adapters against 64 bits: forward, dx and the adapters' gradients."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding
from ops_ref import check
from tune_ref import Lora

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
NAME = {torch.bfloat16: "bf16", torch.float32: "f32"}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


def fn(name, t):
    return getattr(binding, ("adaln_f32_" if t == torch.float32 else "adaln_") + name)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def same(a, b):
    return torch.equal(bits(a), bits(b))


def inputs(t, B, S, K, N, R, NA, seed=0, lens=None, is64=False):
    gen = torch.Generator("cuda").manual_seed(seed + 131 * S + K + N + R)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    c = dict(x=normal(B, S, K).to(t), A=(normal(NA, R, K) / K ** 0.5).to(t), U=(normal(NA, R, N) / R ** 0.5).to(t),
             scale=0.5 + torch.rand(NA, generator=gen, device="cuda"), y=normal(B, S, N).to(t),
             d_out=normal(B, S, N).to(t), dx_base=normal(B, S, K).to(t))
    ids = torch.randint(-1, NA + 1, (B,), generator=gen, device="cuda")
    if B > 1:
        ids[0] = 0
    c["ids"] = ids if is64 else ids.int()
    c["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return c


def run(t, c, **kw):
    """(out, dx, dA, dU) of a forward and a backward, rows past the end at 7."""
    out = torch.full_like(c["y"], 7.0)
    dx = torch.full_like(c["x"], 7.0)
    w = (c["A"], c["U"], c["scale"], c["ids"])
    _, state = fn("lora_fwd", t)(c["x"], *w, y=c["y"], lens=c["lens"], out=out)
    _, dA, dU = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, lens=c["lens"], dx_base=c["dx_base"], dx=dx, **kw)
    return out, dx, dA, dU


def verify(t, c, got, what=""):
    r = Lora(c["x"], c["A"], c["U"], c["scale"], c["ids"], c["y"], c["lens"], c["d_out"], c["dx_base"])
    out, dx, dA, dU = got
    r.check_rows(out, r.out, r.out_err, 7.0, what + "out")
    r.check_rows(dx, r.dx, r.dx_err, 7.0, what + "dx")
    check(dA, r.dA, r.dA_err, what + "dA")
    check(dU, r.dU, r.dU_err, what + "dU")


SIZES = [  # B, S, K, N, R, NA
    (1, 1, 8, 8, 8, 1), (3, 1, 64, 72, 8, 2), (5, 1, 1024, 520, 24, 3), (130, 1, 136, 264, 16, 4), (2, 3, 72, 64, 8, 1),
    (4, 16, 200, 136, 40, 2), (4, 17, 200, 136, 40, 2), (2, 31, 64, 64, 16, 2), (3, 64, 128, 256, 16, 2),
    (2, 65, 136, 8, 32, 1), (3, 127, 8, 392, 64, 2), (2, 129, 520, 128, 128, 3), (1, 300, 264, 136, 104, 1),
    (2, 255, 192, 320, 8, 2), (2, 257, 1000, 1032, 48, 2), (3, 640, 64, 200, 120, 2),
]


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_64_bits(t, size):
    c = inputs(t, *size, is64=size[1] % 2 == 0)
    verify(t, c, run(t, c))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S,lens", [(1, [1, 0, 1, 1, -5]), (9, [9, 0, 1, 8, 100]), (70, [70, 0, 1, 64, 65]),
                                    (260, [259, 256, 257, 128, 0]), (1100, [1100, 1025, 1023, 17, 1024])])
def test_ragged(t, S, lens):
    """Rows past the end may hold anything and are left as they were."""
    c = inputs(t, 5, S, 136, 200, 16, 2, lens=lens)
    clean = run(t, c)
    verify(t, c, clean)
    for b, n in enumerate(lens):
        n = min(max(n, 0), S)
        c["x"][b, n:], c["d_out"][b, n:], c["y"][b, n:] = float("nan"), float("inf"), float("nan")
        c["dx_base"][b, n:] = float("-inf")
    assert all(same(a, b) for a, b in zip(run(t, c), clean))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 8, 100])
def test_no_adapter(t, S):
    """Samples without an adapter: out is y, dx the base, nothing added to the
    gradients, whatever x and the adapters hold."""
    c = inputs(t, 4, S, 72, 88, 8, 2)
    c["ids"] = torch.tensor([-1, 2, 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    verify(t, c, run(t, c))
    c["x"][[0, 1, 3]] = float("nan")
    c["A"][0], c["U"][0], c["scale"][0] = float("nan"), float("inf"), float("nan")
    out, dx, dA, dU = run(t, c)
    for b in (0, 1, 3):
        assert same(out[b], c["y"][b]) and same(dx[b], c["dx_base"][b])
    assert (dA[0] == 0).all() and (dU[0] == 0).all() and dA[1].isfinite().all()
    # no adapters at all
    none = {**c, "A": c["A"][:0], "U": c["U"][:0], "scale": c["scale"][:0]}
    out, dx, dA, dU = run(t, none)
    assert same(out, c["y"]) and same(dx, c["dx_base"]) and dA.numel() == dU.numel() == 0


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 5, 90])
def test_without_base(t, S):
    c = inputs(t, 3, S, 72, 88, 16, 2)
    w = (c["A"], c["U"], c["scale"], c["ids"])
    out, state = fn("lora_fwd", t)(c["x"], *w)
    dx, dA, dU = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w)
    r = Lora(c["x"], *w, None, None, c["d_out"], None)
    check(out, r.out, r.out_err, "out")
    check(dx, r.dx, r.dx_err, "dx")
    # only what is asked for, the same bytes
    got = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, want_w=False)
    assert same(got[0], dx) and got[1] is None and got[2] is None
    got = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, want_x=False)
    assert got[0] is None and same(got[1], dA) and same(got[2], dU)
    for k in ("dA_acc", "dU_acc"):
        acc = torch.full_like(dA if k == "dA_acc" else dU, float("nan"))
        got = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, want_x=False, want_w=False, **{k: acc})
        assert same(acc, dA if k == "dA_acc" else dU)
    # rows past the end of a new tensor are zero
    lens = torch.tensor([S, S - 1, 0], dtype=torch.int32, device="cuda")
    out, state = fn("lora_fwd", t)(c["x"], *w, y=c["y"], lens=lens)
    dx, _, _ = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, lens=lens)
    assert (out[1, S - 1:] == 0).all() and (out[2] == 0).all() and (dx[1, S - 1:] == 0).all() and (dx[2] == 0).all()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 12, 70])
def test_layouts(t, S):
    """Slices of wider tensors, [S, B, C] storage, in place, broadcast, unaligned."""
    B, K, N = 3, 64, 88
    c = inputs(t, B, S, K, N, 16, 2, lens=[S, S // 2, S])
    want = run(t, c)
    step = 16 // c["x"].element_size()
    for how in ("slice", "transposed"):
        def move(v, fill):
            if how == "slice":
                wide = torch.full((B, S, v.shape[-1] + 4 * step), fill, dtype=t, device="cuda")
                place = wide[..., step:step + v.shape[-1]]
            else:
                wide = torch.full((S, B, v.shape[-1]), fill, dtype=t, device="cuda")
                place = wide.transpose(0, 1)
            place.copy_(v)
            return place, wide
        d = {**c, **{k: move(c[k], 9.0)[0] for k in ("x", "y", "d_out", "dx_base")}}
        out, owide = move(torch.full_like(c["y"], 7.0), 5.0)
        dx, dwide = move(torch.full_like(c["x"], 7.0), 5.0)
        w = (c["A"], c["U"], c["scale"], c["ids"])
        _, state = fn("lora_fwd", t)(d["x"], *w, y=d["y"], lens=c["lens"], out=out)
        _, dA, dU = fn("lora_bwd", t)(d["d_out"], d["x"], state, *w, lens=c["lens"], dx_base=d["dx_base"], dx=dx)
        assert all(same(a, b) for a, b in zip((out, dx, dA, dU), want)), how
        if how == "slice":
            for wide, n in ((owide, N), (dwide, K)):
                assert (wide[..., :step] == 5).all() and (wide[..., step + n:] == 5).all()
    # in place
    y, base = c["y"].clone(), c["dx_base"].clone()
    _, state = fn("lora_fwd", t)(c["x"], *w, y=y, lens=c["lens"], out=y)
    fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, lens=c["lens"], dx_base=base, dx=base)
    for got, old, first in ((y, c["y"], want[0]), (base, c["dx_base"], want[1])):
        for b, n in enumerate(c["lens"].tolist()):
            assert same(got[b, :n], first[b, :n]) and same(got[b, n:], old[b, n:])
    # broadcast: one row of y for all, one x for all samples
    y1 = c["y"][:1, :1].expand(B, S, N)
    x1 = c["x"][:1].expand(B, S, K)
    a, _ = fn("lora_fwd", t)(x1, *w, y=y1)
    b, _ = fn("lora_fwd", t)(x1.contiguous(), *w, y=y1.contiguous())
    assert same(a, b)
    # unaligned inputs are copied, unaligned outputs refused
    odd = torch.empty(c["x"].numel() + 1, dtype=t, device="cuda")[1:].view(B, S, K).copy_(c["x"])
    a, _ = fn("lora_fwd", t)(odd, *w, y=c["y"])
    b, _ = fn("lora_fwd", t)(c["x"], *w, y=c["y"])
    assert same(a, b)
    with pytest.raises(ValueError, match="aligned"):
        fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, dx=odd)


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 10, 40, 300, 1500])
def test_invariance(t, S):
    """A sample alone gives the bytes it has in a batch, and gradients do not
    depend on how the samples are split into accumulating calls."""
    B, K, N, R, NA = 6, 136, 72, 24, 2
    c = inputs(t, B, S, K, N, R, NA, lens=[S, S, S - 1, S // 3, S, S])
    want = run(t, c)
    acc = None
    for b0, b1 in ((0, 1), (1, 4), (4, 6)):
        part = {k: v if k in ("A", "U", "scale") else v[b0:b1].contiguous() for k, v in c.items()}
        kw = {} if acc is None else dict(dA_acc=acc[0], dU_acc=acc[1], accumulate=True)
        got = run(t, part, **kw)
        assert same(got[0], want[0][b0:b1]) and same(got[1], want[1][b0:b1])
        acc = got[2:]
    assert same(acc[0], want[2]) and same(acc[1], want[3])
    assert all(same(a, b) for a, b in zip(run(t, c), want))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 40, 300])
def test_accumulate_touches_only_adapters_that_occur(t, S):
    c = inputs(t, 3, S, 64, 72, 8, 4)
    c["ids"] = torch.tensor([2, -1, 2], device="cuda")
    _, _, dA, dU = run(t, c)
    a = torch.full_like(dA, float("nan"))
    u = torch.full_like(dU, float("nan"))
    a[2], u[2] = 1.0, -1.0
    run(t, c, dA_acc=a, dU_acc=u, accumulate=True)
    for got, part, start in ((a, dA, 1.0), (u, dU, -1.0)):
        assert got[[0, 1, 3]].isnan().all()
        assert ((got[2] - start - part[2]).abs() <= 4e-7 * (part[2].abs() + 2) * 8).all()
        assert (part[[0, 1, 3]] == 0).all()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_gradients_against_differences(t):
    """dx, dA, dU against differences of the 64-bit form."""
    c = inputs(t, 3, 4, 16, 24, 8, 2, lens=[4, 3, 2])
    c["ids"] = torch.tensor([0, 1, 0], device="cuda")
    out, dx, dA, dU = run(t, c)
    d = {k: v.double() if torch.is_floating_point(v) else v for k, v in c.items()}

    def loss(x, A, U):
        r = Lora.__new__(Lora)
        at = d["ids"]
        h = d["scale"][at][:, None, None] * (x @ A[at].transpose(1, 2))
        live = (torch.arange(4, device="cuda") < d["lens"][:, None])[..., None]
        return (((h @ U[at]) * d["d_out"]) * live).sum()

    gen = torch.Generator("cuda").manual_seed(5)
    for k, g in (("x", dx.double() - c["dx_base"].double()), ("A", dA.double()), ("U", dU.double())):
        v = torch.randn(d[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        if k == "x":
            v *= (torch.arange(4, device="cuda") < d["lens"][:, None])[..., None]
        a = {n: d[n] for n in ("x", "A", "U")}
        hi, lo = loss(**{**a, k: a[k] + 1e-4 * v}), loss(**{**a, k: a[k] - 1e-4 * v})
        # the loss is linear in each; dx is rounded with its base
        size = (v.abs() * (g.abs() + (c["dx_base"].double().abs() if k == "x" else 0))).sum()
        assert abs((hi - lo) / 2e-4 - (g * v).sum()) <= size * torch.finfo(t).eps, k


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_far_offsets(t):
    """Rows whose offsets pass 2^32 elements, in wide storage."""
    B, S, K, N = 2, 40, 64, 72
    c = inputs(t, B, S, K, N, 8, 1)
    want = run(t, c)
    big = torch.empty((1 << 32) + (1 << 20), dtype=t, device="cuda")
    far = (1 << 32) + 4096
    x = big.as_strided((B, S, K), (far, 128, 1)).copy_(c["x"])
    d_out = big.as_strided((B, S, N), (far, 128, 1), 1 << 18).copy_(c["d_out"])
    out = big.as_strided((B, S, N), (far, 128, 1), 2 << 18).fill_(7)
    w = (c["A"], c["U"], c["scale"], c["ids"])
    _, state = fn("lora_fwd", t)(x, *w, y=c["y"], out=out)
    dx = big.as_strided((B, S, K), (far, 128, 1), 3 << 18).fill_(7)
    _, dA, dU = fn("lora_bwd", t)(d_out, x, state, *w, dx_base=c["dx_base"], dx=dx)
    assert all(same(a, b) for a, b in zip((out, dx, dA, dU), want))


def test_many_samples_and_adapters():
    """More samples than one pass over the ids, every adapter count at its end."""
    for B, S, NA in ((1000, 1, 300), (300, 20, 7), (65535, 1, 2)):
        t = torch.bfloat16
        c = inputs(t, B, S, 16, 8, 8, NA)
        verify(t, c, run(t, c), f"{B}x{S}: ")


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 50, 1200])
def test_captured_and_on_another_stream(t, S):
    c = inputs(t, 3, S, 72, 136, 16, 2)
    want = run(t, c)
    w = (c["A"], c["U"], c["scale"], c["ids"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, state = fn("lora_fwd", t)(c["x"], *w, y=c["y"], stream=s)
    dx, dA, dU = fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, dx_base=c["dx_base"], stream=s.cuda_stream)
    s.synchronize()
    assert all(same(a, b) for a, b in zip((out, dx, dA, dU), want))
    x, ids = c["x"].clone(), c["ids"].clone()
    ws = torch.empty(fn("lora_bwd_workspace_bytes", t)(3, S, 72, 136, 16), dtype=torch.uint8, device="cuda")
    w = (c["A"], c["U"], c["scale"], ids)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn("lora_fwd", t)(x, *w, y=c["y"], out=out, state=state)
        fn("lora_bwd", t)(c["d_out"], x, state, *w, dx_base=c["dx_base"], dx=dx, dA_acc=dA, dU_acc=dU, workspace=ws)
    for k in range(3):
        x.copy_(c["x"].roll(k, 0))
        ids.copy_(c["ids"].roll(k))
        for v in (out, dx, dA, dU):
            v.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip((out, dx, dA, dU), run(t, {**c, "x": x, "ids": ids})))


def test_refusals():
    t = torch.bfloat16
    c = inputs(t, 2, 20, 64, 72, 16, 2)
    w = dict(A=c["A"], U=c["U"], scale=c["scale"], ids=c["ids"])
    f = binding.adaln_lora_fwd
    with pytest.raises(TypeError):
        f(c["x"].float(), **w)
    with pytest.raises(TypeError):
        f(c["x"], **{**w, "ids": c["ids"].float()})
    with pytest.raises(TypeError):
        f(c["x"], **{**w, "scale": c["scale"].double()})
    with pytest.raises(TypeError):
        f(c["x"], **w, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        f(c["x"].cpu(), **w)
    for bad in ({"A": c["A"][:, :8]}, {"U": c["U"][:1]}, {"scale": c["scale"][:1]}, {"ids": c["ids"][:1]},
                {"A": c["A"][..., :56]}):
        with pytest.raises(ValueError):
            f(c["x"], **{**w, **bad})
    with pytest.raises(ValueError):
        f(c["x"], **w, y=c["y"][:, :19])
    with pytest.raises(ValueError, match="state"):
        f(c["x"], **w, state=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.AdaLNError):  # ranks that are not supported
        f(c["x"], **{**w, "A": c["A"][:, :12], "U": c["U"][:, :12]})
    with pytest.raises(binding.AdaLNError):
        f(c["x"], **{**w, "A": c["A"].repeat(1, 9, 1), "U": c["U"].repeat(1, 9, 1)})
    wide = torch.zeros((2, 20, 72), dtype=t, device="cuda")
    with pytest.raises(binding.AdaLNError):  # out in x
        f(wide[..., :64], **w, out=wide)
    with pytest.raises(binding.AdaLNError):  # out a row after y
        buf = torch.zeros((2, 21, 72), dtype=t, device="cuda")
        f(c["x"], **w, y=buf[:, :20], out=buf[:, 1:])
    _, state = f(c["x"], **w)
    g = binding.adaln_lora_bwd
    with pytest.raises(ValueError, match="state"):
        g(c["d_out"], c["x"], state[:-16], **w)
    with pytest.raises(ValueError, match="accumulate"):
        g(c["d_out"], c["x"], state, **w, accumulate=True)
    with pytest.raises(ValueError, match="workspace"):
        g(c["d_out"], c["x"], state, **w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.AdaLNError):
        g(c["d_out"], c["x"], state, **w, dx=c["x"])
