"""8-bit activations against their definition, byte for byte, and the norm's
forward and backward with records against the ones without."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding
from tune_ref import again, record_of, value_of

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


def rows(gen, t, *shape):
    """Values of unlike size, some zero, some groups zero."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x = x * torch.exp(4 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    x[..., ::7] = 0
    if shape[-1] > 64:
        x[..., 32:64] *= (torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < 0.5)
    return x.to(t)


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 64, 248, 264, 520, 1024, 1032, 1160, 2056, 4096, 8192])
def test_records(t, D):
    gen = torch.Generator("cuda").manual_seed(D)
    for n in (1, 3, 70):
        x = rows(gen, t, n, D)
        ckpt = torch.full((n, binding.adaln_ckpt8_row_bytes(D)), 77, dtype=torch.uint8, device="cuda")
        got = fn("ckpt8_pack", t)(x, ckpt)
        assert got is ckpt and torch.equal(got.cpu(), record_of(x))
        out = fn("ckpt8_unpack", t)(ckpt, D)
        assert torch.equal(out.cpu().double(), value_of(ckpt.cpu(), D))
        step = (out.double() - x.double()).abs().cpu()
        top = torch.nn.functional.pad(x.double().abs().cpu(), (0, -D % 32)).unflatten(-1, (-1, 32)).amax(-1)
        assert (step <= torch.repeat_interleave(top, 32, -1)[:, :D] / 127.5).all()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("D", [8, 32, 40, 64, 72, 104, 120, 128, 136, 240, 256, 264, 504, 512, 520, 1048])
def test_records_of_several_rows_a_warp(t, D):
    """Any number of rows, and nothing written behind the last; groups that are not finite
    among them."""
    gen = torch.Generator("cuda").manual_seed(D)
    P = binding.adaln_ckpt8_row_bytes(D)
    for n in (1, 2, 5, 9, 31, 33, 67, 131, 1030):
        x = rows(gen, t, n, D)
        x[n // 2, D // 2] = float("nan")
        x[-1, -1] = float("inf")
        wide = torch.full((n + 40, P), 77, dtype=torch.uint8, device="cuda")
        fn("ckpt8_pack", t)(x, wide[:n])
        assert torch.equal(wide[:n].cpu(), record_of(x)) and (wide[n:] == 77).all()
        out = torch.full((n + 40, D), 5.0, dtype=t, device="cuda")
        fn("ckpt8_unpack", t)(wide[:n], D, out[:n])
        want = value_of(wide[:n].cpu(), D)
        assert torch.equal(out[:n].cpu().double().nan_to_num(7e30), want.nan_to_num(7e30)) and (out[n:] == 5).all()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_every_size_of_a_largest_value(t):
    """Largest magnitudes at and around each border, over the whole range; ties."""
    steps = [127.5, 127.0, 126.5, 64.0, 63.75, 63.5, 0.5, 1.5, 2.5]
    tops = [s * 2.0 ** k for k in range(-133, 122) for s in steps]
    top = torch.tensor(tops, dtype=torch.float64).to(t)
    top = top[torch.isfinite(top)]
    eps = torch.finfo(t).eps
    top = torch.cat((top, top.double().mul(1 - eps / 2).to(t), top.double().mul(1 + eps).to(t)))
    top = top[torch.isfinite(top)]
    part = torch.linspace(-1, 1, 31, dtype=torch.float64)
    x = torch.cat((top.double()[:, None], top.double()[:, None] * part), 1).to(t)
    x = torch.cat((x, torch.full((1, 32), torch.finfo(t).max).to(t), torch.full((1, 32), -torch.finfo(t).max).to(t)))
    ckpt = fn("ckpt8_pack", t)(x.cuda())
    assert torch.equal(ckpt.cpu(), record_of(x))
    assert torch.equal(fn("ckpt8_unpack", t)(ckpt, 32).cpu().double(), value_of(ckpt.cpu(), 32))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_infinity_and_nan_stay_in_their_group(t):
    gen = torch.Generator("cuda").manual_seed(1)
    x = rows(gen, t, 6, 200)
    x[1, 5], x[2, 40], x[3, 199], x[4, 0] = float("inf"), float("-inf"), float("nan"), float("nan")
    ckpt = fn("ckpt8_pack", t)(x)
    assert torch.equal(ckpt.cpu(), record_of(x))
    out = fn("ckpt8_unpack", t)(ckpt, 200).cpu()
    nan = torch.zeros(6, 200, dtype=torch.bool)
    nan[1, :32], nan[2, 32:64], nan[3, 192:], nan[4, :32] = True, True, True, True
    assert torch.equal(out.isnan(), nan)


NORMS = [(1, 1, 8), (3, 5, 40), (2, 33, 264), (2, 31, 1024), (1, 65, 1160), (2, 40, 2056), (2, 33, 3072), (1, 37, 4096)]


def norm_inputs(t, B, S, D, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + D)
    x = (torch.randn((B, S, D), generator=gen, device="cuda") * 2 + 0.5).to(t)
    dy = torch.randn((B, S, D), generator=gen, device="cuda").to(t)
    emb = (0.3 * torch.randn((B, 2 * D), generator=gen, device="cuda")).to(t)
    return x, dy, emb


def check_norm(t, B, S, D, seed=0):
    x, dy, emb = norm_inputs(t, B, S, D, seed)
    out, mean, rstd, ckpt = fn("out_fwd_ckpt8", t)(x, emb)
    for got, want in zip((out, mean, rstd), fn("out_fwd", t)(x, emb)):
        assert same(got, want)
    assert same(ckpt, fn("ckpt8_pack", t)(x))
    x8 = fn("ckpt8_unpack", t)(ckpt, D)
    dx, d_emb = fn("out_bwd_ckpt8", t)(dy, ckpt, emb, mean, rstd)
    for got, want in zip((dx, d_emb), fn("out_bwd", t)(dy, x8, emb, mean, rstd)):
        assert same(got, want)
    o = fn("out_again_ckpt8", t)(ckpt, emb, mean, rstd)
    assert same(o, again(x8, emb, mean, rstd))
    return x, dy, emb, ckpt, mean, rstd


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("B,S,D", NORMS)
def test_norm_with_records(t, B, S, D):
    check_norm(t, B, S, D)


@pytest.mark.parametrize("B,S,D", [(2, 33, 4104), (1, 65, 6144), (1, 40, 8192)])
def test_norm_with_records_long_rows(B, S, D):
    check_norm(torch.bfloat16, B, S, D)


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("D", [8, 16, 72, 128, 248, 256, 264, 504, 512, 520, 1016, 1024, 1032, 1528, 1536, 1544, 2056])
def test_norm_with_records_at_every_form(t, D):
    """The ends of the forms that hold a row in 1, 2, 4, 8, ... vectors a lane; more rows
    than the warps of one wave."""
    check_norm(t, 3, 37, D)
    check_norm(t, 2, 5001 if D <= 256 else 1201, D, seed=1)


def test_norm_with_records_many_rows():
    check_norm(torch.bfloat16, 3, 2053, 3072)
    check_norm(torch.float32, 2, 1029, 3072)


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_a_sample_does_not_depend_on_the_batch(t):
    x, dy, emb, ckpt, mean, rstd = check_norm(t, 5, 70, 520)
    dx, d_emb = fn("out_bwd_ckpt8", t)(dy, ckpt, emb, mean, rstd)
    for b in range(5):
        one = slice(b, b + 1)
        got = fn("out_bwd_ckpt8", t)(dy[one], ckpt[one], emb[one], mean[one], rstd[one])
        assert same(got[0], dx[one]) and same(got[1], d_emb[one])
        assert same(fn("out_fwd_ckpt8", t)(x[one], emb[one])[3], ckpt[one])


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_empty(t):
    D = 72
    assert fn("ckpt8_pack", t)(torch.empty((0, D), dtype=t, device="cuda")).shape == (0, 96)
    assert fn("ckpt8_unpack", t)(torch.empty((4, 0, 96), dtype=torch.uint8, device="cuda"), D).shape == (4, 0, D)
    x, dy, emb = norm_inputs(t, 2, 0, D)
    out, mean, rstd, ckpt = fn("out_fwd_ckpt8", t)(x, emb)
    dx, d_emb = fn("out_bwd_ckpt8", t)(dy, ckpt, emb, mean, rstd)
    assert dx.shape == (2, 0, D) and (d_emb == 0).all() and ckpt.shape == (2, 0, 96)
    assert fn("out_again_ckpt8", t)(ckpt, emb, mean, rstd).shape == (2, 0, D)


def test_layouts_and_given_outputs():
    """Strided and unaligned inputs are copied; outputs are written where given."""
    t = torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(3)
    x = rows(gen, t, 4, 9, 72)
    want = binding.adaln_ckpt8_pack(x)
    wide = torch.zeros((4, 9, 100), dtype=t, device="cuda")
    wide[..., 3:75] = x
    assert same(binding.adaln_ckpt8_pack(wide[..., 3:75]), want)
    assert same(binding.adaln_ckpt8_pack(x.transpose(0, 1)), want.transpose(0, 1))
    odd = torch.zeros(want.numel() + 1, dtype=torch.uint8, device="cuda")
    odd[1:] = want.flatten()
    assert same(binding.adaln_ckpt8_unpack(odd[1:].view(want.shape), 72), binding.adaln_ckpt8_unpack(want, 72))
    with pytest.raises(ValueError, match="aligned"):
        binding.adaln_ckpt8_pack(x, odd[1:].view(want.shape))
    out = torch.empty_like(x)
    assert binding.adaln_ckpt8_unpack(want, 72, out) is out


def test_far_records():
    """Rows whose records and values lie past 2^32 bytes."""
    D, n = 8192, 600_000
    x = torch.zeros((n, D), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(4)
    at = torch.tensor([0, 262_143, 262_144, 524_288, n - 1], device="cuda")
    x[at] = rows(gen, torch.bfloat16, 5, D)
    ckpt = binding.adaln_ckpt8_pack(x)
    assert torch.equal(ckpt[at].cpu(), record_of(x[at]))
    x.fill_(1)
    binding.adaln_ckpt8_unpack(ckpt, D, x)
    assert torch.equal(x[at].cpu().double(), value_of(ckpt[at].cpu(), D))
    assert int((x != 0).any(-1).sum()) == 5


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_captured_and_on_another_stream(t):
    x, dy, emb = norm_inputs(t, 2, 45, 264)
    want = fn("out_fwd_ckpt8", t)(x, emb)
    wdx, wd = fn("out_bwd_ckpt8", t)(dy, want[3], emb, want[1], want[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fn("out_fwd_ckpt8", t)(x, emb, stream=s)
    gdx, gd = fn("out_bwd_ckpt8", t)(dy, got[3], emb, got[1], got[2], stream=s)
    o = fn("out_again_ckpt8", t)(got[3], emb, got[1], got[2], stream=s.cuda_stream)
    s.synchronize()
    assert all(same(a, b) for a, b in zip((*got, gdx, gd), (*want, wdx, wd)))
    buf = [torch.empty_like(v) for v in (*want, wdx, wd)]
    ws = torch.empty(binding.adaln_out_bwd_ckpt8_workspace_bytes(2, 45, 264), dtype=torch.uint8, device="cuda")
    xs, again_out = x.clone(), torch.empty_like(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn("out_fwd_ckpt8", t)(xs, emb, *buf[:4])
        fn("out_bwd_ckpt8", t)(dy, buf[3], emb, buf[1], buf[2], buf[4], buf[5], workspace=ws)
        fn("out_again_ckpt8", t)(buf[3], emb, buf[1], buf[2], again_out)
    for k in range(3):
        xs.copy_(x.roll(k, 1))
        for v in buf:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        w = fn("out_fwd_ckpt8", t)(xs, emb)
        e = fn("out_bwd_ckpt8", t)(dy, w[3], emb, w[1], w[2])
        assert all(same(a, b) for a, b in zip(buf, (*w, *e)))
        assert same(again_out, fn("out_again_ckpt8", t)(w[3], emb, w[1], w[2]))


def test_refusals():
    t = torch.bfloat16
    x, dy, emb = norm_inputs(t, 2, 5, 64)
    out, mean, rstd, ckpt = binding.adaln_out_fwd_ckpt8(x, emb)
    with pytest.raises(TypeError):
        binding.adaln_ckpt8_pack(x.float())
    with pytest.raises(TypeError):
        binding.adaln_ckpt8_pack(x.cpu())
    with pytest.raises(ValueError):
        binding.adaln_ckpt8_pack(x[..., :60])
    with pytest.raises(ValueError):
        binding.adaln_ckpt8_unpack(ckpt, 72 + 64)
    with pytest.raises(ValueError):
        binding.adaln_out_bwd_ckpt8(dy[:, :4], ckpt, emb, mean, rstd)
    with pytest.raises(ValueError, match="workspace"):
        binding.adaln_out_bwd_ckpt8(dy, ckpt, emb, mean, rstd,
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.AdaLNError):
        binding.adaln_out_fwd_ckpt8(x, emb, eps=-1.0)
    with pytest.raises(binding.AdaLNError):
        binding.adaln_out_fwd_ckpt8(x, emb, out=x)
    big = torch.empty((1, 1, 4104), device="cuda")
    with pytest.raises(binding.AdaLNError):
        binding.adaln_f32_out_fwd_ckpt8(big, torch.empty((1, 8208), device="cuda"))
