"""Fine-tuning the projection behind a modulated norm, as the calls are used
together: the norm keeps its input in 8 bits, the projection has adapters, the
backward takes the projection's input again from the records."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b
from ops_ref import check
from tune_ref import Lora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def step(c, buf=None):
    """Conditioning with an adapter of its own, norm, projection with adapters;
    backward.  `buf`: a dict to take outputs from (a captured call)."""
    o = buf if buf is not None else {}
    adapters = (c["A"], c["U"], c["scale"], c["ids"])
    cond = (c["Ac"], c["Uc"], c["scale"], c["ids"])
    emb, u = b.adaln_proj_fwd(c["temb"], c["W"], c["bias"])
    emb3, cstate = b.adaln_lora_fwd(u[:, None], *cond, y=emb[:, None], out=emb[:, None])
    out, mean, rstd, ckpt = b.adaln_out_fwd_ckpt8(c["x"], emb)
    y = out @ c["Wp"].T
    y, state = b.adaln_lora_fwd(out, *adapters, y=y, lens=c["lens"], out=y)
    del out
    base = c["g"] @ c["Wp"]
    again = b.adaln_out_again_ckpt8(ckpt, emb, mean, rstd)
    d_norm, dA, dU = b.adaln_lora_bwd(c["g"], again, state, *adapters, lens=c["lens"], dx_base=base, dx=base)
    dx, d_emb = b.adaln_out_bwd_ckpt8(d_norm, ckpt, emb, mean, rstd)
    d_u, dAc, dUc = b.adaln_lora_bwd(d_emb.bfloat16()[:, None], u[:, None], cstate, *cond)
    r = dict(emb=emb, y=y, again=again, d_norm=d_norm, dx=dx, d_emb=d_emb, dA=dA, dU=dU, d_u=d_u, dAc=dAc, dUc=dUc)
    for k, v in r.items():
        if buf is not None:
            o[k].copy_(v)
    return r


def inputs(B=3, S=70, D=128, N=192, R=16, NA=2):
    gen = torch.Generator("cuda").manual_seed(11)

    def normal(*s, f=1.0):
        return (f * torch.randn(s, generator=gen, device="cuda")).bfloat16()

    return dict(x=normal(B, S, D), temb=normal(B, D), W=normal(2 * D, D, f=0.05), bias=normal(2 * D, f=0.05),
                Wp=normal(N, D, f=0.1), A=normal(NA, R, D, f=0.1), U=normal(NA, R, N, f=0.1),
                Ac=normal(NA, R, D, f=0.1), Uc=normal(NA, R, 2 * D, f=0.1),
                scale=torch.tensor([1.0, 0.5], device="cuda"),
                ids=torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda"),
                lens=torch.tensor([S, S, S - 7], dtype=torch.int32, device="cuda"), g=normal(B, S, N))


def test_step():
    c = inputs()
    r = step(c)
    D = c["x"].shape[-1]
    # each call at the inputs that the step gave it
    emb, mean, rstd = r["emb"], *b.adaln_out_fwd(c["x"], r["emb"])[1:]
    x8 = b.adaln_ckpt8_unpack(b.adaln_ckpt8_pack(c["x"]), D)
    dx, d_emb = b.adaln_out_bwd(r["d_norm"], x8, emb, mean, rstd)
    assert torch.equal(bits(dx), bits(r["dx"])) and torch.equal(bits(d_emb), bits(r["d_emb"]))
    out = b.adaln_out_fwd(c["x"], emb)[0]
    # 8 bits: half a step of a group, over the row's spread and times (1 + scale), and two bf16 roundings
    half = x8.double().sub(c["x"].double()).abs()
    onep = (1 + emb[:, None, :D].double()).abs()
    bound = half * rstd[..., None].double() * onep * 1.01 + 2.0 ** -7 * out.double().abs() + 1e-5
    assert ((r["again"].double() - out.double()).abs() <= bound).all()
    ref = Lora(r["again"], c["A"], c["U"], c["scale"], c["ids"], None, c["lens"], c["g"], c["g"] @ c["Wp"])
    ref.check_rows(r["d_norm"], ref.dx, ref.dx_err, c["g"] @ c["Wp"], "d_norm")
    check(r["dA"], ref.dA, ref.dA_err, "dA")
    # dU is h (from the forward's own input) times g
    ref = Lora(out, c["A"], c["U"], c["scale"], c["ids"], out @ c["Wp"].T, c["lens"], c["g"], None)
    check(r["dU"], ref.dU, ref.dU_err, "dU")
    ref.check_rows(r["y"], ref.out, ref.out_err, out @ c["Wp"].T, "y")
    emb0, u = b.adaln_proj_fwd(c["temb"], c["W"], c["bias"])
    ref = Lora(u[:, None], c["Ac"], c["Uc"], c["scale"], c["ids"], emb0[:, None], None,
               r["d_emb"].bfloat16()[:, None], None)
    ref.check_rows(r["emb"][:, None], ref.out, ref.out_err, 0.0, "emb")
    check(r["dUc"], ref.dU, ref.dU_err, "dUc")
    check(r["dAc"], ref.dA, ref.dA_err, "dAc")


def test_step_captured():
    """Captured while an eager step's results live, and replayed on other inputs."""
    c = inputs()
    eager = step(c)
    held = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    buf = {k: torch.zeros_like(v) for k, v in eager.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(held)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(held, buf)
    for k in range(3):
        for n in ("x", "temb", "g"):
            held[n].copy_(c[n].roll(k, 0))
        g.replay()
        torch.cuda.synchronize()
        want = step({**c, **{n: held[n] for n in ("x", "temb", "g")}})
        for n, v in want.items():
            assert torch.equal(bits(buf[n]), bits(v)), (k, n)


def test_two_streams_at_once():
    """Two steps on two streams, each with its own state and workspaces."""
    c1, c2 = inputs(), inputs(S=45)
    want = [step(c1), step(c2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, c in zip(streams, (c1, c2)):
            with torch.cuda.stream(s):
                got.append(step(c))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for n in w:
                assert torch.equal(bits(g[n]), bits(w[n])), n
