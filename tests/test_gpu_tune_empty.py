"""The fine-tuning operators at sizes of zero, and adapters named the same way twice."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b
from test_gpu_lora import NAME, TYPES, fn, inputs, run, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("B,S", [(0, 5), (3, 0), (0, 0)])
def test_no_rows(t, B, S):
    D = 72
    x, emb = torch.zeros((B, S, D), dtype=t, device="cuda"), torch.zeros((B, 2 * D), dtype=t, device="cuda")
    rec = fn("ckpt8_pack", t)(x)
    assert rec.shape == (B, S, b.adaln_ckpt8_row_bytes(D)) and fn("ckpt8_unpack", t)(rec, D).shape == x.shape
    out, mean, rstd, ckpt = fn("out_fwd_ckpt8", t)(x, emb)
    assert out.shape == x.shape and ckpt.shape == rec.shape and mean.shape == (B, S)
    assert fn("out_again_ckpt8", t)(ckpt, emb, mean, rstd).shape == x.shape
    d_emb = torch.full((B, 2 * D), 3.0, device="cuda")
    dx, _ = fn("out_bwd_ckpt8", t)(x, ckpt, emb, mean, rstd, d_emb=d_emb)
    assert dx.shape == x.shape and (d_emb == 0).all()
    N, R, NA = 40, 8, 2
    A, U = torch.ones((NA, R, D), dtype=t, device="cuda"), torch.ones((NA, R, N), dtype=t, device="cuda")
    w = (A, U, torch.ones(NA, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda"))
    out, state = fn("lora_fwd", t)(x, *w)
    assert out.shape == (B, S, N)
    dA, dU = torch.full((NA, R, D), 3.0, device="cuda"), torch.full((NA, R, N), 3.0, device="cuda")
    dx, _, _ = fn("lora_bwd", t)(out, x, state, *w, dA_acc=dA, dU_acc=dU, accumulate=True)
    assert dx.shape == x.shape and (dA == 3).all() and (dU == 3).all()
    fn("lora_bwd", t)(out, x, state, *w, dA_acc=dA, dU_acc=dU)
    assert (dA == 0).all() and (dU == 0).all()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 16, 40, 700])
def test_back_to_back(t, S):
    """Calls that follow one another without a synchronization, their inputs written
    just before on the same stream: each reads what it is given."""
    B, K, N, R, NA = 5, 264, 328, 16, 3
    cases = [inputs(t, B, S, K, N, R, NA, seed=s) for s in range(4)]
    want = [run(t, c) for c in cases]
    c = {k: torch.zeros_like(v) if torch.is_tensor(v) else v for k, v in cases[0].items()}
    out, dx = torch.empty_like(c["y"]), torch.empty_like(c["x"])
    dA, dU = torch.empty((NA, R, K), device="cuda"), torch.empty((NA, R, N), device="cuda")
    ws = torch.empty(fn("lora_bwd_workspace_bytes", t)(B, S, K, N, R), dtype=torch.uint8, device="cuda")
    state = None
    got = []
    torch.cuda.synchronize()
    for _ in range(3):
        for v in cases:
            for k in c:
                if torch.is_tensor(c[k]):
                    c[k].copy_(v[k])
            w = (c["A"], c["U"], c["scale"], c["ids"])
            _, state = fn("lora_fwd", t)(c["x"], *w, y=c["y"], out=out, state=state)
            fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, dx_base=c["dx_base"], dx=dx, dA_acc=dA, dU_acc=dU,
                              workspace=ws)
            got.append([z.clone() for z in (out, dx, dA, dU)])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(same(a, e) for a, e in zip(g, want[i % 4])), i


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 40])
def test_inputs_of_the_kernel_before(t, S):
    """The base, ids and lens come from the last kernel before the call, a norm of this
    library among them, again and again into the same memory."""
    B, D = 4, 128
    gen = torch.Generator("cuda").manual_seed(1)
    xs = [torch.randn((B, S, D), generator=gen, device="cuda").to(t) for _ in range(6)]
    emb = torch.randn((B, 2 * D), generator=gen, device="cuda").to(t)
    c = inputs(t, B, S, D, D, 8, 2)
    y = torch.empty((B, S, D), dtype=t, device="cuda")
    w = (c["A"], c["U"], c["scale"], c["ids"])
    mean, rstd = torch.empty((B, S), device="cuda"), torch.empty((B, S), device="cuda")
    state = fn("lora_fwd", t)(c["x"], *w)[1]
    got = []
    torch.cuda.synchronize()
    for x in xs:
        fn("out_fwd", t)(x, emb, out=y, mean=mean, rstd=rstd)
        got.append(fn("lora_fwd", t)(c["x"], *w, y=y, state=state)[0])
    torch.cuda.synchronize()
    for x, g in zip(xs, got):
        out = fn("out_fwd", t)(x, emb)[0]
        torch.cuda.synchronize()
        assert same(g, fn("lora_fwd", t)(c["x"], *w, y=out)[0])


def test_the_same_adapter_throughout():
    """Every sample the same adapter, or an adapter each: the gradients of the samples
    alone add up in their order."""
    t = torch.bfloat16
    for S in (1, 30):
        c = inputs(t, 40, S, 64, 72, 8, 40)
        c["ids"] = torch.full((40,), 7, dtype=torch.int32, device="cuda")
        out, dx, dA, dU = run(t, c)
        c["ids"] = torch.arange(40, dtype=torch.int32, device="cuda")
        for k in ("A", "U", "scale"):
            c[k] = c[k][7:8].expand(c[k].shape).contiguous()
        out1, dx1, dA1, dU1 = run(t, c)
        assert same(out, out1) and same(dx, dx1)
        for one, each in ((dA, dA1), (dU, dU1)):
            s = torch.zeros_like(each[0])
            for e in each:
                s = s + e
            assert same(one[7], s) and (one[:7] == 0).all() and (one[8:] == 0).all()
