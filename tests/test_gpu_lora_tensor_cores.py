"""Far offsets, large and small states, inputs of the kernel before and one adapter for
all, at sizes that run on the tensor cores (bf16, S >= 12 and S R >= 640)."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b
from ops_ref import check
from test_gpu_lora import inputs, run, same, verify
from tune_ref import Lora

pytestmark = pytest.mark.gpu
T = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    torch.cuda.synchronize()
    assert b.device_error() == 0


@pytest.mark.parametrize("S,R", [(40, 16), (40, 72), (150, 8), (600, 16)])
def test_far_offsets(S, R):
    """Rows whose offsets pass 2^32 elements: samples far apart, and tokens far apart."""
    B, K, N = 2, 64, 72
    c = inputs(T, B, S, K, N, R, 1)
    want = run(T, c)
    verify(T, c, want)
    big = torch.empty((1 << 32) + (1 << 22), dtype=T, device="cuda")
    w = (c["A"], c["U"], c["scale"], c["ids"])
    for batch, token in (((1 << 32) + 4096, 128), (128, ((1 << 32) + 4096) // (S - 1) // 8 * 8)):
        def place(width, k, fill):
            start = k * (1 << 18) if batch > token else k * 512
            return big.as_strided((B, S, width), (batch, token, 1), start).copy_(fill)

        x, d_out = place(K, 0, c["x"]), place(N, 1, c["d_out"])
        y, base = place(N, 2, c["y"]), place(K, 3, c["dx_base"])
        out, dx = place(N, 4, torch.full_like(c["y"], 7)), place(K, 5, torch.full_like(c["x"], 7))
        assert (x[-1, -1].data_ptr() - x.data_ptr()) // 2 >= 1 << 32 or token > batch
        _, state = b.adaln_lora_fwd(x, *w, y=y, out=out)
        _, dA, dU = b.adaln_lora_bwd(d_out, x, state, *w, dx_base=base, dx=dx)
        assert all(same(p, q) for p, q in zip((out, dx, dA, dU), want))


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 125, 2.0 ** -100])
@pytest.mark.parametrize("S,R", [(40, 16), (150, 64), (600, 16)])
def test_large_and_small_states(S, R, size):
    """h near the ends of what bf16 and fp32 hold, in out and in the gradients."""
    c = inputs(T, 2, S, 64, 72, R, 1)
    c["ids"].fill_(0)
    c["scale"].fill_(size)
    c["U"] = (c["U"].float() / size).to(T)
    c["y"].zero_()
    w = (c["A"], c["U"], c["scale"], c["ids"])
    out, state = b.adaln_lora_fwd(c["x"], *w, y=c["y"])
    d_out = (c["d_out"].float() / size).to(T)
    _, dA, dU = b.adaln_lora_bwd(d_out, c["x"], state, *w, want_x=False)
    r = Lora(c["x"], *w, c["y"], None, d_out, None)
    check(out, r.out, r.out_err, "out")
    check(dU, r.dU, r.dU_err, "dU")
    # e = scale sum_n d_out U, a sum in fp32: its terms are of the size of size^-2, which is
    # below 2^-180 (fp32's smallest number is 2^-149: the sum is zero) or above 2^180
    # (infinite or, of both signs, NaN)
    assert (dA == 0).all() if size > 1 else not dA.isfinite().any()


def test_above_what_the_tensor_cores_hold():
    """An |h| above bf16's largest finite number counts as infinite, and nothing else
    changes."""
    S, R = 40, 16
    c = inputs(T, 2, S, 64, 72, R, 1)
    c["ids"].fill_(0)
    c["y"].zero_()
    c["x"].zero_()
    c["A"].zero_()
    c["x"][:, :, 0], c["A"][:, 3, 0] = 1, 1
    c["x"][0, 5, 0] = 2.0  # the others' h[3] is 2^127 (1 + 255/256) / 2
    c["scale"].fill_(2.0 ** 126 * (2 - 2.0 ** -8))
    c["U"].zero_()
    c["U"][:, 3] = 2.0 ** -100
    w = (c["A"], c["U"], c["scale"], c["ids"])
    out, state = b.adaln_lora_fwd(c["x"], *w, y=c["y"])
    _, _, dU = b.adaln_lora_bwd(c["d_out"], c["x"], state, *w, want_x=False)
    r = Lora(c["x"], *w, c["y"], None, c["d_out"], None)
    assert float(r.h.max()) > torch.finfo(T).max and float(r.h.max()) < torch.finfo(torch.float32).max
    inf = torch.zeros(2, S, 72, dtype=torch.bool)
    inf[0, 5] = True
    assert torch.equal(out.isinf().cpu(), inf)
    keep = ~inf
    assert ((out.cpu().double() - r.out).abs() <= r.out_err)[keep].all()
    dU = dU.cpu()
    assert not dU[0, 3].isfinite().any() and (dU[0, :3] == 0).all() and (dU[0, 4:] == 0).all()


@pytest.mark.parametrize("S,R", [(40, 16), (300, 16), (40, 104)])
def test_inputs_of_the_kernel_before(S, R):
    """x, the base, d_out, ids and lens come from the last kernels before the call, a norm
    of this library among them, again and again into the same memory."""
    B, D = 4, 128
    gen = torch.Generator("cuda").manual_seed(1)
    xs = [torch.randn((B, S, D), generator=gen, device="cuda").to(T) for _ in range(6)]
    ids = [torch.randint(-1, 3, (B,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(6)]
    lens = [torch.randint(0, S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32) for _ in range(6)]
    emb = torch.randn((B, 2 * D), generator=gen, device="cuda").to(T)
    c = inputs(T, B, S, D, D, R, 2)
    w = (c["A"], c["U"], c["scale"])
    buf, i, n = torch.empty((B, S, D), dtype=T, device="cuda"), ids[0].clone(), lens[0].clone()
    mean, rstd = torch.empty((B, S), device="cuda"), torch.empty((B, S), device="cuda")

    def norm(x, out):
        return b.adaln_out_fwd(x, emb, out=out, mean=mean, rstd=rstd)

    def calls(v, i, n):
        """v is x and d_out, then y and dx_base."""
        out, state = b.adaln_lora_fwd(v, *w, i, y=c["y"], lens=n)
        out2, _ = b.adaln_lora_fwd(c["x"], *w, i, y=v, lens=n)
        return [out, out2, *b.adaln_lora_bwd(v, c["x"], state, *w, i, lens=n, dx_base=c["dx_base"]),
                *b.adaln_lora_bwd(c["d_out"], v, state, *w, i, lens=n, dx_base=v)]

    got = []
    torch.cuda.synchronize()
    for k, x in enumerate(xs):
        i.copy_(ids[k])
        n.copy_(lens[k])
        norm(x, buf)
        got.append(calls(buf, i, n))
    torch.cuda.synchronize()
    for k, x in enumerate(xs):
        out = norm(x, torch.empty_like(buf))[0]
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(got[k], calls(out, ids[k], lens[k]))), k


@pytest.mark.parametrize("S,R", [(30, 24), (100, 64), (600, 16)])
def test_the_same_adapter_throughout(S, R):
    """Every sample the same adapter, or an adapter each: the gradients of the samples
    alone add up in their order."""
    c = inputs(T, 40, S, 64, 72, R, 40)
    c["ids"] = torch.full((40,), 7, dtype=torch.int32, device="cuda")
    out, dx, dA, dU = run(T, c)
    c["ids"] = torch.arange(40, dtype=torch.int32, device="cuda")
    for k in ("A", "U", "scale"):
        c[k] = c[k][7:8].expand(c[k].shape).contiguous()
    out1, dx1, dA1, dU1 = run(T, c)
    assert same(out, out1) and same(dx, dx1)
    if S > 512:  # pieces of a sample are added one by one
        return
    for one, each in ((dA, dA1), (dU, dU1)):
        s = torch.zeros_like(each[0])
        for e in each:
            s = s + e
        assert same(one[7], s) and (one[:7] == 0).all() and (one[8:] == 0).all()
