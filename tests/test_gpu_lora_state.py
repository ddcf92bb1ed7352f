"""What the adapters' gradients take: h and e, read through calls whose d_out (or x) has
one element in a row, so that dU[a,r,n] is h of row n, dA[a,r,k] is e of row k, and every
sum has one term."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b
from ops_ref import U
from test_gpu_lora import NAME, TYPES, fn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    torch.cuda.synchronize()
    assert b.device_error() == 0


def states(t, x, A, scale):
    """h = scale x A^T of one sample's rows as the gradients take it, both ways: as the
    forward's (dU) and as the backward's (dA, with U = A and d_out = x)."""
    _, S, K = x.shape
    R = A.shape[1]
    one = torch.eye(S, (S + 7) // 8 * 8, device="cuda").to(t)[None].contiguous()
    other = torch.zeros((1, R, one.shape[-1]), dtype=t, device="cuda")
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, state = fn("lora_fwd", t)(x, A, other, scale, ids)
    dU = fn("lora_bwd", t)(one, x, state, A, other, scale, ids)[2]
    _, state = fn("lora_fwd", t)(one, other, A, scale, ids)
    dA = fn("lora_bwd", t)(x, one, state, other, A, scale, ids)[1]
    return dU[0, :, :S].T, dA[0, :, :S].T


LONG = [(768, 16), (776, 16), (6144, 24), (6152, 16), (9216, 32), (12296, 48), (16384, 64), (20000, 128), (24584, 64),
        (32768, 8), (49160, 32), (65536, 16), (65536, 24), (65536, 72), (65536, 128)]


@pytest.mark.parametrize("K,R", LONG)
@pytest.mark.parametrize("sign", ["any", "one"])
def test_long_rows(K, R, sign):
    """An accumulator takes at most 48 instructions of 16 products, and each may truncate
    what it adds: 2 U of the sum of the magnitudes.  At most 11 accumulators of a range, 8
    ranges, the scale and the parts are rounded, U each; counted as 2 U they cover what
    the truncated steps carry into them."""
    t = torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(K + R)
    x = torch.randn((1, 130, K), generator=gen, device="cuda")
    A = torch.randn((1, R, K), generator=gen, device="cuda") / K ** 0.5
    if sign == "one":
        x, A = x.abs(), A.abs()
    x, A = x.to(t), A.to(t)
    scale = torch.tensor([0.75], device="cuda")
    want = 0.75 * (x[0].double() @ A[0].double().T)
    size = 0.75 * (x[0].double().abs() @ A[0].double().abs().T)
    bound = (48 + 11 + 8 + 2) * 2 * U * size
    for got in states(t, x, A, scale):
        off = (got.double() - want).abs() / bound
        assert (off <= 1).all(), off.max()


def whole_numbers(B, S, R, C, gen):
    """src [B,S,C] and W [2,R,C] in bf16 whose products src W^T are whole numbers of 24 bits,
    with a different number for most rows and ranks: 2^16 of 8 bits, 2^8 of two times 4, and
    two times 4.  No sum of the terms needs more than 24 bits."""
    def draw(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen)

    at = torch.randperm(C, generator=gen)[:3]
    src, W = torch.zeros(B, S, C), torch.zeros(2, R, C)
    src[..., at[0]] = 1
    src[..., at[1:]] = draw(1, 15, B, S, 2).float()
    W[..., at[0]] = draw(128, 255, 2, R).float() * 2 ** 16
    W[..., at[1]] = draw(1, 15, 2, R).float() * 2 ** 8
    W[..., at[2]] = draw(1, 15, 2, R).float()
    return src.bfloat16().cuda(), W.bfloat16().cuda()


@pytest.mark.parametrize("S,lens", [(150, None), (600, None), (700, [700, 513, 64])])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 48, 56, 64, 72, 80, 88, 104, 120, 128])
def test_every_part_of_a_state(R, S, lens):
    """The gradients take h and e whole: with whole numbers of 24 bits, of which two bf16
    parts hold 16 or 17, they are exact, in pieces and by owners."""
    t = torch.bfloat16
    B, C = 3, 72
    gen = torch.Generator().manual_seed(R + S)
    src, W = whole_numbers(B, S, R, C, gen)
    ids = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    n = torch.tensor(lens or [S] * B)
    N = (B * S + 7) // 8 * 8
    one = torch.eye(B * S, N).view(B, S, N)  # row s of sample i: 1 or -2 in channel i S + s
    one[1] *= -2
    one = one.to(t).cuda()
    other = torch.zeros((2, R, N), dtype=t, device="cuda")
    scale = torch.tensor([1.0, 0.25], device="cuda")
    kw = dict(lens=None if lens is None else n.int().cuda())
    # what the sums are: one term each
    s, w = src.cpu().double(), W.cpu().double()
    want = torch.zeros(2, R, N, dtype=torch.float64)
    for i, a in enumerate(ids.tolist()):
        h = scale.cpu().double()[a] * (s[i] @ w[a].T)
        hi = h.float().bfloat16().double()
        mid = (h - hi).float().bfloat16().double()
        assert ((hi + mid) != h).float().mean() > 0.3  # two parts are not enough
        h[n[i]:] = 0
        want[a][:, i * S:(i + 1) * S] = h.T * (-2 if i == 1 else 1)
    _, state = b.adaln_lora_fwd(src, W, other, scale, ids, **kw)
    dU = b.adaln_lora_bwd(one, src, state, W, other, scale, ids, **kw)[2]
    assert torch.equal(dU.cpu().double(), want)
    _, state = b.adaln_lora_fwd(one, other, W, scale, ids, **kw)
    dA = b.adaln_lora_bwd(src, one, state, other, W, scale, ids, **kw)[1]
    assert torch.equal(dA.cpu().double(), want)


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 2, 3, 9])
@pytest.mark.parametrize("K,R", [(8, 8), (264, 16), (3080, 32), (9216, 8), (65536, 24)])
def test_few_tokens(t, S, K, R):
    """On the CUDA cores each of 128 threads sums its 16-byte vectors, even and odd
    channels apart, by fused multiply-adds; then the halves, 32 lanes, 4 warps and the
    scale: that many roundings of at most U."""
    gen = torch.Generator("cuda").manual_seed(K + R + S)
    for sign in (False, True):
        x = torch.randn((1, S, K), generator=gen, device="cuda")
        A = torch.randn((1, R, K), generator=gen, device="cuda") / K ** 0.5
        if sign:
            x, A = x.abs(), A.abs()
        x, A = x.to(t), A.to(t)
        scale = torch.tensor([0.7], device="cuda")
        w = scale.double()
        want = w * (x[0].double() @ A[0].double().T)
        size = w * (x[0].double().abs() @ A[0].double().abs().T)
        E = 16 // x.element_size()
        steps = -(-K // (128 * E)) * E // 2 + 1 + 5 + 3 + 1
        for got in states(t, x, A, scale):
            off = (got.double() - want).abs() / (steps * 1.001 * U * size)
            assert (off <= 1).all(), off.max()
