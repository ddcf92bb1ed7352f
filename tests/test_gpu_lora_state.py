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
