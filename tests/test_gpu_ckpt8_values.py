"""The norm with records where x, dy or the modulation hold infinities and NaN: the bits
of the calls without records at the values that the records stand for."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from test_gpu_ckpt8 import NAME, TYPES, fn, norm_inputs, same
from tune_ref import again, record_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("D", [72, 264, 1160, 2056, 3072, 4096])
def test_infinities_and_nan(t, D):
    B, S = 2, 70
    for where in ("x", "dy", "emb", "large"):
        x, dy, emb = norm_inputs(t, B, S, D, seed=5)
        v = {"x": x, "dy": dy, "emb": emb, "large": x}[where]
        if where == "large":  # the last scale, and squares past the range
            x[0, 3, ::3] = torch.finfo(t).max
            x[1, 69] = -torch.finfo(t).max
            x[0, 64, 40:] = 2.0 ** -130
        else:
            v.view(-1)[7], v.view(-1)[-3], v.view(-1)[D // 2] = float("inf"), float("nan"), float("-inf")
        out, mean, rstd, ckpt = fn("out_fwd_ckpt8", t)(x, emb)
        assert all(same(p, q) for p, q in zip((out, mean, rstd), fn("out_fwd", t)(x, emb))), where
        assert torch.equal(ckpt.cpu(), record_of(x)), where
        x8 = fn("ckpt8_unpack", t)(ckpt, D)
        got = fn("out_bwd_ckpt8", t)(dy, ckpt, emb, mean, rstd)
        assert all(same(p, q) for p, q in zip(got, fn("out_bwd", t)(dy, x8, emb, mean, rstd))), where
        o, want = fn("out_again_ckpt8", t)(ckpt, emb, mean, rstd), again(x8, emb, mean, rstd)
        assert torch.equal(o.isnan().cpu(), want.isnan()), where
        assert same(o.cpu().nan_to_num(3.0), want.nan_to_num(3.0)), where
