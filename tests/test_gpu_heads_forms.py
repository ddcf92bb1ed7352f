"""adaln_qk_norm_rope_* in every form of its kernels: few rows one a lane, more
rows four a lane, and large calls through rings of tiles.  The size of a call
chooses; the bits of a row must not show it."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from test_gpu_heads import BF16, BWD, F32, FWD, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def calls(dtype, d, q, k, gq, gk, inter=True, **out):
    args = (d["wq"], d["wk"], d["cos"], d["sin"])
    return (*FWD[dtype](q, k, *args, pos=d["pos"], interleaved=inter),
            *BWD[dtype](gq, gk, q, k, *args, pos=d["pos"], interleaved=inter))


@pytest.mark.parametrize("B,S", [(2, 37), (2, 20000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dh", [8, 64, 128, 256])
def test_stride_of_one_head_is_not_used(dtype, Dh, B, S):
    """One head cut out of rows whose head stride is no multiple of 16 bytes, as
    queries beside several keys and as keys beside several queries."""
    pad = 4 if dtype == BF16 else 2  # two heads' rows of Dh + pad are a multiple of 16 bytes, one is not
    for Hq, Hk in ((1, 3), (3, 1)):
        d = make(dtype, B, S, Hq, Hk, Dh, 8, P=50)

        def cut(t):
            if t.shape[2] > 1:
                return t
            wide = torch.zeros((B, S, 2, Dh + pad), dtype=dtype, device="cuda")
            one = wide[:, :, :1, :Dh]
            assert one.stride(2) * one.element_size() % 16 and not one.stride(1) * one.element_size() % 16
            return one.copy_(t)

        names = ("q", "k", "gq", "gk")
        want = calls(dtype, d, *(d[n] for n in names))
        got = calls(dtype, d, *(cut(d[n]) for n in names))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # in place, where the rows cannot be copied first
        q, k, gq, gk = (cut(d[n]) for n in names)
        args = (d["wq"], d["wk"], d["cos"], d["sin"])
        BWD[dtype](gq, gk, q, k, *args, pos=d["pos"], d_q=gq, d_k=gk)
        FWD[dtype](q, k, *args, pos=d["pos"], q_out=q, k_out=k)
        assert all(torch.equal(a, b) for a, b in zip((q, k, gq, gk), want))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_of_one_sample_or_token_are_not_used(dtype):
    for B, S in ((1, 30), (30, 1), (1, 1)):
        d = make(dtype, B, S, 4, 2, 64, 64)

        def odd(t):
            st = [n if m > 1 else 3 for n, m in zip(t.stride(), t.shape)]
            return torch.as_strided(t, t.shape, st)

        names = ("q", "k", "gq", "gk")
        want = calls(dtype, d, *(d[n] for n in names))
        got = calls(dtype, d, *(odd(d[n]) for n in names))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_given_accumulators_are_filled(dtype):
    """Whatever want_w says: it allocates those not given."""
    d = make(dtype, 3, 20, 4, 2, 64, 32)

    def back(k=True, **kw):
        keys = (d["gk"], d["k"]) if k else (None, None)
        return BWD[dtype](d["gq"], keys[0], d["q"], keys[1], d["wq"], d["wk"], d["cos"], d["sin"], pos=d["pos"], **kw)

    want = back()
    full = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    added = back(dwq_acc=full[0].clone(), dwk_acc=full[1].clone(), accumulate=True)[2:]
    for want_w in (True, False):
        for give in ((0,), (1,), (0, 1)):
            acc = [full[i].clone() if i in give else None for i in range(2)]
            got = back(dwq_acc=acc[0], dwk_acc=acc[1], want_w=want_w)
            for i in range(2):
                if i in give:
                    assert got[2 + i] is acc[i] or got[2 + i].data_ptr() == acc[i].data_ptr()
                if i in give or want_w:
                    assert torch.equal(got[2 + i], want[2 + i])
                else:
                    assert got[2 + i] is None
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            if len(give) == 2 or not want_w:
                acc = [full[i].clone() if i in give else None for i in range(2)]
                got = back(dwq_acc=acc[0], dwk_acc=acc[1], want_w=want_w, accumulate=True)
                for i in range(2):
                    assert torch.equal(acc[i], added[i]) if i in give else got[2 + i] is None
    alone = back(k=False, want_w=False, dwq_acc=full[0].clone())
    assert torch.equal(alone[2], back(k=False)[2]) and alone[1] is None and alone[3] is None


def test_nothing_for_keys_without_keys():
    d = make(BF16, 1, 5, 4, 2, 64, 32)
    args = (None, d["wq"], d["wk"], d["cos"], d["sin"])
    with pytest.raises(ValueError, match="k_out"):
        FWD[BF16](d["q"], *args, k_out=torch.empty_like(d["k"]))
    w = torch.zeros(64, device="cuda")
    for name, value in (("d_k", torch.empty_like(d["k"])), ("dwk_acc", w)):
        for want_w in (True, False):
            with pytest.raises(ValueError, match=name):
                BWD[BF16](d["gq"], None, d["q"], *args, want_w=want_w, **{name: value})
    with pytest.raises(ValueError, match="d_k_out"):
        BWD[BF16](d["gq"], d["gk"], d["q"], *args)
    assert FWD[BF16](d["q"], *args)[1] is None
