"""adaln_qk_norm_rope_* in every form of its kernels: few rows one a lane, more
rows four a lane, and large calls through rings of tiles.  The size of a call
chooses; the bits of a row must not show it."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from test_gpu_heads import BF16, BWD, F32, FWD, check_both, make

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


def form(B, S, Hq, Hk, Dh):
    """The forward's form: rows a lane of the direct kernel (1 or 4), or "ring"."""
    lanes = 4
    while 8 * lanes < Dh:
        lanes *= 2
    per = 32 // lanes
    if B * S * (Hq + Hk) // (4 * per) < 16 * torch.cuda.get_device_properties(0).multi_processor_count:
        return 1
    h = max(Hq, Hk)

    def ceil(a, b):
        return -(-a // b)

    tasks = ceil(h, per * (2 if h > per else 1))
    tile = min(1 if tasks >= 24 else 24 // tasks, max(1, S // 64))
    return 4 if tile * ceil(Hq, per * (2 if h > per else 1)) < 16 else "ring"


# every lane count, whole and partial rows, heads that fill a warp's rows and not; [B, S] large enough for the
# ring and, as [B S / 40, 40], for four rows a lane
FORMS = [(2, 4000, 8, 5, 8, 8), (2, 4000, 5, 3, 40, 16), (2, 2000, 8, 4, 64, 64), (2, 2000, 6, 3, 72, 72),
         (2, 1200, 8, 4, 128, 128), (2, 1200, 5, 1, 136, 64), (2, 1200, 5, 2, 256, 256)]


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", FORMS)
def test_rows_do_not_show_the_form(shape, dtype, inter):
    """A row's bits are the same in a large call, in its sample's call, among
    many short samples, and in a call of a few tokens."""
    B, S, Hq, Hk, Dh, Dr = shape
    d = make(dtype, *shape, P=S)
    args = (d["wq"], d["wk"], d["cos"], d["sin"])
    yq, yk = FWD[dtype](d["q"], d["k"], *args, pos=d["pos"], interleaved=inter)
    short = (B * S // 40, 40)
    assert (form(B, S, Hq, Hk, Dh), form(*short, Hq, Hk, Dh), form(1, 40, Hq, Hk, Dh)) == ("ring", 4, 1)
    a, b = FWD[dtype](d["q"].view(*short, Hq, Dh), d["k"].view(*short, Hk, Dh), *args, pos=d["pos"].view(short),
                      interleaved=inter)
    assert torch.equal(a.view(yq.shape), yq) and torch.equal(b.view(yk.shape), yk)
    for i in range(B):
        a, b = FWD[dtype](d["q"][i:i + 1], d["k"][i:i + 1], *args, pos=d["pos"][i:i + 1], interleaved=inter)
        assert torch.equal(a[0], yq[i]) and torch.equal(b[0], yk[i])
    for s in range(0, S, 333):
        at = slice(s, s + 40)
        a, b = FWD[dtype](d["q"][:, at], d["k"][:, at], *args, pos=d["pos"][:, at], interleaved=inter)
        assert torch.equal(a, yq[:, at]) and torch.equal(b, yk[:, at])


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(150, 40, 12, 12, 8, 8), (200, 40, 5, 1, 40, 16), (90, 40, 7, 6, 96, 64),
                                   (60, 40, 5, 1, 256, 256)])
def test_four_rows_a_lane(shape, dtype, inter):
    """... against 64 bits."""
    assert form(*shape[:5]) == 4
    check_both(make(dtype, *shape, P=60), dtype, inter)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,S,kind", [(2, 2000, "ring"), (100, 40, 4)])
def test_layouts_of_large_calls(B, S, kind, dtype):
    """Fused buffers, in place, [B,H,S,Dh] storage, broadcast rows, padding that
    holds infinities and NaN: the bits of the dense call, and nothing else written."""
    Hq, Hk, Dh = 8, 4, 128
    assert form(B, S, Hq, Hk, Dh) == kind and form(B, S, Hq, 0, Dh) == kind
    d = make(dtype, B, S, Hq, Hk, Dh, 96, P=S)
    names = ("q", "k", "gq", "gk")
    want = calls(dtype, d, *(d[n] for n in names), inter=False)
    args = (d["wq"], d["wk"], d["cos"], d["sin"])
    bad = ((d["pos"] < 0) | (d["pos"] >= S))[:, :, None, None]
    assert bad.any() and not bad.all()
    for n, v in (("q", float("nan")), ("k", float("inf")), ("gq", float("-inf")), ("gk", float("nan"))):
        d[n] = torch.where(bad, torch.full_like(d[n], v), d[n])
    # one fused projection output: read, then normed in place; gradients into one fused buffer
    qkv = torch.cat((d["q"], d["k"], torch.full_like(d["k"], 3.0)), 2)
    q, k, v = qkv.split((Hq, Hk, Hk), 2)
    d_qkv = torch.full_like(qkv, 7.0)
    dq, dk, dv = d_qkv.split((Hq, Hk, Hk), 2)
    got = BWD[dtype](d["gq"], d["gk"], q, k, *args, pos=d["pos"], d_q=dq, d_k=dk, interleaved=False)
    assert all(torch.equal(a, b) for a, b in zip(got, want[2:])) and (dv == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(calls(dtype, d, q, k, d["gq"], d["gk"], inter=False), want))
    FWD[dtype](q, k, *args, pos=d["pos"], q_out=q, k_out=k, interleaved=False)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and (v == 3).all()
    # heads before tokens, outputs as rows 3 .. of a longer buffer, gradients in place
    turned = [d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in names]
    joint = torch.full((B, Hq, S + 8, Dh), 7.0, dtype=dtype, device="cuda")
    to = joint.transpose(1, 2)[:, 3:3 + S]
    a, b = FWD[dtype](*turned[:2], *args, pos=d["pos"], q_out=to, interleaved=False)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert (joint[:, :, :3] == 7).all() and (joint[:, :, 3 + S:] == 7).all()
    got = BWD[dtype](turned[2], turned[3], turned[0], turned[1], *args, pos=d["pos"], d_q=turned[2], d_k=turned[3],
                     interleaved=False)
    assert all(torch.equal(x, y) for x, y in zip(got, want[2:])) and torch.equal(turned[2], want[2])
    # one head, and one sample, broadcast
    for one in (d["k"][:, :, :1].expand(B, S, Hq, Dh), d["q"][:1].expand(B, S, Hq, Dh)):
        a, _ = FWD[dtype](one, None, *args, pos=d["pos"], interleaved=False)
        b, _ = FWD[dtype](one.contiguous(), None, *args, pos=d["pos"], interleaved=False)
        # bits: sample 0's padding, of NaN, is real in the others
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(a.view(bits), b.view(bits))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_rows_of_large_calls(dtype):
    """Samples 2^32 elements apart, through the ring."""
    B, S, H, Dh = 2, 2000, 6, 64
    d = make(dtype, B, S, H, H, Dh, 64, P=S)
    want = calls(dtype, d, d["q"], d["k"], d["gq"], d["gk"])
    far = (1 << 32) + 1024
    buf = torch.empty(far + S * 2 * H * Dh, dtype=dtype, device="cuda")
    qk = torch.as_strided(buf, (B, S, 2 * H, Dh), (far, 2 * H * Dh, Dh, 1))
    qk.copy_(torch.cat((d["q"], d["k"]), 2))
    q, k = qk.split(H, 2)
    got = calls(dtype, d, q, k, d["gq"], d["gk"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    FWD[dtype](q, k, d["wq"], d["wk"], d["cos"], d["sin"], pos=d["pos"], q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(2, 33, 1, 1, 64, 64), (1, 70, 3, 5, 128, 128), (2, 40, 5, 3, 32, 16),
                                   (2, 2000, 5, 3, 72, 72)])
def test_without_eps(shape, dtype, inter):
    """eps = 0, with lanes that hold no row: theirs would be of infinite length."""
    check_both(make(dtype, *shape, P=shape[1]), dtype, inter, eps=0.0)


def test_zero_rows_without_eps():
    """... and a row of zeros is 0 * inf, in itself and in dw alone."""
    d = make(BF16, 1, 50, 3, 1, 64, 64, pads=False)
    q = d["q"].clone()
    q[0, 7, 1] = 0
    y, _ = FWD[BF16](q, None, d["wq"], None, d["cos"], d["sin"], pos=d["pos"], eps=0.0)
    dq, _, _, _ = BWD[BF16](d["gq"], None, q, None, d["wq"], None, d["cos"], d["sin"], pos=d["pos"], eps=0.0)
    rest = torch.ones((50, 3), dtype=torch.bool, device="cuda")
    rest[7, 1] = False
    assert y[0, 7, 1].isnan().all() and y[0][rest].isfinite().all() and dq[0][rest].isfinite().all()
