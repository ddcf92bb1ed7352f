"""adaln_qk_norm_rope_*: head rows against the 64-bit form, and what must hold
bit for bit."""

from __future__ import annotations

import pytest
import torch

import ops_ref
from gpu_util import lib
from invariant_dit_adaln_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FWD = {BF16: binding.adaln_qk_norm_rope_fwd, F32: binding.adaln_f32_qk_norm_rope_fwd}
BWD = {BF16: binding.adaln_qk_norm_rope_bwd, F32: binding.adaln_f32_qk_norm_rope_bwd}


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def tables(P, Dr):
    inv = 10000.0 ** (-torch.arange(Dr // 2, dtype=torch.float64) / max(1, Dr // 2))
    a = torch.arange(P, dtype=torch.float64)[:, None] * inv
    return a.cos().float().cuda(), a.sin().float().cuda()


def make(dtype, B, S, Hq, Hk, Dh, Dr, seed=0, P=None, pads=True):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g)

    size = torch.exp(rand(B, S, 1, 1))
    d = {"q": rand(B, S, Hq, Dh) * size, "k": rand(B, S, Hk, Dh) * size, "gq": rand(B, S, Hq, Dh),
         "gk": rand(B, S, Hk, Dh), "wq": 1 + 0.2 * rand(Dh), "wk": 1 + 0.2 * rand(Dh)}
    d = {n: t.to(dtype).cuda() for n, t in d.items()}
    P = P or S + 3
    d["cos"], d["sin"] = tables(P, Dr)
    pos = torch.randint(0, P, (B, S), generator=g)
    if pads:
        pos[torch.rand((B, S), generator=g) < 0.2] = -1
        pos[torch.rand((B, S), generator=g) < 0.1] = P
    d["pos"] = pos.cuda()
    return d


def check_both(d, dtype, interleaved, eps=1e-6):
    q, k, pos = d["q"], d["k"], d["pos"]
    yq, yk = FWD[dtype](q, k, d["wq"], d["wk"], d["cos"], d["sin"], pos=pos, eps=eps, interleaved=interleaved)
    dq, dk, dwq, dwk = BWD[dtype](d["gq"], d["gk"], q, k, d["wq"], d["wk"], d["cos"], d["sin"], pos=pos, eps=eps,
                                  interleaved=interleaved)
    for n, x, gy, w, y, dx, dw in (("q", q, d["gq"], d["wq"], yq, dq, dwq), ("k", k, d["gk"], d["wk"], yk, dk, dwk)):
        B, S, H, Dh = x.shape
        want, err = ops_ref.heads_fwd(x, w, d["cos"], d["sin"], pos, eps, interleaved)
        ops_ref.check(y, want, err, n)
        want, err, want_w, err_w = ops_ref.heads_bwd(gy, x, w, d["cos"], d["sin"], pos, eps, interleaved)
        ops_ref.check(dx, want, err, "d" + n)
        ops_ref.check(dw, want_w, err_w, "dw" + n)
    return yq, yk, dq, dk, dwq, dwk


# head sizes at both sides of each lane count, rotations of a part and none, odd
# head counts, one token, one row, shared key heads
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 1, 24, 24, 128, 128), (3, 7, 5, 2, 32, 16), (2, 33, 3, 1, 40, 40),
          (1, 50, 16, 4, 64, 32), (5, 9, 12, 12, 72, 72), (2, 65, 9, 3, 96, 64), (1, 129, 24, 24, 128, 128),
          (2, 17, 7, 7, 136, 8), (1, 40, 8, 2, 256, 256), (1, 31, 33, 1, 256, 0), (6, 3, 2, 2, 16, 0)]


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_64_bits(shape, dtype, interleaved):
    check_both(make(dtype, *shape), dtype, interleaved)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_rows(dtype):
    """Enough rows for the forms that take several heads a warp."""
    check_both(make(dtype, 2, 1000, 24, 6, 128, 128), dtype, True)
    check_both(make(dtype, 2, 1500, 10, 10, 64, 32), dtype, False)


def test_no_weights_no_keys_no_positions():
    d = make(BF16, 2, 10, 4, 4, 64, 64, pads=False)
    y, none = FWD[BF16](d["q"], None, None, None, d["cos"], d["sin"])
    assert none is None
    want, err = ops_ref.heads_fwd(d["q"], None, d["cos"], d["sin"], None, 1e-6, True)
    ops_ref.check(y, want, err, "q")
    dq, dk, dwq, dwk = BWD[BF16](d["gq"], None, d["q"], None, None, None, d["cos"], d["sin"])
    want, err, want_w, err_w = ops_ref.heads_bwd(d["gq"], d["q"], None, d["cos"], d["sin"], None, 1e-6, True)
    ops_ref.check(dq, want, err, "dq")
    ops_ref.check(dwq, want_w, err_w, "dwq")
    assert dk is None and dwk is None
    # the norm alone
    y, _ = FWD[BF16](d["q"], None, d["wq"], None, None, None)
    want, err = ops_ref.heads_fwd(d["q"], d["wq"], d["cos"][:, :0], d["sin"][:, :0], None, 1e-6, True)
    ops_ref.check(y, want, err, "norm")
    # without weight gradients, int32 positions
    dq2, _, w, _ = BWD[BF16](d["gq"], None, d["q"], None, None, None, d["cos"], d["sin"],
                             pos=torch.arange(10, dtype=torch.int32, device="cuda").expand(2, 10), want_w=False)
    assert w is None and torch.equal(dq, dq2)


def test_empty():
    d = make(BF16, 2, 4, 4, 2, 64, 64)
    for cut in (lambda t: t[:0], lambda t: t[:, :0]):
        q, k, gq, gk, pos = (cut(d[n]) for n in ("q", "k", "gq", "gk", "pos"))
        yq, yk = FWD[BF16](q, k, d["wq"], d["wk"], d["cos"], d["sin"], pos=pos)
        assert yq.shape == q.shape and yk.shape == k.shape
        one = torch.ones(64, device="cuda")
        _, _, dwq, dwk = BWD[BF16](gq, gk, q, k, d["wq"], d["wk"], d["cos"], d["sin"], pos=pos, dwq_acc=one.clone())
        assert not dwq.any() and not dwk.any()
        _, _, dwq, dwk = BWD[BF16](gq, gk, q, k, d["wq"], d["wk"], d["cos"], d["sin"], pos=pos, dwq_acc=one.clone(),
                                   dwk_acc=one.clone(), accumulate=True)
        assert torch.equal(dwq, one) and torch.equal(dwk, one)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_padding_is_not_read(dtype):
    """Infinities and NaN in padded rows change nothing; all rows padded gives zeros."""
    d = make(dtype, 3, 20, 4, 2, 64, 32)
    want = check_both(d, dtype, False)
    bad = ((d["pos"] < 0) | (d["pos"] >= d["cos"].shape[0]))[:, :, None, None]
    for n, v in (("q", float("nan")), ("k", float("inf")), ("gq", float("-inf")), ("gk", float("nan"))):
        d[n] = torch.where(bad, torch.full_like(d[n], v), d[n])
    d["pos"] = d["pos"].clone()
    yq, yk = FWD[dtype](d["q"], d["k"], d["wq"], d["wk"], d["cos"], d["sin"], pos=d["pos"], interleaved=False)
    got = (yq, yk, *BWD[dtype](d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["cos"], d["sin"], pos=d["pos"],
                               interleaved=False))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    none = torch.full_like(d["pos"], 1 << 40)
    out = BWD[dtype](d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["cos"], d["sin"], pos=none)
    assert all(not t.any() for t in out)


def test_infinite_row_stays_in_its_row():
    d = make(BF16, 1, 6, 4, 4, 64, 64, pads=False)
    yq, _ = FWD[BF16](d["q"], d["k"], d["wq"], d["wk"], d["cos"], d["sin"], pos=d["pos"])
    q = d["q"].clone()
    q[0, 2, 1, 5] = float("inf")
    got, _ = FWD[BF16](q, d["k"], d["wq"], d["wk"], d["cos"], d["sin"], pos=d["pos"])
    same = torch.ones((6, 4), dtype=torch.bool)
    same[2, 1] = False
    assert torch.equal(got[0][same], yq[0][same])
    assert got[0, 2, 1].isnan().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layouts(dtype):
    """Slices of fused buffers, [B,H,S,Dh] storage, broadcast inputs, in place,
    rows of a longer buffer: the bits of the dense call, and nothing else written."""
    B, S, Hq, Hk, Dh = 2, 21, 6, 2, 64
    d = make(dtype, B, S, Hq, Hk, Dh, 64)
    args = (d["wq"], d["wk"], d["cos"], d["sin"])
    yq, yk = FWD[dtype](d["q"], d["k"], *args, pos=d["pos"])
    back = BWD[dtype](d["gq"], d["gk"], d["q"], d["k"], *args, pos=d["pos"])
    # one fused projection output, normed in place
    qkv = torch.cat((d["q"], d["k"], d["k"] * 2), 2)
    q, k, v = qkv.split((Hq, Hk, Hk), 2)
    a, b = FWD[dtype](q, k, *args, pos=d["pos"])
    assert torch.equal(a, yq) and torch.equal(b, yk)
    FWD[dtype](q, k, *args, pos=d["pos"], q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(v, d["k"] * 2)
    # gradients into one fused buffer
    d_qkv = torch.full((B, S, Hq + 2 * Hk, Dh), 7.0, dtype=dtype, device="cuda")
    dq, dk, dv = d_qkv.split((Hq, Hk, Hk), 2)
    out = BWD[dtype](d["gq"], d["gk"], d["q"], d["k"], *args, pos=d["pos"], d_q=dq, d_k=dk)
    assert all(torch.equal(x, y) for x, y in zip(out, back)) and (dv == 7).all()
    # heads before tokens, and outputs as rows 3 .. of a longer joint buffer
    joint = torch.full((B, Hq, S + 8, Dh), 7.0, dtype=dtype, device="cuda")
    to = joint.transpose(1, 2)[:, 3:3 + S]
    qt = d["q"].transpose(1, 2).contiguous().transpose(1, 2)
    kt = d["k"].transpose(1, 2).contiguous().transpose(1, 2)
    a, b = FWD[dtype](qt, kt, *args, pos=d["pos"], q_out=to)
    assert torch.equal(a, yq) and torch.equal(b, yk)
    assert (joint[:, :, :3] == 7).all() and (joint[:, :, 3 + S:] == 7).all()
    # gradients in place of the output gradients, in that layout
    gq = d["gq"].transpose(1, 2).contiguous().transpose(1, 2)
    gk = d["gk"].clone()
    out = BWD[dtype](gq, gk, qt, kt, *args, pos=d["pos"], d_q=gq, d_k=gk)
    assert all(torch.equal(x, y) for x, y in zip(out, back)) and torch.equal(gq, back[0])
    # one head broadcast to all; rows that are not 16-byte aligned are copied
    one = d["q"][:, :, :1].expand(B, S, Hq, Dh)
    a, _ = FWD[dtype](one, None, *args, pos=d["pos"])
    b, _ = FWD[dtype](one.contiguous(), None, *args, pos=d["pos"])
    assert torch.equal(a, b)
    odd = torch.zeros(d["q"].numel() + 1, dtype=dtype, device="cuda")[1:].view(d["q"].shape)
    odd.copy_(d["q"])
    a, _ = FWD[dtype](odd, None, *args, pos=d["pos"])
    assert torch.equal(a, yq)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batch_and_chunk_invariance(dtype):
    """Rows and dw do not depend on the batch or on how samples are split."""
    for B, S in ((7, 40), (3, 300)):
        d = make(dtype, B, S, 6, 2, 128, 128)
        args = (d["wq"], d["wk"], d["cos"], d["sin"])
        yq, yk = FWD[dtype](d["q"], d["k"], *args, pos=d["pos"])
        full = BWD[dtype](d["gq"], d["gk"], d["q"], d["k"], *args, pos=d["pos"])
        for cuts in ([1] * B, [2] * (B // 2) + [B - 2 * (B // 2)]):
            acc = [torch.zeros(128, device="cuda") for _ in range(2)]
            b = 0
            for n in cuts:
                s = slice(b, b + n)
                b += n
                a, c = FWD[dtype](d["q"][s], d["k"][s], *args, pos=d["pos"][s])
                assert torch.equal(a, yq[s]) and torch.equal(c, yk[s])
                dq, dk, *acc = BWD[dtype](d["gq"][s], d["gk"][s], d["q"][s], d["k"][s], *args, pos=d["pos"][s],
                                          dwq_acc=acc[0], dwk_acc=acc[1], accumulate=True)
                assert torch.equal(dq, full[0][s]) and torch.equal(dk, full[1][s])
            assert torch.equal(acc[0], full[2]) and torch.equal(acc[1], full[3])


def test_far_offsets():
    """Rows beyond 2^32 elements of their buffer, and positions beyond 2^24."""
    d = make(BF16, 2, 3, 2, 2, 64, 64, P=8, pads=False)
    far = (1 << 32) + 1024
    buf = torch.empty(far + 2 * 3 * 4 * 64, dtype=BF16, device="cuda")
    qkv = torch.as_strided(buf, (2, 3, 4, 64), (far, 256, 64, 1))
    qkv.copy_(torch.cat((d["q"], d["k"]), 2))
    args = (d["wq"], d["wk"], d["cos"], d["sin"])
    want = FWD[BF16](d["q"], d["k"], *args, pos=d["pos"])
    back = BWD[BF16](d["gq"], d["gk"], d["q"], d["k"], *args, pos=d["pos"])
    q, k = qkv[:, :, :2], qkv[:, :, 2:]
    got = BWD[BF16](d["gq"], d["gk"], q, k, *args, pos=d["pos"])
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    FWD[BF16](q, k, *args, pos=d["pos"], q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    del buf, qkv, q, k
    P = (1 << 24) + 5
    cos = torch.zeros((P, 32), device="cuda")
    sin = torch.zeros((P, 32), device="cuda")
    cos[-8:], sin[-8:] = d["cos"], d["sin"]
    got = FWD[BF16](d["q"], d["k"], d["wq"], d["wk"], cos, sin, pos=d["pos"] + (P - 8))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("shape", [(65535, 1, 1, 1, 8, 8), (1, 262144, 1, 2, 8, 0), (1, 2, 1024, 1, 256, 64),
                                   (2, 1, 1, 1024, 16, 16), (300, 2, 2, 2, 128, 128)])
def test_largest(shape):
    """The most samples, tokens and heads."""
    check_both(make(BF16, *shape, P=40, pads=False), BF16, True)


def test_graph_and_stream():
    """Captured and replayed on new data; called on another stream with copies made there."""
    d = make(BF16, 2, 30, 4, 4, 64, 64)
    args = (d["wq"], d["wk"], d["cos"], d["sin"])
    run = lambda: (*FWD[BF16](d["q"], d["k"], *args, pos=d["pos"]),  # noqa: E731
                   *BWD[BF16](d["gq"], d["gk"], d["q"], d["k"], *args, pos=d["pos"]))
    want = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in got:
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d["q"].mul_(-2)
    want = run()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    odd = d["gq"].transpose(2, 3).contiguous().transpose(2, 3)  # channels not dense: copied on the side stream
    dq, *_ = BWD[BF16](odd, d["gk"], d["q"], d["k"], *args, pos=d["pos"], stream=side)
    dq2, *_ = BWD[BF16](odd, d["gk"], d["q"], d["k"], *args, pos=d["pos"], stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(dq, want[2]) and torch.equal(dq2, want[2])


def test_refusals():
    d = make(BF16, 1, 4, 2, 2, 64, 64, pads=False)
    q, k, w, cos, sin = d["q"], d["k"], d["wq"], d["cos"], d["sin"]
    fwd = FWD[BF16]
    for bad in (lambda: fwd(q.float(), k, w, w, cos, sin), lambda: fwd(q, k, w.float(), w, cos, sin),
                lambda: fwd(q, k, w, w, cos.double(), sin), lambda: fwd(q.cpu(), k, w, w, cos, sin),
                lambda: fwd(q, k, w, w, cos, sin, pos=torch.zeros((1, 4), device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fwd(q, k[:, :3], w, w, cos, sin), lambda: fwd(q, k, w[:8], w, cos, sin),
                lambda: fwd(q, k, w, w, cos, None), lambda: fwd(q, k, w, w, cos, sin[:2]),
                lambda: fwd(q, k, w, w, cos, sin, pos=d["pos"][:, :2]),
                lambda: fwd(q, k, w, w, cos, sin, q_out=q[:, :2]),
                lambda: fwd(q, k, w, w, cos, sin, q_out=torch.empty((1, 4, 64, 2), dtype=BF16,
                                                                    device="cuda").transpose(2, 3)),
                lambda: BWD[BF16](q, k, q, k, w, w, cos, sin, accumulate=True),
                lambda: BWD[BF16](q, k, q, k, w, w, cos, sin,
                                  workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fwd(q, k, w, w, cos[:2], sin[:2]), lambda: fwd(q, k, w, w, cos, sin, q_out=k),
                lambda: fwd(q, k, w, w, cos, sin, eps=-1.0), lambda: BWD[BF16](q, k, q, k, w, w, cos, sin, d_q=k)):
        with pytest.raises(binding.AdaLNError):
            bad()
