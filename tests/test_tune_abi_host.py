"""The checks of include/adaln_tune.h on the host: every refusal comes before
the device check and before any launch.  Pointers are fake addresses that are
never dereferenced; calls that pass every check run only without a GPU, where
they stop at the device check."""

from __future__ import annotations

import ctypes
import os

import pytest
import torch

from invariant_dit_adaln_gb300 import binding, build
from tune_ref import record_of, value_of

OK, NULL, SHAPE, ALIGN, ALIAS, WORKSPACE, DEVICE, CUDA, ARG = range(9)
TB = 1 << 44


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.load()


@pytest.fixture(autouse=True)
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer checks run only on machines without a GPU")


def at(i, off=0):
    return (i + 1) * TB + off


def test_exports(L):
    names = binding.declared_symbols(os.path.join(build.INCLUDE, "adaln_tune.h"))
    assert len(names) == len(set(names)) == 19
    for n in names:
        assert hasattr(L, n) and hasattr(binding, n), n
    assert set(names) <= set(binding._SIGNATURES) and set(names) <= set(binding._BOUND)


# --- records ------------------------------------------------------------------

def test_row_bytes(L):
    for D, want in ((8, 32), (16, 32), (24, 48), (32, 48), (512, 528), (520, 560), (3072, 3168), (8192, 8448)):
        assert L.adaln_ckpt8_row_bytes(D) == want
    for D in (-8, 0, 4, 12, 8200, 2 ** 31 - 8):
        assert L.adaln_ckpt8_row_bytes(D) == 0


def test_record_reference():
    """The records' definition against itself: the least exponent, half a step."""
    x = torch.randn(50, 72, dtype=torch.float64) * torch.exp(5 * torch.randn(50, 72, dtype=torch.float64))
    rec = record_of(x)
    assert rec.shape == (50, 96)
    v = value_of(rec, 72)
    step = torch.repeat_interleave(torch.exp2(rec[:, 80:83].double() - 127), 32, 1)[:, :72]
    assert ((v - x).abs() <= step / 2).all()
    top = torch.nn.functional.pad(v.abs() / step, (0, 24)).view(50, 3, 32).amax(-1)
    assert (top >= 63.5).all() and (top <= 127).all()


@pytest.mark.parametrize("name", ["adaln_ckpt8_pack", "adaln_f32_ckpt8_pack", "adaln_ckpt8_unpack",
                                  "adaln_f32_ckpt8_unpack"])
def test_pack(L, name):
    f = getattr(L, name)
    assert f(at(0), at(1), 5, 64, None) == DEVICE
    assert f(None, None, 0, 64, None) == DEVICE
    for rows, D in ((5, 4), (5, 12), (5, 8200), (-1, 64), (1 << 40, 8), (1 << 34, 64)):
        assert f(at(0), at(1), rows, D, None) == SHAPE
    assert f(None, at(1), 5, 64, None) == NULL and f(at(0), None, 5, 64, None) == NULL
    assert f(at(0, 8), at(1), 5, 64, None) == ALIGN and f(at(0), at(1, 4), 5, 64, None) == ALIGN
    assert f(at(0), at(0), 5, 64, None) == ALIAS
    es = 4 if "f32" in name else 2
    first, second = (5 * 64 * es, 5 * 80) if "_pack" in name else (5 * 80, 5 * 64 * es)
    assert f(at(0), at(0, first), 5, 64, None) == DEVICE and f(at(0), at(0, first - 16), 5, 64, None) == ALIAS
    assert f(at(0, second), at(0), 5, 64, None) == DEVICE and f(at(0, second - 16), at(0), 5, 64, None) == ALIAS


@pytest.mark.parametrize("f32", [False, True])
def test_norm(L, f32):
    p = "adaln_f32_" if f32 else "adaln_"
    fwd, bwd, again = (getattr(L, p + n) for n in ("out_fwd_ckpt8", "out_bwd_ckpt8", "out_again_ckpt8"))
    need = L.adaln_out_bwd_ckpt8_workspace_bytes(2, 40, 64)
    assert need > 0

    def calls(B=2, S=40, D=64, eps=1e-6, nbytes=None, ptrs=None):
        q = ptrs or {}
        a = [q.get(i, at(i)) for i in range(8)]
        n = L.adaln_out_bwd_ckpt8_workspace_bytes(B, S, D) if nbytes is None else nbytes
        return (fwd(*a[:6], B, S, D, eps, None), bwd(*a, n, B, S, D, None), again(*a[:5], B, S, D, None))

    assert calls() == (DEVICE,) * 3
    assert calls(S=0) == calls(B=0) == (DEVICE,) * 3
    assert calls(B=0, S=0, ptrs={i: None for i in range(8)}) == (DEVICE,) * 3
    for bad in (dict(D=4), dict(D=20), dict(D=4104 if f32 else 8200), dict(B=-1), dict(B=65536), dict(S=-1),
                dict(S=262145), dict(B=65535, S=262144, D=128)):
        assert calls(**bad, nbytes=1 << 40) == (SHAPE,) * 3, bad
    for eps in (-1.0, float("nan"), float("inf")):
        assert calls(eps=eps)[0] == ARG
    for i in range(8):
        got = calls(ptrs={i: None})
        assert got[0] == (NULL if i < 6 else DEVICE) and got[1] == (NULL if i < 7 else WORKSPACE)
        assert got[2] == (NULL if i < 5 else DEVICE)
        got = calls(ptrs={i: at(i, 8)})
        assert got[0] == (ALIGN if i < 6 else DEVICE) and got[1] == ALIGN and got[2] == (ALIGN if i < 5 else DEVICE)
    assert calls(nbytes=need - 1)[1] == WORKSPACE
    # outputs: 2..5 of the forward, 5..7 of the backward, 4 of the last
    for o in range(2, 6):
        for i in range(6):
            if i != o:
                assert calls(ptrs={o: at(i)})[0] == ALIAS
    for o in (5, 6, 7):
        for i in range(8):
            if i != o:
                assert calls(ptrs={o: at(i)})[1] == ALIAS
    for i in range(4):
        assert calls(ptrs={4: at(i)})[2] == ALIAS


def test_norm_workspace_of_refused_sizes(L):
    f = L.adaln_out_bwd_ckpt8_workspace_bytes
    assert f(0, 5, 64) == f(2, 0, 64) == f(2, 5, 60) == f(2, 5, 8200) == f(-1, 5, 64) == f(2, 262145, 64) == 0


# --- adapters -----------------------------------------------------------------

class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64)]


BASE = dict(B=2, S=20, K=64, N=72, R=16, NA=3, is64=0, acc=0)


def rows(i, C, S=20, off=0, strides=None):
    return Rows(i if i is None else at(i, off), *(strides or (S * C, C)))


def fwd(L, f32=False, x=None, y=None, out=None, A=at(3), U=at(4), scale=at(5), ids=at(6), lens=at(7), state=at(8),
        nbytes=1 << 40, **kw):
    a = {**BASE, **kw}
    x, out = x or rows(0, a["K"], a["S"]), out or rows(2, a["N"], a["S"])
    y = rows(1, a["N"], a["S"]) if y is None else y
    f = L.adaln_f32_lora_fwd if f32 else L.adaln_lora_fwd
    ref = ctypes.byref
    return f(ref(x), A, U, scale, ids, a["is64"], lens, ref(y) if y else None, ref(out), state, nbytes, a["B"], a["S"],
             a["K"], a["N"], a["R"], a["NA"], None)


def bwd(L, f32=False, d_out=None, x=None, base=None, dx=None, A=at(4), U=at(5), scale=at(6), ids=at(7), lens=at(8),
        state=at(9), dA=at(10), dU=at(11), ws=at(12), nbytes=1 << 40, **kw):
    a = {**BASE, **kw}
    d_out, x = d_out or rows(0, a["N"], a["S"]), x or rows(1, a["K"], a["S"])
    base = rows(2, a["K"], a["S"]) if base is None else base
    dx = rows(3, a["K"], a["S"]) if dx is None else dx
    f = L.adaln_f32_lora_bwd if f32 else L.adaln_lora_bwd
    ref = ctypes.byref
    return f(ref(d_out), ref(x), state, A, U, scale, ids, a["is64"], lens, ref(base) if base else None,
             ref(dx) if dx else None, dA, dU, a["acc"], ws, nbytes, a["B"], a["S"], a["K"], a["N"], a["R"], a["NA"], None)


@pytest.mark.parametrize("f32", [False, True])
def test_lora_accepts(L, f32):
    assert fwd(L, f32) == bwd(L, f32) == DEVICE
    assert fwd(L, f32, lens=None) == bwd(L, f32, lens=None) == DEVICE
    assert fwd(L, f32, y=False) == bwd(L, f32, base=False) == DEVICE
    assert fwd(L, f32, y=Rows(None, 0, 0)) == DEVICE
    assert bwd(L, f32, dx=False) == bwd(L, f32, dA=None) == bwd(L, f32, dU=None, dx=False, dA=None) == DEVICE
    assert bwd(L, f32, acc=1) == fwd(L, f32, is64=1) == DEVICE
    # in place; a stride of a dimension of size 1 is not used
    assert fwd(L, f32, out=rows(1, 72)) == bwd(L, f32, dx=rows(2, 64)) == DEVICE
    assert fwd(L, f32, S=1, x=rows(0, 64, strides=(64, 3))) == fwd(L, f32, B=1, x=rows(0, 64, strides=(-5, 64))) == DEVICE
    # [S, B, C] storage, slices of a wider tensor, broadcast bases
    assert fwd(L, f32, x=rows(0, 64, strides=(64, 128)), out=rows(2, 72, strides=(72, 144))) == DEVICE
    assert fwd(L, f32, out=rows(2, 72, strides=(20 * 256, 256))) == DEVICE
    assert fwd(L, f32, y=rows(1, 72, strides=(0, 0))) == bwd(L, f32, base=rows(2, 64, strides=(64, 0))) == DEVICE
    # x and y interleaved in one buffer, out in place there
    w = 20 * 144, 144
    es = 4 if f32 else 2
    assert fwd(L, f32, x=rows(0, 64, strides=w), y=rows(0, 72, off=64 * es, strides=w),
               out=rows(0, 72, off=64 * es, strides=w)) == DEVICE
    # no adapters: none to point at; no rows: nothing to point at
    assert fwd(L, f32, NA=0, A=None, U=None, scale=None) == DEVICE
    assert bwd(L, f32, NA=0, A=None, U=None, scale=None, dA=None, dU=None) == DEVICE
    none = Rows(None, 0, 0)
    for empty in (dict(B=0), dict(S=0)):
        assert fwd(L, f32, x=none, y=none, out=none, A=None, U=None, scale=None, ids=None, lens=None, state=None,
                   nbytes=0, **empty) == DEVICE
        assert bwd(L, f32, d_out=none, x=none, base=none, dx=none, A=None, U=None, scale=None, ids=None, lens=None,
                   state=None, ws=None, nbytes=0, **empty) == DEVICE
    big = dict(B=65535, S=64, K=64, N=64, R=8, NA=65535)
    assert fwd(L, f32, **big) == bwd(L, f32, **big) == DEVICE


@pytest.mark.parametrize("f32", [False, True])
def test_lora_refuses(L, f32):
    es = 4 if f32 else 2
    for bad in (dict(R=0), dict(R=4), dict(R=12), dict(R=136), dict(K=4), dict(K=65544), dict(K=20), dict(N=0),
                dict(N=65544), dict(N=12), dict(B=-1), dict(B=65536), dict(S=-1), dict(S=262145), dict(NA=-1),
                dict(NA=65536), dict(B=65535, S=262144)):
        assert fwd(L, f32, **bad) == bwd(L, f32, **bad) == SHAPE, bad
    for st in ((-1280, 64), (20 * 64, -64), (0, 64), (1280, 0), (1 << 50, 64), (1280, (1 << 40) // es)):
        assert fwd(L, f32, x=rows(0, 64, strides=st)) == SHAPE, st
        assert bwd(L, f32, x=rows(1, 64, strides=st)) == SHAPE, st
    for st in ((20 * 72, 0), (0, 72)):
        assert fwd(L, f32, out=rows(2, 72, strides=st)) == bwd(L, f32, d_out=rows(0, 72, strides=st)) == SHAPE
    assert fwd(L, f32, is64=2) == bwd(L, f32, is64=-1) == bwd(L, f32, acc=2) == ARG
    none = Rows(None, 1, 1)
    assert fwd(L, f32, x=none) == fwd(L, f32, out=none) == bwd(L, f32, x=none) == bwd(L, f32, d_out=none) == NULL
    for k in ("A", "U", "scale", "ids"):
        assert fwd(L, f32, **{k: None}) == bwd(L, f32, **{k: None}) == NULL, k
    assert bwd(L, f32, state=None) == NULL
    assert fwd(L, f32, state=None) == WORKSPACE and bwd(L, f32, ws=None) == WORKSPACE
    assert fwd(L, f32, nbytes=L.adaln_lora_state_bytes(2, 20, 16) - 1) == WORKSPACE
    need = (L.adaln_f32_lora_bwd_workspace_bytes if f32 else L.adaln_lora_bwd_workspace_bytes)(2, 20, 64, 72, 16)
    assert bwd(L, f32, nbytes=need) == DEVICE and bwd(L, f32, nbytes=need - 1) == WORKSPACE
    for k in ("A", "U", "scale", "ids", "lens", "state"):
        i = {"A": 3, "U": 4, "scale": 5, "ids": 6, "lens": 7, "state": 8}[k]
        assert fwd(L, f32, **{k: at(i, 8)}) == bwd(L, f32, **{k: at(i + 1, 4)}) == ALIGN, k
    assert bwd(L, f32, dA=at(10, 8)) == bwd(L, f32, dU=at(11, 8)) == bwd(L, f32, ws=at(12, 8)) == ALIGN
    assert fwd(L, f32, x=rows(0, 64, off=8)) == fwd(L, f32, y=rows(1, 72, off=4)) == fwd(L, f32, out=rows(2, 72, off=8)) == ALIGN
    odd = (20 * 64 + 16 // es, 64 + 2)
    assert fwd(L, f32, x=rows(0, 64, strides=odd)) == bwd(L, f32, base=rows(2, 64, strides=odd)) == ALIGN


@pytest.mark.parametrize("f32", [False, True])
def test_lora_overlaps(L, f32):
    es = 4 if f32 else 2
    for i in (0, 3, 4, 5, 6, 7, 8):
        assert fwd(L, f32, out=rows(i, 72)) == ALIAS, i
    assert fwd(L, f32, out=rows(1, 72, off=72 * es)) == ALIAS  # a row further on
    for i in (0, 1, 4, 5, 6, 7, 8, 9, 10, 11, 12):
        assert bwd(L, f32, dx=rows(i, 64)) == ALIAS, i
    for k, i in (("dA", 10), ("dU", 11), ("ws", 12)):
        for j in range(13):
            if j != i:
                assert bwd(L, f32, **{k: at(j)}) == ALIAS, (k, j)
    for j in (0, 1, 2, 3, 4, 5, 6, 7):
        assert fwd(L, f32, state=at(j)) == ALIAS, j
    # outputs whose rows share elements
    assert fwd(L, f32, out=rows(2, 72, strides=(20 * 72, 64))) == ALIAS
    assert fwd(L, f32, out=rows(2, 72, strides=(19 * 72, 72))) == ALIAS
    # ends of the buffers
    last = (2 * 20 - 1) * 72 * es + 72 * es
    assert fwd(L, f32, lens=at(2, last)) == DEVICE and fwd(L, f32, lens=at(2, last - 16)) == ALIAS


def test_lora_sizes(L):
    s = L.adaln_lora_state_bytes
    assert s(2, 20, 16) == 2 * 24 * 16 * 6 and s(0, 5, 8) == s(5, 0, 8) == 0
    for bad in ((-1, 5, 8), (65536, 5, 8), (1, 262145, 8), (1, 5, 4), (1, 5, 136)):
        assert s(*bad) == 0
    for f in (L.adaln_lora_bwd_workspace_bytes, L.adaln_f32_lora_bwd_workspace_bytes):
        assert f(2, 20, 64, 72, 16) >= s(2, 20, 16)
        for bad in ((0, 5, 64, 64, 8), (2, 0, 64, 64, 8), (2, 5, 60, 64, 8), (2, 5, 64, 65544, 8), (2, 5, 64, 64, 0)):
            assert f(*bad) == 0
        # never much more than what is read: the state, and sums no larger than x and d_out
        for S in (1, 16, 17, 100, 256, 257, 4096):
            for R in (8, 64, 128):
                es = 2 if f == L.adaln_lora_bwd_workspace_bytes else 4
                assert f(3, S, 512, 1024, R) <= s(3, S, R) + 3 * S * 1536 * es + 512
