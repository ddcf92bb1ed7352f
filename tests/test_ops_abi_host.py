"""The checks of include/adaln_ops.h on the host: every refusal comes before
the device check and before any launch.  Pointers are fake addresses that are
never dereferenced; calls that pass every check run only without a GPU, where
they stop at the device check."""

from __future__ import annotations

import ctypes
import os

import pytest
import torch

from invariant_dit_adaln_gb300 import binding, build

OK, NULL, SHAPE, ALIGN, ALIAS, WORKSPACE, DEVICE, CUDA, ARG = range(9)
TB = 1 << 40


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
    names = binding.declared_symbols(os.path.join(build.INCLUDE, "adaln_ops.h"))
    assert len(names) == 13
    for n in names:
        assert hasattr(L, n) and hasattr(binding, n) or n.endswith("workspace_bytes"), n


# --- head rows --------------------------------------------------------------

class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


def rows(i, B=2, S=5, H=4, Dh=64, off=0, strides=None):
    st = strides or (S * H * Dh, H * Dh, Dh)
    return Heads(i if i is None else at(i, off), *st)


BASE = dict(B=2, S=5, Hq=4, Hk=2, Dh=64, Dr=64, P=8, inter=1, eps=1e-6, is64=0)


def heads_fwd(L, f32=False, q=None, k=None, qo=None, ko=None, wq=at(4), wk=at(5), cos=at(6), sin=at(7), pos=at(8), **kw):
    a = {**BASE, **kw}
    q = q or rows(0, H=a["Hq"], Dh=a["Dh"])
    k = k or rows(1, H=a["Hk"], Dh=a["Dh"])
    qo = qo or rows(2, H=a["Hq"], Dh=a["Dh"])
    ko = ko or rows(3, H=a["Hk"], Dh=a["Dh"])
    fn = L.adaln_f32_qk_norm_rope_fwd if f32 else L.adaln_qk_norm_rope_fwd
    ref = ctypes.byref
    return fn(ref(q), ref(k), wq, wk, cos, sin, pos, a["is64"], ref(qo), ref(ko), a["B"], a["S"], a["Hq"], a["Hk"],
              a["Dh"], a["Dr"], a["P"], a["inter"], a["eps"], None)


def test_heads_fwd_accepts(L):
    assert heads_fwd(L) == DEVICE
    assert heads_fwd(L, f32=True) == DEVICE
    assert heads_fwd(L, pos=None, P=5) == DEVICE
    assert heads_fwd(L, wq=None, wk=None) == DEVICE
    assert heads_fwd(L, Dr=0, cos=None, sin=None, P=0) == DEVICE
    assert heads_fwd(L, Hk=0, wk=None) == DEVICE
    assert heads_fwd(L, S=0) == DEVICE and heads_fwd(L, B=0) == DEVICE
    # in place
    assert heads_fwd(L, qo=rows(0)) == DEVICE
    # q and k as slices of one fused buffer [B, S, 8, 64], and both in place there
    st = (5 * 512, 512, 64)
    q, k = rows(0, strides=st), rows(0, off=4 * 128, strides=st)
    assert heads_fwd(L, q=q, k=k) == DEVICE
    assert heads_fwd(L, q=q, k=k, qo=q, ko=k) == DEVICE
    # [B, H, S, Dh] storage; broadcast inputs
    assert heads_fwd(L, q=rows(0, strides=(4 * 5 * 64, 64, 5 * 64)), qo=rows(2, strides=(4 * 5 * 64, 64, 5 * 64))) == DEVICE
    assert heads_fwd(L, q=rows(0, strides=(0, 0, 0))) == DEVICE
    # outputs that interleave in one buffer; a stride of a dimension of size 1 is not used
    assert heads_fwd(L, qo=rows(2, strides=st), ko=rows(2, off=512, strides=st)) == DEVICE
    assert heads_fwd(L, B=1, q=rows(0, strides=(3, 256, 64))) == DEVICE


def test_heads_fwd_refuses(L):
    for bad in ({"Dh": 4}, {"Dh": 12}, {"Dh": 264}, {"Dr": 4}, {"Dr": 72}, {"Dr": -8}, {"Hq": 0}, {"Hq": 1025},
                {"Hk": -1}, {"Hk": 1025}, {"B": -1}, {"B": 65536}, {"S": -1}, {"S": 262145}, {"P": -1},
                {"pos": None, "P": 4}, {"B": 65535, "S": 262144, "Hq": 1024}):
        assert heads_fwd(L, **bad) == SHAPE, bad
    assert heads_fwd(L, q=rows(0, strides=(-1280, 256, 64))) == SHAPE
    assert heads_fwd(L, q=rows(0, strides=(1 << 50, 256, 64))) == SHAPE
    for bad in ({"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"is64": 2}, {"inter": 2}, {"Hk": 0}):
        assert heads_fwd(L, **bad) == ARG, bad
    assert heads_fwd(L, q=rows(None)) == NULL
    assert heads_fwd(L, ko=rows(None)) == NULL
    assert heads_fwd(L, cos=None) == NULL
    assert heads_fwd(L, q=rows(0, off=8)) == ALIGN
    assert heads_fwd(L, q=rows(0, strides=(1280, 260, 64))) == ALIGN
    assert heads_fwd(L, f32=True, q=rows(0, strides=(1280, 258, 64))) == ALIGN
    assert heads_fwd(L, wq=at(4, 8)) == ALIGN
    assert heads_fwd(L, pos=at(8, 4)) == ALIGN
    # overlaps: output in another input, shifted in place, in the other output, in a weight, in itself
    assert heads_fwd(L, qo=rows(1)) == ALIAS
    assert heads_fwd(L, qo=rows(0, off=128)) == ALIAS
    assert heads_fwd(L, ko=rows(2, H=2, off=128)) == ALIAS
    assert heads_fwd(L, wq=at(2, 64)) == ALIAS
    assert heads_fwd(L, cos=at(3, 16)) == ALIAS
    assert heads_fwd(L, qo=rows(2, strides=(0, 256, 64))) == ALIAS
    assert heads_fwd(L, qo=rows(2, strides=(1280, 128, 64))) == ALIAS
    st = (5 * 512, 512, 64)
    assert heads_fwd(L, qo=rows(2, strides=st), ko=rows(2, off=256, strides=st)) == ALIAS
    assert heads_fwd(L, q=rows(0, strides=st), k=rows(0, off=512, strides=st), qo=rows(0, strides=st),
                     ko=rows(0, off=384, strides=st)) == ALIAS


def test_lattices_against_brute_force(L):
    """The overlap check of strided rows against the byte sets themselves."""
    import random
    r = random.Random(0)
    seen = set()
    for _ in range(400):
        B, S, Hq, Hk, Dh = r.randint(1, 3), r.randint(1, 4), r.randint(1, 3), r.randint(1, 3), 8
        tok = 8 * r.randint(Hq + Hk - 1, Hq + Hk + 2)
        bat = tok * S + 8 * r.choice([0, 0, 1, 3])
        st = (bat, tok, 8) if r.random() < 0.7 else (bat, 8, 8 * S)
        off = 8 * r.randint(0, 2 * (Hq + Hk))

        def cells(H, o):
            return [o + b * st[0] + s * st[1] + h * st[2] for b in range(B) for s in range(S) for h in range(H)]

        q, k = cells(Hq, 0), cells(Hk, off)
        own = len(set(q)) < len(q) or len(set(k)) < len(k)
        clash = bool(set(q) & set(k))
        got = heads_fwd(L, B=B, S=S, Hq=Hq, Hk=Hk, Dh=8, Dr=8, q=rows(0, B, S, Hq, 8), k=rows(1, B, S, Hk, 8),
                        qo=rows(2, strides=st), ko=rows(2, off=2 * off, strides=st))
        if own or clash:
            assert got == ALIAS, (B, S, Hq, Hk, st, off)
        elif st[2] == 8:  # slices of one token-major buffer are told apart exactly
            assert got == DEVICE, (B, S, Hq, Hk, st, off)
        seen.add((got, st[2] == 8))
    assert len(seen) >= 3


def heads_bwd(L, f32=False, ws=at(20), nws=None, acc=0, dwq=at(18), dwk=at(19), wq=at(10), wk=at(11), over=None, **kw):
    a = {**BASE, **kw}
    h = {n: rows(i, H=a["Hq"] if n.endswith("q") else a["Hk"], Dh=a["Dh"])
         for i, n in enumerate(("gq", "gk", "q", "k", "dq", "dk"))}
    h.update(over or {})
    if nws is None:
        nws = L.adaln_qk_norm_rope_bwd_workspace_bytes(a["B"], a["S"], a["Hq"], a["Hk"], a["Dh"])
    fn = L.adaln_f32_qk_norm_rope_bwd if f32 else L.adaln_qk_norm_rope_bwd
    ref = ctypes.byref
    return fn(ref(h["gq"]), ref(h["gk"]), ref(h["q"]), ref(h["k"]), wq, wk, at(12), at(13), at(14), a["is64"],
              ref(h["dq"]), ref(h["dk"]), dwq, dwk, acc, ws, nws, a["B"], a["S"], a["Hq"], a["Hk"], a["Dh"], a["Dr"],
              a["P"], a["inter"], a["eps"], None)


def test_heads_bwd_checks(L):
    assert heads_bwd(L) == DEVICE
    assert heads_bwd(L, f32=True, acc=1) == DEVICE
    assert heads_bwd(L, dwq=None, dwk=None, ws=None, nws=0) == DEVICE
    assert heads_bwd(L, over={"dq": rows(0), "dk": rows(1, H=2)}) == DEVICE      # in place of the output gradients
    assert heads_bwd(L, Hk=0, dwk=None, wk=None) == DEVICE
    assert heads_bwd(L, Hk=0, wk=None) == ARG
    assert heads_bwd(L, acc=2) == ARG
    assert heads_bwd(L, over={"gq": rows(None)}) == NULL
    assert heads_bwd(L, ws=at(20, 8)) == ALIGN
    assert heads_bwd(L, dwq=at(18, 4)) == ALIGN
    assert heads_bwd(L, over={"dq": rows(2)}) == ALIAS                           # d_q over q
    assert heads_bwd(L, over={"dk": rows(4, H=2)}) == ALIAS                      # d_k over d_q
    assert heads_bwd(L, dwk=at(18, 16)) == ALIAS
    assert heads_bwd(L, dwq=at(2, 64)) == ALIAS                                  # dw inside q
    assert heads_bwd(L, ws=at(4, 256)) == ALIAS                                  # workspace inside d_q
    assert heads_bwd(L, nws=16) == WORKSPACE
    assert heads_bwd(L, ws=None) == WORKSPACE
    assert L.adaln_qk_norm_rope_bwd_workspace_bytes(0, 5, 4, 2, 64) == 0
    assert L.adaln_qk_norm_rope_bwd_workspace_bytes(2, 5, 4, 2, 264) == 0


# --- embedding ----------------------------------------------------------------

def embed_fwd(L, f32=False, tok=at(0), table=at(1), out=at(2), is64=1, scale=1.0, n=10, V=20, D=64):
    return (L.adaln_f32_embed_fwd if f32 else L.adaln_embed_fwd)(tok, is64, table, scale, out, n, V, D, None)


def test_embed_fwd_checks(L):
    assert embed_fwd(L) == DEVICE and embed_fwd(L, f32=True) == DEVICE
    assert embed_fwd(L, n=0, tok=None, out=None, table=None) == DEVICE
    assert embed_fwd(L, V=0, table=None) == DEVICE
    for bad in ({"D": 4}, {"D": 12}, {"D": 8200}, {"n": -1}, {"n": (1 << 24) + 1}, {"V": -1}, {"V": (1 << 24) + 1}):
        assert embed_fwd(L, **bad) == SHAPE, bad
    assert embed_fwd(L, is64=2) == ARG and embed_fwd(L, scale=float("inf")) == ARG
    assert embed_fwd(L, tok=None) == NULL and embed_fwd(L, table=None) == NULL and embed_fwd(L, out=None) == NULL
    assert embed_fwd(L, tok=at(0, 8)) == ALIGN and embed_fwd(L, out=at(2, 4)) == ALIGN
    assert embed_fwd(L, out=at(1, 1024)) == ALIAS and embed_fwd(L, out=at(0, 16)) == ALIAS


def embed_bwd(L, f32=False, g=at(0), tok=at(1), acc=at(2), tab=None, accumulate=0, ws=at(4), nws=None, n=10, V=20, D=64):
    need = L.adaln_embed_bwd_workspace_bytes(n, V, D) if nws is None else nws
    if f32:
        return L.adaln_f32_embed_bwd(g, tok, 1, 1.0, acc, accumulate, ws, need, n, V, D, None)
    return L.adaln_embed_bwd(g, tok, 1, 1.0, acc, tab, accumulate, ws, need, n, V, D, None)


def test_embed_bwd_checks(L):
    assert embed_bwd(L) == DEVICE and embed_bwd(L, f32=True, accumulate=1) == DEVICE
    assert embed_bwd(L, acc=None, tab=at(3)) == DEVICE
    assert embed_bwd(L, n=0, g=None, tok=None, ws=None) == DEVICE
    assert embed_bwd(L, tab=at(3)) == ARG and embed_bwd(L, acc=None) == ARG
    assert embed_bwd(L, acc=None, tab=at(3), accumulate=1) == ARG and embed_bwd(L, accumulate=3) == ARG
    assert embed_bwd(L, f32=True, acc=None) == ARG
    assert embed_bwd(L, D=20) == SHAPE and embed_bwd(L, n=-1) == SHAPE
    assert embed_bwd(L, g=None) == NULL
    assert embed_bwd(L, ws=at(4, 4)) == ALIGN
    assert embed_bwd(L, acc=at(0, 64)) == ALIAS and embed_bwd(L, ws=at(2, 256)) == ALIAS
    assert embed_bwd(L, nws=16) == WORKSPACE and embed_bwd(L, ws=None) == WORKSPACE
    assert L.adaln_embed_bwd_workspace_bytes(0, 20, 64) == 0
    assert L.adaln_embed_bwd_workspace_bytes(-1, 20, 64) == 0


# --- gradient norm ------------------------------------------------------------

class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def tensors(*specs):
    arr = (Tensor * len(specs))()
    for a, (p, n, d) in zip(arr, specs):
        a.data, a.numel, a.dtype = p, n, d
    return arr


def norm(L, arr, count=None, out=at(50), ws=at(51), nws=None):
    count = len(arr) if count is None else count
    need = L.adaln_grad_norm_workspace_bytes(arr, count) if nws is None else nws
    return L.adaln_grad_norm(arr, count, out, ws, need, None)


def clip(L, arr, outs, max_norm=1.0, stats=at(50), ws=at(51)):
    return L.adaln_grad_clip(arr, outs, len(arr), max_norm, stats, ws, L.adaln_grad_norm_workspace_bytes(arr, len(arr)),
                             None)


def test_grad_norm_checks(L):
    good = tensors((at(0), 100, 0), (at(1, 2), 7, 1), (None, 0, 0))
    assert norm(L, good) == DEVICE
    assert norm(L, tensors((at(0), 5, 0), (at(0), 5, 0))) == DEVICE  # the same tensor twice
    assert L.adaln_grad_norm_workspace_bytes(good, 3) == 256
    assert L.adaln_grad_norm_workspace_bytes(tensors((at(0), 4096 * 40 + 1, 0)), 1) == 512
    assert L.adaln_grad_norm_workspace_bytes(tensors((at(0), 8192 * 32, 1)), 1) == 256
    assert norm(L, good, count=-1, nws=0) == SHAPE and norm(L, good, count=65537, nws=0) == SHAPE
    assert norm(L, tensors((at(0), -1, 0))) == SHAPE and norm(L, tensors((at(0), 1 << 40, 0))) == SHAPE
    assert norm(L, tensors((at(0), 5, 2))) == ARG
    assert norm(L, tensors((None, 5, 0))) == NULL and norm(L, good, out=None) == NULL
    assert norm(L, tensors((at(0, 2), 5, 0))) == ALIGN and norm(L, tensors((at(0, 1), 5, 1))) == ALIGN
    assert norm(L, good, ws=at(51, 8)) == ALIGN and norm(L, good, out=at(50, 4)) == ALIGN
    assert norm(L, good, out=at(0, 16)) == ALIAS and norm(L, good, ws=at(1)) == ALIAS
    assert norm(L, good, ws=None) == WORKSPACE and norm(L, good, nws=8) == WORKSPACE


def test_grad_clip_checks(L):
    g = tensors((at(0), 100, 0), (at(1, 2), 7, 1))
    o = tensors((at(2, 4), 100, 0), (at(3, 6), 7, 1))
    assert clip(L, g, o) == DEVICE and clip(L, g, g) == DEVICE
    assert clip(L, g, o, max_norm=float("inf")) == DEVICE
    assert clip(L, g, o, max_norm=-1.0) == ARG and clip(L, g, o, max_norm=float("nan")) == ARG
    assert clip(L, g, None) == NULL
    assert clip(L, g, tensors((at(2), 99, 0), (at(3), 7, 1))) == SHAPE
    assert clip(L, g, tensors((at(2), 100, 1), (at(3), 7, 1))) == ARG
    assert clip(L, g, tensors((at(2, 2), 100, 0), (at(3), 7, 1))) == ALIGN
    assert clip(L, g, tensors((at(0, 4), 100, 0), (at(3), 7, 1))) == ALIAS     # shifted over its own input
    assert clip(L, g, tensors((at(1), 100, 0), (at(3), 7, 1))) == ALIAS        # over another input
    assert clip(L, g, tensors((at(2), 100, 0), (at(2, 398), 7, 1))) == ALIAS   # over another output
    assert clip(L, g, tensors((at(2), 100, 0), (at(2, 400), 7, 1))) == DEVICE  # directly behind it
    twice = tensors((at(0), 100, 0), (at(0), 100, 0))
    assert clip(L, twice, twice) == ALIAS                                      # would be scaled twice
    assert clip(L, g, o, stats=at(2, 16)) == ALIAS
    many = tensors(*[(at(0, 400 * i), 100, 0) for i in range(500)])
    assert clip(L, many, many) == DEVICE
    many[499].data = at(0, 396)
    assert clip(L, many, many) == ALIAS


def test_binding_refuses_host_tensors(L):
    x = torch.zeros((1, 2, 2, 16), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.adaln_qk_norm_rope_fwd(x, x, None, None, None, None)
    with pytest.raises(ValueError):
        binding.adaln_qk_norm_rope_fwd(x[0], x, None, None, None, None)
    with pytest.raises(TypeError):
        binding.adaln_embed_fwd(torch.zeros(3, dtype=torch.int64), torch.zeros((4, 8), dtype=torch.bfloat16))
