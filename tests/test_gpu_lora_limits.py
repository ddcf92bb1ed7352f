"""The adapters' calls at the most samples, adapters and tokens, at two calls at once and
at replayed graphs that run side by side."""

from __future__ import annotations

import threading

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b
from test_gpu_lora import NAME, TYPES, fn, inputs, run, same, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    torch.cuda.synchronize()
    assert b.device_error() == 0


BF, F32 = TYPES
MOST = [(BF, (65535, 16, 8, 16, 40, 3)), (BF, (65535, 2, 8, 16, 8, 3)), (F32, (65535, 5, 8, 16, 8, 3)),
        (BF, (300, 20, 8, 16, 40, 65535)), (BF, (300, 700, 8, 16, 8, 65535)), (F32, (300, 2, 8, 8, 8, 65535)),
        (BF, (2, 262144, 8, 16, 8, 2)), (F32, (2, 262144, 8, 16, 8, 2))]


@pytest.mark.parametrize("t,size", MOST, ids=lambda v: NAME[v] if v in NAME else "x".join(map(str, v)))
def test_most(t, size):
    B, S = size[:2]
    c = inputs(t, *size, lens=[(S, 1, 0, S - 1)[i % 4] for i in range(B)])
    verify(t, c, run(t, c))
    if size[-1] == 65535:  # the last adapter, and ids just past it
        c["ids"][:3] = torch.tensor([65534, 65535, 65534])
        verify(t, c, run(t, c))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 40, 600])
def test_two_threads(t, S):
    """Calls of two host threads on streams of their own and on one stream."""
    cases = [inputs(t, 5, S, 264, 328, 16, 3, seed=s) for s in range(2)]
    want = [run(t, c) for c in cases]
    torch.cuda.synchronize()
    for shared in (False, True):
        one = torch.cuda.Stream()
        got = [[], []]

        def work(i):
            with torch.cuda.stream(one if shared else torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(run(t, cases[i]))

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        torch.cuda.synchronize()
        for i in range(2):
            assert len(got[i]) == 20
            assert all(same(p, q) for g in got[i] for p, q in zip(g, want[i]))


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
def test_graphs_side_by_side(t):
    """Two captured steps with their own states and workspaces, replayed on two streams."""
    made = []
    for i, (S, K, N, R) in enumerate(((300, 264, 328, 16), (90, 9224, 264, 64))):
        c = inputs(t, 3, S, K, N, R, 2, seed=i)
        w = (c["A"], c["U"], c["scale"], c["ids"])
        want = run(t, c)
        buf = [torch.empty_like(v) for v in want]
        state = torch.empty(b.adaln_lora_state_bytes(3, S, R), dtype=torch.uint8, device="cuda")
        ws = torch.empty(fn("lora_bwd_workspace_bytes", t)(3, S, K, N, R), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn("lora_fwd", t)(c["x"], *w, y=c["y"], out=buf[0], state=state)
            fn("lora_bwd", t)(c["d_out"], c["x"], state, *w, dx_base=c["dx_base"], dx=buf[1], dA_acc=buf[2],
                              dU_acc=buf[3], workspace=ws)
        made.append((g, buf, want, torch.cuda.Stream(), (c, state, ws)))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, buf, want, s, _ in made:
            with torch.cuda.stream(s):
                for v in buf:
                    v.fill_(3)
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        for g, buf, want, s, _ in made:
            assert all(same(p, q) for p, q in zip(buf, want))


def test_long_rows_beside_others():
    """Clusters that hold 64, 256 and 512 columns of tensor memory and the conditioning's
    projection, on streams of their own."""
    t = torch.bfloat16
    cases = [inputs(t, 2, 300, *size, 2, seed=i) for i, size in enumerate(((65536, 264, 16), (20000, 136, 128),
                                                                          (9216, 3080, 32)))]
    want = [run(t, c) for c in cases]
    gen = torch.Generator("cuda").manual_seed(1)
    temb, W, bias = (torch.randn(s, generator=gen, device="cuda").to(t) for s in ((130, 1024), (2048, 1024), (2048,)))
    emb = b.adaln_proj_fwd(temb, W, bias)[0]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got, embs = [[], [], []], []
    for _ in range(10):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(t, c))
        with torch.cuda.stream(streams[3]):
            embs += [b.adaln_proj_fwd(temb, W, bias)[0] for _ in range(4)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(same(p, q) for r in g for p, q in zip(r, w))
    assert all(same(e, emb) for e in embs)
