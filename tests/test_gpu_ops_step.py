"""The operators together, as a training step uses them: labels -> temb ->
modulated norm -> q/k norm and rotation, backward to the table's gradient, and the
gradients of all of it clipped by their global norm."""

from __future__ import annotations

import pytest
import torch

import ops_ref
from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b

pytestmark = pytest.mark.gpu


def step(p, labels, x, pos, cos, sin, g_attn, H, max_norm):
    """One forward and backward through a block's conditioning and attention norms; the clipped gradients."""
    B, S, D = x.shape
    V = p["table"].shape[0]
    temb = b.adaln_embed_fwd(labels, p["table"])
    emb, u = b.adaln_proj_fwd(temb, p["W"], p["b"])
    h, mean, rstd = b.adaln_out_fwd(x, emb)
    q = k = h.view(B, S, H, D // H)  # the projections to q and k are the identity here
    yq, yk = b.adaln_qk_norm_rope_fwd(q, k, p["wq"], p["wk"], cos, sin, pos=pos)
    dq, dk, dwq, dwk = b.adaln_qk_norm_rope_bwd(g_attn[0], g_attn[1], q, k, p["wq"], p["wk"], cos, sin, pos=pos)
    dh = (dq + dk).view(B, S, D)
    dx, d_emb = b.adaln_out_bwd(dh, x, emb, mean, rstd)
    dW, db = torch.empty((2 * D, D), device="cuda"), torch.empty(2 * D, device="cuda")
    d_temb, _, _, _, _ = b.adaln_proj_bwd(d_emb, temb, u, p["W"], dW_acc=dW, db_acc=db)
    d_table = b.adaln_embed_bwd(d_temb, labels, V)
    grads = [dW, db, dwq, dwk, d_table]
    kept = [g.clone() for g in grads]
    _, stats = b.adaln_grad_clip(grads, max_norm, outs=grads)
    return {"q": q, "yq": yq, "yk": yk, "dx": dx, "temb": temb, "d_temb": d_temb, "grads": kept, "clipped": grads,
            "stats": stats}


def test_training_step():
    lib()
    B, S, D, H, V = 3, 37, 512, 8, 11
    g = torch.Generator().manual_seed(0)

    def rand(*shape, scale=1.0):
        return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16).cuda()

    p = {"table": rand(V, D), "W": rand(2 * D, D, scale=0.02), "b": rand(2 * D, scale=0.02),
         "wq": 1 + rand(D // H, scale=0.1), "wk": 1 + rand(D // H, scale=0.1)}
    labels = torch.tensor([4, -1, 4], device="cuda")
    angle = torch.rand((S, D // H // 2), generator=g, dtype=torch.float64) * 6
    cos, sin = angle.cos().float().cuda(), angle.sin().float().cuda()
    pos = torch.arange(S).expand(B, S).clone()
    pos[1, 20:] = -1
    x, g_attn = rand(B, S, D), [rand(B, S, H, D // H) for _ in range(2)]
    args = (p, labels, x, pos.cuda(), cos, sin, g_attn, H)
    r = step(*args, 1.0)
    # each stage against its 64-bit form on the inputs it got
    for n, w, gy in (("yq", "wq", g_attn[0]), ("yk", "wk", g_attn[1])):
        want, err = ops_ref.heads_fwd(r["q"], p[w], cos, sin, pos, 1e-6, True)
        ops_ref.check(r[n], want, err, n)
        _, _, dw, err = ops_ref.heads_bwd(gy, r["q"], p[w], cos, sin, pos, 1e-6, True)
        ops_ref.check(r["grads"][2 if n == "yq" else 3], dw, err, w)
    want, size, _ = ops_ref.embed_bwd(r["d_temb"], labels, V, 1.0)
    ops_ref.check(r["grads"][4], want, 4 * ops_ref.U * size, "d_table")
    assert not r["temb"][1].any() and (r["grads"][4][4] != 0).any()
    norm = sum(float(t.double().square().sum()) for t in r["grads"]) ** 0.5
    assert abs(float(r["stats"][0]) - norm) <= 17 * ops_ref.U * norm
    for t, c in zip(r["grads"], r["clipped"]):
        want = t.double().cpu() * min(1.0, 1.0 / (norm + 1e-6))
        ops_ref.check(c, want, 20 * ops_ref.U * want.abs() + 1e-40, "clipped")
    # the same bits from a captured step
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*args, 1.0)
    graph.replay()
    assert torch.equal(got["stats"], r["stats"])
    assert all(torch.equal(a, c) for a, c in zip(got["clipped"], r["clipped"]))


def test_calls_at_once():
    """Calls on two streams, each with its own workspace and outputs, give the bits of the calls one by one."""
    lib()
    g = torch.Generator().manual_seed(3)
    sets = []
    for seed in range(2):
        n, V, D = (3000, 200, 512) if seed else (9000, 5000, 256)
        t = torch.randint(-1, V, (n,), generator=g).cuda()
        d = torch.randn((n, D), generator=g).to(torch.bfloat16).cuda()
        q = torch.randn((2, 300, 8, 64), generator=g).to(torch.bfloat16).cuda()
        cos, sin = torch.rand((300, 32), generator=g).cuda(), torch.rand((300, 32), generator=g).cuda()
        sets.append((t, d, V, q, cos, sin))

    def run(t, d, V, q, cos, sin):
        table = b.adaln_embed_bwd(d, t, V)
        dq, _, dw, _ = b.adaln_qk_norm_rope_bwd(q, None, q, None, None, None, cos, sin)
        outs, stats = b.adaln_grad_clip([table, dw], 0.1)
        return [table, dq, dw, *outs, stats]

    want = [run(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for k in range(20):
        with torch.cuda.stream(streams[k % 2]):
            got.append(run(*sets[k % 2]))
    torch.cuda.synchronize()
    for k, r in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(r, want[k % 2]))
