"""adaln_embed_*: the lookup bit for bit, the gradient by its documented order
bit for bit and against 64 bits."""

from __future__ import annotations

import pytest
import torch

import ops_ref
from gpu_util import lib
from invariant_dit_adaln_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FWD = {BF16: binding.adaln_embed_fwd, F32: binding.adaln_f32_embed_fwd}
BWD = {BF16: binding.adaln_embed_bwd, F32: binding.adaln_f32_embed_bwd}


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def make(kind, n, V, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "even":
        t = torch.randint(0, V, (n,), generator=g)
    elif kind == "one":
        t = torch.full((n,), V - 1)
    elif kind == "skew":
        t = (torch.rand(n, generator=g) ** 6 * V).long().clamp(max=V - 1)
        t[torch.rand(n, generator=g) < 0.1] = -1
        t[torch.rand(n, generator=g) < 0.05] = V
    else:
        t = torch.full((n,), -1)
    return t.cuda(), torch.randn((n, D), generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,V,D", [(1, 1, 8), (3, 5, 24), (257, 1001, 1032), (40, 7, 8192), (5000, 300, 64)])
def test_lookup(n, V, D, dtype):
    t, _ = make("skew", n, V, 8, dtype)
    table = torch.randn((V, D), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    for scale in (1.0, 0.37, -32.0):
        want = (table.float() * torch.tensor(scale)).to(dtype)[t.clamp(0, V - 1)]
        want = torch.where(((t >= 0) & (t < V))[:, None], want, torch.zeros((), dtype=dtype, device="cuda"))
        assert torch.equal(FWD[dtype](t, table, scale=scale), want)
        assert torch.equal(FWD[dtype](t.to(torch.int32), table, scale=scale), want)


# around the sizes of the sorts (one CTA to 4096 and a cluster to 32768 if token
# and place fit 32 bits, kernels over tiles of 1024 otherwise), one to three
# digits, one occurrence to all, trees of one to three levels
BACK = [(1, 1, 8, "even"), (31, 4, 16, "even"), (32, 3, 8, "one"), (33, 3, 8, "one"), (500, 40, 264, "even"),
        (1000, 255, 8, "skew"), (1000, 256, 8, "skew"), (4096, 257, 40, "skew"), (4097, 65535, 24, "skew"),
        (9000, 65536, 16, "skew"), (20000, 200, 8, "even"), (6000, 300000, 8, "even"), (4096, 1001, 16, "one"),
        (8192, 2, 8, "one"), (16384, 500, 8, "skew"), (16385, 70000, 8, "skew"),
        (32768, 130000, 8, "skew"), (32769, 3, 8, "skew"), (32768, 131071, 8, "even"), (32768, 131072, 8, "even"),
        (40000, 1, 8, "one"), (2000, (1 << 21) - 1, 8, "even"), (2000, 1 << 21, 8, "even"),
        (131072, 32767, 8, "one"), (131072, 32768, 8, "one"), (131072, 1500, 8, "skew"), (131073, 500, 8, "skew"), (100000, 2000, 8, "even"),
        (300, 65535, 8, "none"), (5000, 10, 8, "none"), (700, 1 << 24, 8, "even")]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,V,D,kind", BACK)
def test_gradient(n, V, D, kind, dtype):
    t, g = make(kind, n, V, D, dtype)
    scale = 0.37
    got = BWD[dtype](g, t, V, scale=scale).cpu()
    if V <= 70000:
        want, size, count = ops_ref.embed_bwd(g, t, V, scale)
        # 32 a level, at most three levels here, the scale
        depth = 32.0 + 32 * (count > 32) + 32 * (count > 1024) + 1
        ops_ref.check(got, want, depth[:, None] * ops_ref.U * size, "gradient")
    used = t[(t >= 0) & (t < V)].unique().cpu()
    rows = ops_ref.embed_bwd_order(g, torch.where((t >= 0) & (t < V), torch.searchsorted(used.cuda(), t), -1),
                                   len(used), scale)
    assert torch.equal(got[used], rows)
    got[used] = 0
    assert not got.any()
    if dtype == BF16:
        low = torch.full((V, D), 7.0, dtype=BF16, device="cuda")
        assert BWD[BF16](g, t.to(torch.int32), V, scale=scale, d_table=low) is low
        assert torch.equal(low[used.cuda()].cpu(), rows.to(BF16))
        low[used.cuda()] = 0
        assert not low.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_accumulate(dtype):
    """Rows of tokens that occur are added to; the others are left as they were."""
    for n, V, kind in ((300, 50, "skew"), (6000, 9000, "skew"), (6000, 9, "even")):
        t, g = make(kind, n, V, 72, dtype)
        fresh = BWD[dtype](g, t, V, scale=0.5)
        acc = torch.randn((V, 72), device="cuda")
        acc[V - 1] = float("nan")
        t = torch.where(t == V - 1, -1, t)
        fresh[V - 1] = 0
        want = acc + fresh
        BWD[dtype](g, t, V, scale=0.5, d_table_acc=acc, accumulate=True)
        used = torch.zeros(V, dtype=torch.bool, device="cuda")
        used[t[(t >= 0) & (t < V)]] = True
        assert torch.equal(acc[used], want[used])
        assert acc[V - 1].isnan().all()


def test_order_depends_on_the_count_alone():
    """The same rows of a token give the same bits wherever they stand."""
    g = torch.randn((100, 64), device="cuda")
    want = BWD[F32](g, torch.zeros(100, dtype=torch.int64, device="cuda"), 1)
    for n, V in ((4000, 900), (20000, 50000)):
        t = torch.randint(1, V, (n,), device="cuda")
        at = torch.randperm(n, device="cuda")[:100].sort()[0]
        t[at] = 0
        d = torch.randn((n, 64), device="cuda")
        d[at] = g
        assert torch.equal(BWD[F32](d, t, V)[0], want[0])


def test_empty_and_far():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert FWD[BF16](none, torch.ones((3, 8), dtype=BF16, device="cuda")).shape == (0, 8)
    low = torch.ones((3, 8), dtype=BF16, device="cuda")
    BWD[BF16](torch.empty((0, 8), dtype=BF16, device="cuda"), none, 3, d_table=low)
    assert not low.any()
    assert not BWD[F32](torch.empty((0, 8), device="cuda"), none, 3).any()
    keep = torch.ones((3, 8), device="cuda")
    BWD[F32](torch.empty((0, 8), device="cuda"), none, 3, d_table_acc=keep, accumulate=True)
    assert (keep == 1).all()
    t = torch.tensor([0, 5], device="cuda")
    assert not FWD[F32](t, torch.empty((0, 8), device="cuda")).any()
    # a table beyond 2^32 elements, tokens of two dimensions
    V, D = (1 << 20) + 3, 4096
    table = torch.zeros((V, D), dtype=BF16, device="cuda")
    table[V - 1], table[1] = 3.0, 2.0
    t = torch.tensor([[V - 1, 1], [0, V]], device="cuda")
    out = FWD[BF16](t, table)
    assert out.shape == (2, 2, D) and (out[0, 0] == 3).all() and (out[0, 1] == 2).all() and not out[1].any()
    table.fill_(7.0)
    BWD[BF16](out, t, V, d_table=table)
    assert (table[V - 1] == 3).all() and (table[1] == 2).all() and not table[2:V - 1].any() and not table[0].any()


@pytest.mark.parametrize("n", [1 << 24, 3000001])
def test_most_tokens(n):
    """Sums of small whole numbers are exact in any order."""
    g = torch.Generator("cuda").manual_seed(n)
    t = torch.randint(-1, 1000, (n,), generator=g, device="cuda", dtype=torch.int32)
    t[: n // 8] = 7  # a tree of four levels
    d = torch.randint(-1, 2, (n, 8), generator=g, device="cuda").to(BF16)
    want = torch.zeros((1001, 8), device="cuda", dtype=torch.float64)
    want.index_add_(0, torch.where(t < 0, 1000, t).long(), d.double())
    assert torch.equal(BWD[BF16](d, t, 1000).double(), want[:1000])


def test_graph_and_stream():
    for n, V in ((1000, 77), (7000, 777)):
        t, g = make("skew", n, V, 128, BF16)
        ws = torch.empty(binding.adaln_embed_bwd_workspace_bytes(n, V, 128), dtype=torch.uint8, device="cuda")
        want = BWD[BF16](g, t, V)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = BWD[BF16](g, t, V, workspace=ws)
        t2, g2 = make("skew", n, V, 128, BF16, seed=5)
        for tt, gg in ((t, g), (t2, g2), (t, g)):
            want = BWD[BF16](gg, tt, V)
            keep_t, keep_g = t.clone(), g.clone()
            t.copy_(tt), g.copy_(gg)
            ws.fill_(255)
            graph.replay()
            assert torch.equal(got, want)
            t.copy_(keep_t), g.copy_(keep_g)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a = BWD[BF16](g[:, ::2], t, V, stream=side)  # copied there
        b = FWD[BF16](t, g[:V, ::2], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, BWD[BF16](g[:, ::2], t, V)) and torch.equal(b, FWD[BF16](t, g[:V, ::2]))


def test_refusals():
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    table, g = torch.zeros((3, 8), dtype=BF16, device="cuda"), torch.zeros((4, 8), dtype=BF16, device="cuda")
    for bad in (lambda: FWD[BF16](t.float(), table), lambda: FWD[F32](t, table), lambda: FWD[BF16](t.cpu(), table),
                lambda: BWD[F32](g, t, 3), lambda: BWD[BF16](g, t, 3, d_table=g[:3].float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: FWD[BF16](t, table[0]), lambda: BWD[BF16](g[:3], t, 3),
                lambda: BWD[BF16](g, t, 3, accumulate=True), lambda: BWD[BF16](g, t, 3, d_table=g),
                lambda: BWD[BF16](g, t, 3, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: FWD[BF16](t, table, scale=float("nan")),
                lambda: FWD[BF16](t, torch.zeros((3, 12), dtype=BF16, device="cuda")),
                lambda: BWD[BF16](g, t, 3, d_table=table, accumulate=True),
                lambda: BWD[BF16](g, t, 3, d_table_acc=torch.zeros((3, 8), device="cuda"), d_table=table)):
        with pytest.raises(binding.AdaLNError):
            bad()
