"""adaln_embed_bwd where tokens occur often and rows span several groups of 256
columns: tickets, partial sums and dead lanes of every group."""

from __future__ import annotations

import pytest
import torch

import ops_ref
from gpu_util import lib
from test_gpu_embed import BF16, BWD, F32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def check(t, g, V, dtype, scale=0.37):
    """Bit for bit in the documented order, and within its error of 64 bits; into an accumulator too."""
    want = ops_ref.embed_bwd_order(g, t, V, scale)
    exact, size, count = ops_ref.embed_bwd(g, t, V, scale)
    got = BWD[dtype](g, t, V, scale=scale)
    assert torch.equal(got.cpu(), want)
    # 32 a level, three levels here, the scale
    depth = 32.0 + 32 * (count > 32) + 32 * (count > 1024) + 1
    ops_ref.check(got, exact, depth[:, None] * ops_ref.U * size, "gradient")
    if dtype == BF16:
        low = torch.full(got.shape, 7.0, dtype=BF16, device="cuda")
        BWD[BF16](g, t, V, scale=scale, d_table=low)
        assert torch.equal(low.cpu(), want.to(BF16))
    acc = torch.full(got.shape, 0.5, device="cuda")
    BWD[dtype](g, t, V, scale=scale, d_table_acc=acc, accumulate=True)
    assert torch.equal(acc.cpu(), torch.where(count[:, None] > 0, 0.5 + want, torch.tensor(0.5)))
    return count


def rows(n, D, dtype, seed):
    return torch.randn((n, D), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [256, 264, 520, 1032])
def test_counts_around_the_trees(D, dtype):
    """Tokens of 1 to 1100 occurrences at the edges of pieces and nodes, shuffled."""
    counts = [1, 31, 32, 33, 34, 63, 64, 65, 0, 96, 97, 1023, 1024, 1025, 1056, 1057, 1100]
    t = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    t = t[torch.randperm(len(t), generator=torch.Generator().manual_seed(D))].cuda()
    got = check(t, rows(len(t), D, dtype, D), len(counts), dtype)
    assert got.tolist() == counts


# one CTA's sort, the cluster's, and the kernels' (more than 32768 tokens; a token and a place beyond 32 bits)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,V,D", [(4096, 1001, 520), (4097, 37, 264), (20000, 300, 264), (33000, 500, 264),
                                   (3000, 1 << 21, 520)])
def test_labels_with_a_tenth_on_one(n, V, D, dtype):
    g = torch.Generator().manual_seed(n)
    t = torch.randint(0, min(V, 1200), (n,), generator=g)
    t[torch.rand(n, generator=g) < 0.1] = min(V, 1200) - 1
    t[torch.rand(n, generator=g) < 0.02] = -1
    if V > 70000:  # the reference's tables are of the tokens used
        small = check(t.cuda(), rows(n, D, dtype, 1), 1200, dtype)
        wide = BWD[dtype](rows(n, D, dtype, 1), torch.where(t >= 0, t + (V - 1200), -1).cuda(), V)
        assert torch.equal(wide[-1200:], BWD[dtype](rows(n, D, dtype, 1), t.cuda(), 1200))
        assert not wide[:-1200].any() and small.max() > 200
    else:
        check(t.cuda(), rows(n, D, dtype, 1), V, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V,kind", [(2000, "skew"), (40000, "even"), (1500, "even")])
def test_tasks_of_32_places(V, kind, dtype):
    """Enough rows for the larger tasks: runs within them, across them, and long ones."""
    n, D = 50000, 1032
    assert n * 5 >= 2 * 32 * 3 * torch.cuda.get_device_properties(0).multi_processor_count * 8
    t, _ = make(kind, n, V, 8, dtype, seed=V)
    check(t, rows(n, D, dtype, V), V, dtype)


def test_captured_with_a_kept_workspace():
    """Replayed on other tokens, with rubbish in the workspace."""
    from invariant_dit_adaln_gb300 import binding
    n, V, D = 6000, 90, 520
    t, _ = make("skew", n, V, 8, BF16)
    g = rows(n, D, BF16, 2)
    ws = torch.empty(binding.adaln_embed_bwd_workspace_bytes(n, V, D), dtype=torch.uint8, device="cuda")
    BWD[BF16](g, t, V, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = BWD[BF16](g, t, V, workspace=ws)
    for kind, seed in (("skew", 1), ("even", 2), ("one", 3), ("none", 4), ("skew", 5)):
        t.copy_(make(kind, n, V, 8, BF16, seed=seed)[0])
        ws.fill_(255)
        graph.replay()
        assert torch.equal(got.cpu(), ops_ref.embed_bwd_order(g, t, V, 1.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_padding_are_not_read(dtype):
    """NaN and infinities at padding tokens change nothing; a NaN at a token stays in its row and column."""
    for n, V, D in ((700, 50, 264), (9000, 40, 264), (33000, 3000, 8)):
        t, _ = make("skew", n, V, 8, dtype, seed=n)
        g = rows(n, D, dtype, n)
        want = BWD[dtype](g, t, V)
        bad = (t < 0) | (t >= V)
        assert bad.sum() > 32
        g[bad] = float("nan")
        g[bad.nonzero()[::2, 0]] = float("-inf")
        assert torch.equal(BWD[dtype](g, t, V), want)
        token = int(t[t >= 0].mode().values)
        g[(t == token).nonzero()[-1, 0], D - 3] = float("nan")
        got = BWD[dtype](g, t, V)
        assert got[token, D - 3].isnan()
        got[token, D - 3] = want[token, D - 3]
        assert torch.equal(got, want)
