"""The calls of include/adaln_ops.h on the stream they are given: a raw handle
means that stream, and the default stream's own handle is 0."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def L():
    return lib()


def calls():
    """One input a call and the call itself, its result as a list of tensors."""
    g = torch.Generator().manual_seed(0)
    q = torch.randn((2, 40, 4, 64), generator=g)
    cos, sin = torch.rand((40, 32), generator=g).cuda(), torch.rand((40, 32), generator=g).cuda()
    t = torch.randint(0, 9, (50,), generator=g).cuda()
    rows = torch.randn((50, 64), generator=g)
    table = torch.randn((9, 64), generator=g)
    out = []
    for f32 in (False, True):
        def to(x, f32=f32):
            return x.cuda() if f32 else x.to(torch.bfloat16).cuda()

        pre = "adaln_f32_" if f32 else "adaln_"
        fwd, bwd = getattr(b, pre + "qk_norm_rope_fwd"), getattr(b, pre + "qk_norm_rope_bwd")
        look, back = getattr(b, pre + "embed_fwd"), getattr(b, pre + "embed_bwd")
        out += [(to(q), lambda x, s, f=fwd: [f(x, None, None, None, cos, sin, stream=s)[0]]),
                (to(q), lambda x, s, f=bwd: [f(x, None, x, None, None, None, cos, sin, stream=s)[i] for i in (0, 2)]),
                (to(table), lambda x, s, f=look: [f(t, x, stream=s)]),
                (to(rows), lambda x, s, f=back: [f(x, t, 9, stream=s)])]
    out += [(torch.randn(5000, generator=g).cuda(), lambda x, s: [b.adaln_grad_norm([x], stream=s)]),
            (torch.randn(5000, generator=g).cuda(),
             lambda x, s: [*(r := b.adaln_grad_clip([x], 0.5, stream=s))[0], r[1]])]
    return out


@pytest.mark.parametrize("handle", [0, 1])
def test_default_stream_by_its_handle(handle):
    """A call given the default stream's handle waits for what was enqueued there, whatever stream is current."""
    torch.zeros(1, device="cuda")
    assert torch.cuda.default_stream().cuda_stream == 0
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for x, call in calls():
        want = call(x * 2, None)
        torch.cuda.synchronize()
        for _ in range(20):  # several milliseconds on the default stream, then the input changes
            big.add_(1)
        x.mul_(2)
        with torch.cuda.stream(side):
            got = call(x, handle)
            assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want))


def test_other_streams_by_their_handles():
    """A stream's handle and the stream itself are the same: the call follows what was enqueued there."""
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        for x, call in calls():
            want = call(x * 2, None)
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                for _ in range(20):
                    big.add_(1)
                x.mul_(2)
            got = call(x, s)
            torch.cuda.synchronize()
            assert all(torch.equal(a, w) for a, w in zip(got, want))
