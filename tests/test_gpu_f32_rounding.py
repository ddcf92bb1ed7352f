"""The fp32 norm's stated roundings, bit for bit: every product that the contract
rounds before it is added is rounded."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


# a row in 2, 4, 8, 12, 24 and 32 vectors a lane, whole and with empty steps
SIZES = [(2, 300, 64), (3, 50, 200), (2, 33, 256), (1, 70, 504), (2, 65, 512), (2, 40, 1024), (2, 64, 1160),
         (1, 64, 1536), (2, 33, 2056), (2, 70, 3072), (1, 65, 3080), (1, 64, 4096)]


def same(a, b):
    return torch.equal(a.contiguous().cpu().view(torch.int32), b.contiguous().cpu().view(torch.int32))


def inputs(B, S, D):
    gen = torch.Generator("cuda").manual_seed(D)
    x = torch.randn((B, S, D), generator=gen, device="cuda") + 0.3
    return x, 0.3 * torch.randn((B, 2 * D), generator=gen, device="cuda")


def parts(x, emb, mean, rstd):
    """xhat, onep, shift on the CPU, where each operation is rounded by itself."""
    D = x.shape[-1]
    e = emb.cpu()[:, None]
    return (x.cpu() - mean.cpu()[..., None]) * rstd.cpu()[..., None], 1 + e[..., :D], e[..., D:]


@pytest.mark.parametrize("B,S,D", SIZES)
def test_output(B, S, D):
    """out = fp32(fp32(xhat * onep) + shift), with records and without; taken again from
    records that hold x exactly, it is the same."""
    x, emb = inputs(B, S, D)
    for exact in (False, True):
        if exact:
            x = binding.adaln_f32_ckpt8_unpack(binding.adaln_f32_ckpt8_pack(x), D)
        out, mean, rstd = binding.adaln_f32_out_fwd(x, emb)
        xhat, onep, shift = parts(x, emb, mean, rstd)
        assert same(out, xhat * onep + shift)
        out8, mean8, rstd8, ckpt = binding.adaln_f32_out_fwd_ckpt8(x, emb)
        assert same(out8, out) and same(mean8, mean) and same(rstd8, rstd)
        if exact:
            assert same(binding.adaln_f32_out_again_ckpt8(ckpt, emb, mean, rstd), out)


@pytest.mark.parametrize("B,S,D", SIZES + [(4, 77, 768), (1, 65, 2304), (1, 40, 2688)])
def test_gradient(B, S, D):
    """dx = fp32(rstd * fp32(fp32(gh - c1) - fp32(xhat * c2))), gh = fp32(g * onep), from x
    and from its records.  One g that is not zero in a row, so that the row's sums have
    one term: c1 = fp32(gh / D) and c2 = fp32(fp32(p * onep) / D), p = fp32(g * xhat)."""
    x, emb = inputs(B, S, D)
    gen = torch.Generator().manual_seed(S)
    at = torch.randint(0, D, (B, S, 1), generator=gen)
    dy = torch.zeros(B, S, D).scatter_(-1, at, torch.randn((B, S, 1), generator=gen))
    _, mean, rstd, ckpt = binding.adaln_f32_out_fwd_ckpt8(x, emb)
    for src, dx in ((x, binding.adaln_f32_out_bwd(dy.cuda(), x, emb, mean, rstd)[0]),
                    (binding.adaln_f32_ckpt8_unpack(ckpt, D),
                     binding.adaln_f32_out_bwd_ckpt8(dy.cuda(), ckpt, emb, mean, rstd)[0])):
        xhat, onep, _ = parts(src, emb, mean, rstd)
        gh, p = dy * onep, dy * xhat
        c1 = gh.gather(-1, at) / D
        c2 = (p * onep).gather(-1, at) / D
        assert same(dx, rstd.cpu()[..., None] * ((gh - c1) - xhat * c2))
