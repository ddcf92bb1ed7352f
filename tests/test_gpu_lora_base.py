"""Samples without an adapter: out is y and dx the base, whatever bits they hold."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from test_gpu_lora import NAME, TYPES, fn, inputs, run, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("S", [1, 2, 3, 4, 8, 100, 700])
def test_bits_of_the_base_are_kept(t, S):
    """-0 and the other bit patterns, in place and not, with adapters for other samples
    and with none at all."""
    B, K, N = 4, 72, 136
    c = inputs(t, B, S, K, N, 16, 2)
    c["ids"] = torch.tensor([-1, 1, 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    gen = torch.Generator("cuda").manual_seed(S)
    whole = torch.int16 if t == torch.bfloat16 else torch.int32
    for k in ("y", "dx_base"):
        i = torch.iinfo(whole)
        v = torch.randint(i.min, i.max, c[k].shape, generator=gen, device="cuda", dtype=whole)
        v[..., ::3] = i.min  # -0
        c[k][[0, 2, 3]] = v.view(t)[[0, 2, 3]]
    free = [0, 2, 3]
    none = {**c, "A": c["A"][:0], "U": c["U"][:0], "scale": c["scale"][:0]}
    for d, which in ((c, free), (none, list(range(B)))):
        out, dx, _, _ = run(t, d)
        assert same(out[which], d["y"][which]) and same(dx[which], d["dx_base"][which])
        w = (d["A"], d["U"], d["scale"], d["ids"])
        y, base = d["y"].clone(), d["dx_base"].clone()
        _, state = fn("lora_fwd", t)(d["x"], *w, y=y, out=y)
        fn("lora_bwd", t)(d["d_out"], d["x"], state, *w, dx_base=base, dx=base)
        assert same(y, out) and same(base, dx)
