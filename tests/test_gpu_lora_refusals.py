"""Sizes that the adapters' calls do not take are refused as sizes, whichever dimension
it is and whether out and dx are given or not."""

from __future__ import annotations

import pytest
import torch

from gpu_util import lib
from invariant_dit_adaln_gb300 import binding as b
from test_gpu_lora import NAME, TYPES, fn, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    return lib()


@pytest.mark.parametrize("t", TYPES, ids=NAME.get)
@pytest.mark.parametrize("K,N,R", [(100, 64, 8), (64, 100, 8), (64, 60, 8), (4, 64, 8), (64, 65544, 8), (64, 64, 12),
                                   (64, 64, 136)])
def test_sizes(t, K, N, R):
    c = inputs(t, 2, 5, K, N, R, 1)
    w = (c["A"], c["U"], c["scale"], c["ids"])
    with pytest.raises(b.AdaLNError, match="SHAPE"):
        fn("lora_fwd", t)(c["x"], *w)
    state = torch.zeros(b.adaln_lora_state_bytes(2, 5, 136 if R > 128 else 16) or 65536, dtype=torch.uint8,
                        device="cuda")
    with pytest.raises(b.AdaLNError, match="SHAPE"):
        fn("lora_bwd", t)(c["d_out"], c["x"], state, *w)
