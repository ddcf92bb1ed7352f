"""include/adaln_ops.h on the host: arguments that a call does not use, and size
queries for what the calls refuse.  Pointers are fake addresses that are never
dereferenced."""

from __future__ import annotations

import pytest

from test_ops_abi_host import (ALIAS, DEVICE, L, heads_bwd, heads_fwd, no_gpu, rows)  # noqa: F401  (fixtures)


@pytest.mark.parametrize("odd", [3, 68, -5, (1 << 62) + 1, -(1 << 63)])
def test_strides_of_size_one_are_not_used(L, odd):  # noqa: F811
    """They may hold anything, and enter no overlap check either."""
    assert heads_fwd(L, B=1, q=rows(0, strides=(odd, 256, 64)), qo=rows(2, strides=(odd, 256, 64))) == DEVICE
    assert heads_fwd(L, S=1, q=rows(0, strides=(256, odd, 64)), qo=rows(2, strides=(256, odd, 64))) == DEVICE
    assert heads_fwd(L, Hq=1, q=rows(0, strides=(680, 136, odd)), qo=rows(2, strides=(680, 136, odd))) == DEVICE
    assert heads_fwd(L, Hk=1, ko=rows(3, strides=(680, 136, odd))) == DEVICE
    one = rows(0, strides=(680, 136, odd))
    assert heads_fwd(L, Hq=1, q=one, qo=one) == DEVICE
    # rows of 128 bytes, 272 apart: behind each other 128 bytes on, overlapping 64 bytes on
    assert heads_fwd(L, Hq=1, q=one, qo=rows(0, off=128, strides=(680, 136, odd))) == DEVICE
    assert heads_fwd(L, Hq=1, q=one, qo=rows(0, off=64, strides=(680, 136, odd))) == ALIAS
    over = {n: rows(i, strides=(680, 136, odd)) for i, n in ((0, "gq"), (2, "q"), (4, "dq"))}
    assert heads_bwd(L, Hq=1, over=over) == DEVICE


def test_workspace_sizes_of_refused_calls(L):  # noqa: F811
    """0, as for a call without partial sums, whatever the numbers are."""
    most, least = (1 << 31) - 1, -(1 << 31)
    heads, embed = L.adaln_qk_norm_rope_bwd_workspace_bytes, L.adaln_embed_bwd_workspace_bytes
    good = (2, 5, 4, 2, 64)
    assert heads(*good) > 0
    limits = (65535, 262144, 1024, 1024, 256)
    for i, top in enumerate(limits):
        for bad in (most, least, -1, top + 1, most - 1):
            assert heads(*good[:i], bad, *good[i + 1:]) == 0, (i, bad)
    assert heads(1, 1, most, most, 8) == 0 and heads(most, most, most, most, most) == 0
    assert heads(2, 5, 0, 2, 64) == 0 and heads(2, 5, 4, 2, 12) == 0
    assert heads(65535, 262144, 1024, 0, 256) == 0  # 2^40 elements and more
    assert heads(1, 262144, 1024, 1024, 256) > 0
    assert embed(10, 20, 64) > 0
    for bad in ((most, 20, 64), (10, most, 64), (10, 20, most), (least, least, least), (10, 20, 12), (-1, 20, 64)):
        assert embed(*bad) == 0, bad
