"""include/adaln_ops.h on the host: arguments that a call does not use, and size
queries for what the calls refuse.  Pointers are fake addresses that are never
dereferenced."""

from __future__ import annotations

import os
import random
import subprocess

import pytest

from invariant_dit_adaln_gb300 import binding, build
from test_ops_abi_host import (ALIAS, DEVICE, L, at, clip, heads_bwd, heads_fwd, no_gpu, norm, rows,  # noqa: F401
                               tensors)


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


@pytest.mark.parametrize("count", [1, 60, 79, 80, 2047, 2048, 2049, 5000, 20001, 65536])
def test_overlaps_of_lists_of_any_length(L, count):  # noqa: F811
    """Lists in order, in reverse and shuffled, in place and not; then one tensor
    that reaches into another by its last byte."""
    r = random.Random(count)
    sizes = [r.randint(1, 200) for _ in range(count)]
    starts, end = [], 0
    for n in sizes:
        starts.append(end)
        end += 4 * n
    for order in ("up", "down", "any"):
        places = list(range(count))
        if order == "down":
            places.reverse()
        elif order == "any":
            r.shuffle(places)
        grads = [(at(0, starts[i]), sizes[i], 0) for i in places]
        outs = [(at(1, starts[i]), sizes[i], 0) for i in places]
        g, o = tensors(*grads), tensors(*outs)
        assert norm(L, g) == DEVICE and clip(L, g, o) == DEVICE and clip(L, g, g) == DEVICE
        k = r.randrange(count)
        half = tensors(*[grads[i] if i % 2 else outs[i] for i in range(count)])  # every second in place
        assert clip(L, g, half) == DEVICE
        assert norm(L, g, out=at(0, starts[places[k]] // 16 * 16)) == ALIAS
        if count > 1:
            j = r.choice([i for i in range(count) if i != k])
            wrong = list(outs)
            wrong[k] = (outs[j][0] + 4 * (sizes[places[j]] - 1), *outs[k][1:])  # behind the start of output j
            assert clip(L, g, tensors(*wrong)) == ALIAS
            wrong[k] = (grads[j][0] + 4 * (sizes[places[j]] - 1), *outs[k][1:])  # inside gradient j
            assert clip(L, g, tensors(*wrong)) == ALIAS
            wrong = list(grads)
            wrong[k] = wrong[j]  # scaled twice in place
            assert clip(L, g if sizes[places[k]] != sizes[places[j]] else tensors(*wrong),
                        tensors(*[(p, grads[i][1], t) for i, (p, _, t) in enumerate(wrong)])) == ALIAS


def test_overlaps_against_brute_force(L):  # noqa: F811
    r = random.Random(1)
    seen = set()
    for _ in range(300):
        count = r.randint(1, 12)
        sizes = [r.randint(0, 6) for _ in range(count)]
        space = r.choice([40, 400])
        grads = [(at(0, 4 * r.randrange(space)), n, 0) for n in sizes]
        outs = [g if r.random() < 0.4 else (at(0, 4 * r.randrange(space)), n, 0) for g, n in zip(grads, sizes)]
        written, bad = [], False
        for p, n, _ in outs:
            cells = set(range(p, p + 4 * n, 4))
            bad |= any(cells & w for w in written)
            written.append(cells)
        for i, (p, n, _) in enumerate(grads):
            cells = set(range(p, p + 4 * n, 4))
            bad |= any(cells & w for j, w in enumerate(written) if j != i or outs[j][0] != p)
        got = clip(L, tensors(*grads), tensors(*outs))
        assert got == (ALIAS if bad else DEVICE), (grads, outs)
        seen.add(got)
    assert len(seen) == 2


COUNT_MALLOC = r"""
#include <stdio.h>
#include <stdlib.h>
#include <dlfcn.h>
#include "adaln_ops.h"
static int calls, counting;
extern void *__libc_malloc(size_t), *__libc_calloc(size_t, size_t), *__libc_realloc(void *, size_t);
void *malloc(size_t n) { calls += counting; return __libc_malloc(n); }
void *calloc(size_t n, size_t m) { calls += counting; return __libc_calloc(n, m); }
void *realloc(void *p, size_t n) { calls += counting; return __libc_realloc(p, n); }
static adaln_tensor g[65536], o[65536];
int main(int argc, char **argv) {
    void *lib = dlopen(argv[1], RTLD_NOW);
    if (!lib) return puts(dlerror()), 2;
    adaln_status (*clip)(const adaln_tensor *, const adaln_tensor *, int, double, float *, void *, size_t, void *) =
        (adaln_status (*)(const adaln_tensor *, const adaln_tensor *, int, double, float *, void *, size_t, void *))
            dlsym(lib, "adaln_grad_clip");
    for (int i = 0; i < 65536; ++i) {
        int k = (int)(40503u * (unsigned)i % 65536u); /* every place once, out of order */
        g[i].data = (void *)(((size_t)1 << 40) + 512 * (size_t)k);
        o[i].data = (void *)(((size_t)2 << 40) + 512 * (size_t)k);
        g[i].numel = o[i].numel = 100;
    }
    int counts[] = {1, 79, 80, 500, 65536};
    for (int i = 0; i < 5; ++i) {
        counting = 1;
        /* a workspace of 16 bytes is too small: the last check before the device's */
        adaln_status st = clip(g, o, counts[i], 1.0, (float *)((size_t)3 << 40), (void *)((size_t)4 << 40), 4, 0);
        counting = 0;
        printf("%d %d %d\n", counts[i], (int)st, calls);
    }
    return 0;
}
"""


def test_checks_allocate_nothing(L, tmp_path):  # noqa: F811
    """The header promises it: counted in a C program whose malloc the library uses."""
    src, exe = tmp_path / "count.c", tmp_path / "count"
    src.write_text(COUNT_MALLOC)
    subprocess.run(["gcc", "-O1", "-rdynamic", f"-I{build.INCLUDE}", str(src), "-o", str(exe), "-ldl"], check=True)
    out = subprocess.run([str(exe), build.LIB], capture_output=True, text=True, check=True).stdout
    assert [tuple(map(int, line.split())) for line in out.splitlines()] == [(n, 5, 0) for n in (1, 79, 80, 500, 65536)]


def test_every_function_is_exported_and_bound(L):  # noqa: F811
    names = binding.declared_symbols(os.path.join(build.INCLUDE, "adaln_ops.h"))
    assert len(names) == 13
    for n in names:
        assert hasattr(L, n), n
        assert callable(getattr(binding, n, None)), n
