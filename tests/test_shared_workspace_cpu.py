"""The workspace of a shared decode, reserved once for a server's maxima,
holds every call that has no more of anything."""
from __future__ import annotations

import random

import pytest

from test_abi_cpu import lib  # noqa: F401  (the built library, a fixture)


def size(lib, B, Q, G, prefix, own, heads=(32, 8), page=16):  # noqa: F811
    return lib.paged_decode_shared_workspace_size(B, Q, *heads, 128, G, prefix, own, page)


@pytest.mark.parametrize("heads", [(64, 8), (32, 8), (28, 4), (8, 8), (64, 1), (48, 1)])
def test_smaller_calls_need_no_more(lib, heads):  # noqa: F811
    g = random.Random(heads[0])
    most_q = max(1, 64 // (heads[0] // heads[1]))
    top = (512, min(8, most_q), 512, 200000, 70000)
    for _ in range(4000):
        a = [max(1, round(t ** g.random())) for t in top]
        b = [max(0 if i > 1 else 1, round(x * g.random() ** 0.3)) if g.random() < 0.6 else x for i, x in enumerate(a)]
        large, small = size(lib, *a, heads=heads), size(lib, *b, heads=heads)
        assert 0 < small <= large, (a, b)


@pytest.mark.parametrize("which", range(5))
def test_one_size_at_a_time(lib, which):  # noqa: F811
    base, steps = [64, 2, 3, 9000, 3000], [range(1, 600), range(1, 9), range(0, 300), range(0, 40000, 37), range(0, 40000, 37)]
    last = 0
    for x in steps[which]:
        a = list(base)
        a[which] = x
        n = size(lib, *a)
        assert n >= last, (a, n, last)
        last = n


def test_a_longer_prefix(lib):  # noqa: F811
    # (the longer one's CTAs come in teams, which leave some SMs out)
    assert size(lib, 256, 1, 1, 4096, 8192, heads=(64, 8)) <= size(lib, 256, 1, 1, 32768, 8192, heads=(64, 8))
