"""Merged states whose parts lie far apart: what a part holds counts the same
wherever it stands among the parts."""
from __future__ import annotations

import itertools
import math

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("x", [math.nan, math.inf])
@pytest.mark.parametrize("n", [2, 5, 9])
def test_a_part_of_no_weight_left(n, x):
    # the weight of a part 200 below the others is 0 in fp32; its log-sum-exp is finite, so the row sees its keys
    g = wl.generator(n)
    for at in range(n):
        states = [(torch.randn(3, 2, 128, generator=g).to(torch.bfloat16), torch.randn(3, 2, generator=g)) for _ in range(n)]
        states[at][1][1] = -200.0
        clean = pk.paged_merge_states([(o.to(DEV), l.to(DEV)) for o, l in states])
        states[at][0][1, 0, 7] = x
        out, lse = pk.paged_merge_states([(o.to(DEV), l.to(DEV)) for o, l in states])
        assert not out[1, 0, 7].isfinite() and torch.equal(lse, clean[1])
        keep = torch.ones(3, 2, 128, dtype=torch.bool, device=DEV)
        keep[1, 0, 7] = False
        assert torch.equal(out[keep], clean[0][keep]) and out[keep].isfinite().all()


def test_parts_that_see_nothing_count_for_nothing():
    o = torch.randn(3, 1, 1, 8).to(torch.float16).to(DEV)
    o[1] = math.nan
    l = torch.tensor([0.5, -math.inf, 0.25], device=DEV).view(3, 1, 1)
    want = pk.paged_merge_states([(o[0], l[0]), (o[2], l[2])])
    for order in itertools.permutations(range(3)):
        got = pk.paged_merge_states([(o[i], l[i]) for i in order])
        assert got[0].isfinite().all() and (got[0] - want[0]).abs().max() <= 2.0 ** -9
