"""The C++ part of the binding (_calls.so) without a GPU: what it refuses, and
that a refused call keeps no reference to its arguments."""
from __future__ import annotations

import sys

import pytest
import torch

import paged_kv_cache_316_gb300 as pk

I32 = dict(dtype=torch.int32)


def rotary_args():
    return dict(query=torch.zeros(4, 32, 128, dtype=torch.bfloat16), key=torch.zeros(4, 8, 128, dtype=torch.bfloat16),
                positions=torch.zeros(4, **I32), frequencies=torch.ones(64, dtype=torch.float64))


@pytest.mark.parametrize("over", [
    dict(query=None), dict(query=[1.0]), dict(key=3), dict(positions="0"), dict(frequencies=None), dict(query_weight=1.0),
    dict(query=torch.zeros(4, 128)), dict(query=torch.zeros(4, 32, 128, dtype=torch.float64)),
])
def test_what_is_no_such_tensor_is_refused(over):
    with pytest.raises(pk.PagedKVError):
        pk.paged_rotary(**dict(rotary_args(), **over))


@pytest.mark.parametrize("states", [
    [], [3], [(torch.zeros(2, 2, 8, dtype=torch.half),)], [(torch.zeros(2, 2, 8, dtype=torch.half), None)],
    [(torch.zeros(2, 2, 8, dtype=torch.half), torch.zeros(2, 2), torch.zeros(2, 2))], 5,
])
def test_what_is_no_state_is_refused(states):
    with pytest.raises((pk.PagedKVError, TypeError)):
        pk.paged_merge_states(states)


def test_numbers_that_are_none():
    with pytest.raises((pk.PagedKVError, TypeError)):
        pk.paged_rotary(**rotary_args(), magnitude="one")
    with pytest.raises((pk.PagedKVError, TypeError)):
        pk.paged_rotary(**rotary_args(), rotary_start=1.5)
    with pytest.raises((pk.PagedKVError, OverflowError)):
        pk.paged_rotary(**rotary_args(), rotary_start=1 << 40)


@pytest.mark.parametrize("layout", ["NDH", 2, None, 1 << 80, b"NHD"])
def test_layouts(layout):
    a = rotary_args()
    i = torch.zeros(4, **I32)
    with pytest.raises(pk.PagedKVError, match="kv_layout"):
        pk.paged_append_rotary(a["query"], a["key"], a["key"], i, i, torch.zeros(4, 2, 16, 8, 128, dtype=torch.bfloat16), i, i[:3],
                               i[:2], a["frequencies"], kv_layout=layout)


def test_references_stay_as_they_were():
    a = rotary_args()
    o, l = torch.zeros(4, 32, 128, dtype=torch.bfloat16), torch.zeros(4, 32)
    pair = (o, l)
    states = [pair, [o, l]]
    held = [o, l, pair, states, states[1], *a.values()]
    before = [sys.getrefcount(x) for x in held]
    for _ in range(50):
        for call in (lambda: pk.paged_merge_states(states), lambda: pk.paged_merge_states(iter(states)),
                     lambda: pk.paged_merge_states(tuple(states), out=o, lse=l), lambda: pk.paged_merge_states([pair, (o,)]),
                     lambda: pk.paged_rotary(**a), lambda: pk.paged_rotary(**a, query_out=a["query"], key_out=a["key"])):
            with pytest.raises(pk.PagedKVError):
                call()
    assert [sys.getrefcount(x) for x in held] == before
