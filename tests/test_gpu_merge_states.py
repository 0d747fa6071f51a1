"""Merging attention over separate parts of the keys, against 64 bits.

Bound: a weight e^(l - L) is off by (4 + |l - m| log2 e) 2^-22 of itself (the
exponent's fp32 argument, 2^x and the division), a result by twice that of
each part's share, then one rounding to its type."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def plain(states):
    o = torch.stack([x.double() for x, _ in states])
    l = torch.stack([y.double() for _, y in states])
    gone = torch.isneginf(l)
    o = torch.where(gone[..., None], 0.0, o)
    lse = torch.logsumexp(l, 0)
    none = torch.isneginf(lse)
    w = torch.where(gone, 0.0, torch.exp(l - torch.where(none, 0.0, lse)))
    out = (w[..., None] * o).sum(0)
    m = torch.where(none, 0.0, l.amax(0))
    rel = torch.where(gone, 0.0, (4 + (l - m).abs() * 1.4427) * 2.0 ** -22)
    share = (w * rel).sum(0)
    room = 2 * ((w * rel)[..., None] * o.abs()).sum(0) + 2 * share[..., None] * out.abs()
    return out, lse, room, 2 * share + 2.0 ** -22 * (1 + torch.where(none, 0.0, lse).abs())


def check(got, states, dtype):
    out, lse, room, lse_room = plain([(o.cpu(), l.cpu()) for o, l in states])
    g, gl = got[0].cpu().double(), got[1].cpu().double()
    assert ((g - out).abs() <= room + U[dtype] * (out.abs() + room) + 2.0 ** -25).all()
    assert torch.equal(torch.isneginf(gl), torch.isneginf(lse))
    seen = ~torch.isneginf(lse)
    assert ((gl - lse).abs()[seen] <= lse_room[seen]).all()
    assert (g[~seen] == 0).all()


def make(n, rows, heads, d, dtype, seed, spread=2.0, empty=0.3):
    g = wl.generator(seed)
    states = []
    for _ in range(n):
        l = torch.randn(rows, heads, generator=g) * spread
        l[torch.rand(rows, heads, generator=g) < empty] = -math.inf
        o = torch.randn(rows, heads, d, generator=g).to(dtype)
        o[torch.isneginf(l)] = math.nan  # counts for nothing
        states.append((o.to(DEV), l.to(DEV)))
    return states


@pytest.mark.parametrize("n,rows,heads,d,dtype,spread,empty", [
    (1, 1, 1, 8, torch.bfloat16, 1.0, 0.0), (2, 64, 32, 128, torch.bfloat16, 2.0, 0.3), (3, 7, 5, 64, torch.float16, 20.0, 0.2),
    (5, 33, 3, 192, torch.bfloat16, 60.0, 0.5), (4, 100, 1, 256, torch.float16, 2.0, 0.8), (16, 9, 2, 72, torch.float16, 5.0, 0.4),
    (2, 3, 4, 128, torch.bfloat16, 1.0, 1.0), (8, 1000, 3, 24, torch.bfloat16, 3.0, 0.1),
])
def test_merge(n, rows, heads, d, dtype, spread, empty):
    states = make(n, rows, heads, d, dtype, n * 100 + d, spread, empty)
    check(pk.paged_merge_states(states), states, dtype)


def test_large_log_sum_exps():
    states = make(3, 20, 4, 128, torch.bfloat16, 9, spread=0.5, empty=0.0)
    states = [(o, l + 30000.0) for o, l in states]
    check(pk.paged_merge_states(states), states, torch.bfloat16)
    states = [(o, l - 60000.0) for o, l in states]
    check(pk.paged_merge_states(states), states, torch.bfloat16)


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("d", [24, 128, 192])
def test_result_in_place_of_a_part(which, d):
    states = make(2, 301, 7, d, torch.bfloat16, 11)
    want = pk.paged_merge_states(states)
    mine = [(o.clone(), l.clone()) for o, l in states]
    got = pk.paged_merge_states(mine, out=mine[which][0], lse=mine[which][1])
    assert got[0] is mine[which][0] and got[1] is mine[which][1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_nan_stays_in_its_row():
    states = make(3, 10, 4, 128, torch.bfloat16, 12, empty=0.0)
    want = pk.paged_merge_states(states)
    states[1][1][2, 3] = math.nan
    states[0][0][5, 1, 17] = math.nan
    got = pk.paged_merge_states(states)
    assert got[0][2, 3].isnan().all() and got[1][2, 3].isnan()
    assert got[0][5, 1, 17].isnan() and torch.equal(got[1][5], want[1][5])
    keep = torch.ones(10, 4, dtype=torch.bool, device=DEV)
    keep[2, 3] = keep[5, 1] = False
    assert torch.equal(got[0][keep], want[0][keep])
    assert got[0][5, 1].isnan().sum() == 1


def test_the_same_part_twice_and_no_rows():
    states = make(1, 5, 3, 128, torch.float16, 13, empty=0.0)
    check(pk.paged_merge_states(states * 2), states * 2, torch.float16)
    o, l = states[0]
    out, lse = pk.paged_merge_states([(o[:0], l[:0])])
    assert out.shape == (0, 3, 128) and lse.shape == (0, 3)
