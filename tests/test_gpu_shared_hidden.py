"""NaN and infinities among a request's newest tokens in a shared decode: they
reach the tokens that see them and no other."""
from __future__ import annotations

import math

import pytest
import torch

from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_decode_shared import DEV, QLEN, check, make, run

pytestmark = pytest.mark.gpu


def slot(c, b, j):
    """(page, slot) of own key j of request b."""
    return int(c["btab"][b][j // c["S"]]), j % c["S"]


def put(c, b, j, z, h, d, x):
    page, s = slot(c, b, j)
    c["pool"][(page, z, s, h, d) if c["layout"] == wl.NHD else (page, z, h, s, d)] = x


# rows of an item up to 16, 32, 64; newest keys in one tile of 64 keys and across two; a whole request of drafts
CASES = [
    (4, 8, 2, 16, wl.HND, torch.bfloat16), (4, 8, 2, 64, wl.NHD, torch.float16), (8, 8, 2, 8, wl.HND, torch.float16),
    (7, 28, 4, 32, wl.NHD, torch.bfloat16), (2, 64, 2, 16, wl.HND, torch.bfloat16), (64, 2, 2, 16, wl.HND, torch.float16),
]


@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q,Hq,H,S,layout,dtype", CASES)
def test_values_that_some_tokens_do_not_see(q, Hq, H, S, layout, dtype, x):
    lens = [q, q + 1, 63 + q // 2, 65, 64 + q, 200, 300]
    c = make([100], [5], lens, S=S, Hq=Hq, H=H, layout=layout, dtype=dtype, q=q, seed=q + S)
    base, base_lse, err = run(c)
    assert err == 0
    check(c, base, base_lse)
    group, at = Hq // H, {}  # request: {dimension: (kv head, first token that sees it)}
    for b, L in enumerate(lens):
        at[b] = {}
        for d, t in ((3, q - 1), (40, q // 2), (127, 1)):  # a value that tokens t and on see
            put(c, b, L - q + t, 1, d % H, d, x)
            at[b][d] = (d % H, t)
    out, lse, err = run(c)
    assert err == 0 and torch.equal(lse, base_lse)
    for b in at:
        want = base[b * q:(b + 1) * q].clone()
        reached = torch.zeros(want.shape, dtype=torch.bool, device=DEV)
        for d, (h, t) in at[b].items():
            reached[t:, h * group:(h + 1) * group, d] = True
        got = out[b * q:(b + 1) * q]
        assert torch.equal(got[~reached], want[~reached]), b
        assert (got[reached].isnan() if math.isnan(x) else ~got[reached].isfinite()).all(), b


@pytest.mark.parametrize("q,Hq,H,S,layout,dtype", CASES)
def test_keys_that_some_tokens_do_not_see(q, Hq, H, S, layout, dtype):
    lens = [q, 65, 64 + q, 200]
    c = make([100], [3], lens, S=S, Hq=Hq, H=H, layout=layout, dtype=dtype, q=q, seed=q + S + 1)
    base, base_lse, _ = run(c)
    group, t = Hq // H, q // 2
    for b, L in enumerate(lens):
        put(c, b, L - q + t, 0, 1, 5, math.nan)
    out, lse, err = run(c)
    assert err == 0
    for b in range(len(lens)):
        rows, seen = slice(b * q, (b + 1) * q), torch.zeros(q, Hq, dtype=torch.bool, device=DEV)
        seen[t:, group:2 * group] = True
        assert out[rows][seen].isnan().all() and lse[rows][seen].isnan().all()
        assert torch.equal(out[rows][~seen], base[rows][~seen]) and torch.equal(lse[rows][~seen], base_lse[rows][~seen])


def test_requests_shorter_than_their_tokens():
    # tokens before the own keys see the prefix alone, whatever the keys hold
    q, lens = 5, [0, 1, 3, 4]
    c = make([90], [3], lens, q=q, seed=3)
    base, base_lse, err = run(c)
    assert err == QLEN
    for b, L in enumerate(lens):
        for j in range(L):
            put(c, b, j, 1, 0, 9, math.nan)
    out, lse, err = run(c)
    assert err == QLEN and torch.equal(lse, base_lse)
    for b, L in enumerate(lens):
        rows, seen = slice(b * q, (b + 1) * q), torch.zeros(q, 8, 128, dtype=torch.bool, device=DEV)
        seen[q - L:, :4, 9] = True
        assert out[rows][seen].isnan().all() and torch.equal(out[rows][~seen], base[rows][~seen])
