"""What a NaN or an infinity among the visible keys and values does to the
rows that see it, in attention under a window with first tokens and over E4M3
caches with block scales: as in the formula, a NaN key makes out and lse NaN."""
from __future__ import annotations

import pytest
import torch

import _plain
import test_gpu_prefill_window as pw
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

PREFILL = [
    # q len, kv len, page, block, Hq, H, d, layout, dtype, window, first
    (300, 500, 16, None, 4, 2, 128, wl.HND, torch.bfloat16, 100, 4),
    (300, 500, 16, None, 4, 2, 192, wl.NHD, torch.float16, 100, 4),
    (300, 500, 32, None, 4, 2, 128, wl.NHD, torch.float16, 5000, 4),   # a window that reaches every key
    (300, 500, 16, 16, 4, 2, 128, wl.HND, torch.bfloat16, -1, 0),
    (300, 500, 32, 8, 4, 2, 192, wl.NHD, torch.float16, -1, 0),
    (300, 500, 16, 16, 4, 2, 128, wl.HND, torch.float16, 130, 7),
]


P_BAD = [(i, bad) for i, c in enumerate(PREFILL) for bad in (NAN, INF) if bad != INF or not c[3]]  # (E4M3 has no infinity)


@pytest.mark.parametrize("key", [250, 499, 0])
@pytest.mark.parametrize("case, bad", [(PREFILL[i], bad) for i, bad in P_BAD], ids=[f"p{i}-{bad}" for i, bad in P_BAD])
def test_prefill_key(case, key, bad):
    n, L, S, G, Hq, H, d, layout, dtype, window, first = case
    c = pw.make([n, 40], [L, 200], S, Hq, H, d, layout, dtype, 3, window, first, G=G)
    page, slot = c["pt"].pages[0][key // S], key % S
    raw = c["k"].view(torch.uint8) if G else c["k"]
    row = raw[page, slot, 1] if layout == wl.NHD else raw[page, 1, slot]
    c["q"][..., 7] = c["q"][..., 7].abs() + 0.125  # (an infinite logit has one sign)
    row[7] = 0x7F if G else bad
    out, lse = pw.call(c, 0.05)
    sees = _plain.visible(torch.arange(L), torch.arange(L - n, L), window, first)[:, key]
    o, l = out.cpu().float(), lse.cpu()
    assert torch.isnan(o[:n][sees][:, Hq // 2:]).all() and torch.isnan(l[:n][sees][:, Hq // 2:]).all()
    # the rows and heads that do not see it are those of a cache without it
    row[7] = 0
    ok = torch.ones(n + 40, Hq, dtype=torch.bool)
    ok[:n, Hq // 2:] = ~sees[:, None]
    want = pw.call(c, 0.05)
    assert torch.equal(o[ok], want[0].cpu().float()[ok]) and torch.equal(l[ok], want[1].cpu()[ok])
    pw.compare(c, *want, 0.05)


@pytest.mark.parametrize("case", PREFILL, ids=[f"p{i}" for i in range(len(PREFILL))])
def test_prefill_value(case):
    """A NaN in a value that every query sees: that column of out, no other, and not lse."""
    n, L, S, G, Hq, H, d, layout, dtype, window, first = case
    n = min(n, 60)
    c = pw.make([n, 40], [L, 200], S, Hq, H, d, layout, dtype, 4, window, first, G=G)
    key = L - n - 20
    page, slot = c["pt"].pages[0][key // S], key % S
    raw = c["v"].view(torch.uint8) if G else c["v"]
    row = raw[page, slot, 1] if layout == wl.NHD else raw[page, 1, slot]
    row[7] = 0x7F if G else NAN
    out, lse = pw.call(c, 0.05)
    o = out.cpu().float()
    assert torch.isnan(o[:n, Hq // 2:, 7]).all()
    o[:n, Hq // 2:, 7] = 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
