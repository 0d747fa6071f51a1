"""What a NaN or an infinity among the visible keys and values does to the
rows that see it, in attention under a window with first tokens and over E4M3
caches with block scales: as in the formula, a NaN key makes out and lse NaN."""
from __future__ import annotations

import pytest
import torch

import _plain
import test_gpu_decode_window as dw
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


DECODE = [
    # L, block (None: 16-bit cache), E4M3 without block scales, Hq, dtype, window, first, sinks
    (100, None, False, 8, torch.bfloat16, 5000, 1, False),
    (3000, None, False, 8, torch.float16, 5000, 1, True),       # several splits
    (100, None, False, 8, torch.bfloat16, -1, 3, False),        # no window: the first tokens have no effect
    (3000, None, False, 8, torch.float16, -1, 3, False),
    (3000, None, True, 8, torch.bfloat16, -1, 3, True),
    (100, 16, False, 8, torch.bfloat16, -1, 0, False),
    (3000, 8, False, 32, torch.float16, -1, 0, True),
    (3000, 16, False, 32, torch.bfloat16, 2500, 9, False),
]
D_IDS = [f"d{i}" for i in range(len(DECODE))]


def decode_case(case):
    L, G, e4m3, Hq, dtype, window, first, sinks = case
    c = dw.make([L, L], 16, Hq, 2, wl.HND, dtype, 39, scaled=bool(G), G=G, e4m3=e4m3, sinks=sinks, window=window,
                first=first, poison=False)
    return c, (c["pool"].view(torch.uint8) if G or e4m3 else c["pool"]), Hq // 2


D_BAD = [(i, bad) for i, c in enumerate(DECODE) for bad in (NAN, INF) if bad != INF or not (c[1] or c[2])]


@pytest.mark.parametrize("every", [False, True])  # one key; or one in each 16, so that every split has some
@pytest.mark.parametrize("case, bad", [(DECODE[i], bad) for i, bad in D_BAD], ids=[f"d{i}-{bad}" for i, bad in D_BAD])
def test_decode_key(case, every, bad):
    c, raw, half = decode_case(case)
    c["query"][..., 7] = c["query"][..., 7].abs() + 0.125  # (an infinite logit has one sign)
    pages = c["pt"].pages[0] if every else c["pt"].pages[0][-2:-1]
    raw[pages, 0, 1, 1, 7] = 0x7F if raw.dtype == torch.uint8 else bad
    out, lse = dw.call(c, 0.05)
    assert torch.isnan(out[0, half:].float()).all() and torch.isnan(lse[0, half:]).all()
    # the other head and request are those of a cache without it
    raw[pages, 0, 1, 1, 7] = 0
    want = dw.call(c, 0.05)
    assert torch.equal(out[0, :half], want[0][0, :half]) and torch.equal(out[1], want[0][1])
    assert torch.equal(lse[0, :half], want[1][0, :half]) and torch.equal(lse[1], want[1][1])
    dw.compare(c, *want, 0.05)


@pytest.mark.parametrize("case", DECODE, ids=D_IDS)
def test_decode_value(case):
    """A NaN in a value: that column of out, no other, and not lse; so an infinity, which may stay one."""
    c, raw, half = decode_case(case)
    bads = [0x7F] if raw.dtype == torch.uint8 else [NAN, INF]
    page = c["pt"].pages[0][-2]
    for bad in bads:
        raw[page, 1, 1, 3, 7] = bad
        out, lse = dw.call(c, 0.05)
        o = out.cpu().float()
        assert not torch.isfinite(o[0, half:, 7]).any()
        assert bad is INF or torch.isnan(o[0, half:, 7]).all()
        o[0, half:, 7] = 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
