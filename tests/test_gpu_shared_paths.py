"""The paths of decode over shared prefixes that sizes, strides and the
device's own numbers choose between: page strides that no wide map fits,
teams of CTAs (some of whose members have no tile), many groups, own keys in
several splits and more items than CTAs, pools past 32 bits.  Against the
definition in 64 bits, under the bounds that the roundings allow."""
from __future__ import annotations

import math

import pytest
import torch

import _plain
import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_decode_shared import DEV, I32, QLEN, U, args, check, make, run

pytestmark = pytest.mark.gpu


def padded(c, extra):
    """The pool's K and V with `extra` elements (NaN) between pages."""
    P, page = c["pool"].shape[0], c["pool"][0, 0].numel()
    out = []
    for z in range(2):
        flat = torch.full((P, page + extra), math.nan, dtype=c["dtype"], device=DEV)
        flat[:, :page] = c["pool"][:, z].reshape(P, page).to(DEV)
        out.append(flat[:, :page].view(P, *c["pool"].shape[2:]))
    return tuple(out)


@pytest.mark.parametrize("extra", [8, 128, 4096])
@pytest.mark.parametrize("S,layout", [(8, wl.HND), (16, wl.HND), (16, wl.NHD), (64, wl.NHD), (128, wl.HND), (256, wl.NHD)])
def test_pages_with_gaps(S, layout, extra):
    c = make([515, 30], [40, 3], [1 + (i * 13) % 200 for i in range(45)], S=S, layout=layout, seed=S + extra)
    out, lse, err = run(c, kv_cache=padded(c, extra))
    assert err == 0
    check(c, out, lse, requests=[0, 5, 39, 40, 42, 43, 44])
    # the same bits from pages without gaps: other maps, the same tiles
    want, want_lse, _ = run(c)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("B,q,Hq,sizes", [
    (70, 1, 64, [70]),       # teams
    (70, 1, 64, [33]),       # a team's last members without a tile
    (70, 1, 64, [5]),        # one tile in a team
    (70, 1, 64, [3, 60, 7]),  # several groups
    (100, 2, 32, [100]),
])
def test_long_prefixes_in_teams(B, q, Hq, sizes):
    # 16,500 keys of 8 heads: 68 MB, more than the prefixes that stay without teams
    P = [16500, 300, 9000][:len(sizes)]
    c = make(P, sizes, [q + (i * 7) % 40 for i in range(B)], S=64, Hq=Hq, H=8, q=q, seed=B + len(sizes) + sizes[0], poison=False)
    out, lse, err = run(c)
    assert err == 0
    check(c, out, lse, requests=sorted({0, sizes[0] - 1, min(sizes[0], B - 1), B // 2, B - 1}))
    again, again_lse, _ = run(c)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_more_than_32_groups():
    sizes = [i % 4 for i in range(70)]
    prefix = [(i * 37) % 300 if i % 5 else 0 for i in range(70)]
    B = sum(sizes) + 2
    c = make(prefix, sizes, [1 + i % 20 for i in range(B)], Hq=4, H=2, seed=21)
    out, lse, err = run(c)
    assert err == 0
    check(c, out, lse)


@pytest.mark.parametrize("S,Hq,H,q,dtype", [
    (8, 8, 2, 1, torch.bfloat16), (16, 16, 1, 1, torch.float16), (256, 14, 2, 4, torch.float16), (64, 16, 2, 8, torch.bfloat16),
])
def test_own_keys_in_splits(S, Hq, H, q, dtype):
    c = make([300], [4], [700, q, 255, 1601, 256, 5000], S=S, Hq=Hq, H=H, q=q, dtype=dtype, seed=S, sinks=True)
    out, lse, err = run(c)
    assert err == 0
    check(c, out, lse)


def test_more_items_than_ctas():
    lens = [(i * 331) % 900 for i in range(150)]  # 0 among them
    c = make([64], [150], lens, Hq=8, H=4, S=32, seed=31)
    out, lse, err = run(c)
    assert err == QLEN
    check(c, out, lse, requests=[0, 1, 2, 50, 77, 120, 148, 149])
    for _ in range(3):
        again, again_lse, _ = run(c)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_requests_without_own_keys():
    c = make([200], [3], [0, 0, 0, 0], seed=32, Hq=16, H=2)
    out, lse, err = run(c)
    assert err == QLEN
    check(c, out, lse)
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()


def test_replays_follow_the_prefixes():
    c = make([900, 700], [20, 30], [1 + i % 70 for i in range(50)], seed=33)
    a = args(c)
    pk.paged_decode_shared(**a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.paged_decode_shared(**a)
    for prefix in ([900, 700], [1, 700], [513, 0], [0, 0], [640, 129]):
        a["prefix_lens"].copy_(torch.tensor(prefix, device=DEV, **I32))
        g.replay()
        torch.cuda.synchronize()
        c["prefix"] = prefix
        check(c, a["out"], a["lse"], requests=[0, 19, 20, 49])


def test_pools_past_32_bits():
    # 4.9 GB of pages, the ones in use at the end
    S, Hq, H, P, lens = 16, 8, 2, 200, [40, 3, 300]
    n = 300000
    g = wl.generator(41)
    need = [-(-x // S) for x in [P] + lens]
    ids = n - 1 - torch.randperm(sum(need), generator=g).to(torch.int32)
    pool = torch.empty(n, 2, H, S, 128, dtype=torch.bfloat16, device=DEV)
    part = torch.randn(sum(need), 2, H, S, 128, generator=g).to(torch.bfloat16)
    pool[n - sum(need):] = part.to(DEV)
    table = torch.full((4, max(need)), 0x7FFFFFFF, **I32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = ids[at:at + k]
        at += k
    q = torch.randn(3, Hq, 128, generator=g).to(torch.bfloat16)
    ws = torch.empty(pk.paged_decode_shared_workspace_size(3, 1, Hq, H, 128, 1, P, 300, S), dtype=torch.uint8, device=DEV)
    lse = torch.empty(3, Hq, device=DEV)
    out = pk.paged_decode_shared(q.to(DEV), pool, ws, table[:1].to(DEV), torch.tensor([P], device=DEV, **I32),
                                 torch.tensor([0, 3], device=DEV, **I32), P, table[1:].to(DEV),
                                 torch.tensor(lens, device=DEV, **I32), 300, bmm1_scale=0.09, lse=lse)
    local = table - (n - sum(need))
    for b in range(3):
        kv = [torch.cat((_plain.tokens(part[:, z], local[0], P, S, wl.HND),
                         _plain.tokens(part[:, z], local[1 + b], lens[b], S, wl.HND))).double() for z in range(2)]
        o, l, bo, bl = _plain.attention(q[b:b + 1].double(), *kv, P + lens[b], 0.09, u_p=U[torch.bfloat16], u_out=U[torch.bfloat16])
        _plain.check(out[b:b + 1], o, bo, f"out {b}")
        _plain.check(lse[b:b + 1], l, bl, f"lse {b}")


def test_on_a_stream_of_its_own_while_others_run():
    c = make([600], [30], [1 + (i * 11) % 300 for i in range(30)], seed=42)
    a, b = args(c), args(c)
    want = pk.paged_decode_shared(**a).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device=DEV)
    for _ in range(10):
        y = x @ x
        b["out"].zero_()
        side.wait_stream(torch.cuda.current_stream())
        pk.paged_decode_shared(**b, stream=side)
        a["out"].zero_()
        pk.paged_decode_shared(**a)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(a["out"], want) and torch.equal(b["out"], want)
    assert y.isfinite().all()
