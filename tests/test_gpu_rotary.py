"""Norms, rotations and the append of rotated keys against the definition in
64 bits.

Bound of a rotated element y' = m (u cos a - v sin a): one rounding to its type
(u_out |y'|, or half a step of fp16's smallest), and in fp32: the sum of up to
256 squares, the reciprocal root and two products leave y off by at most
12 * 2^-24 of itself; the angle's fp32 form, cos and sin are off by 3 * 2^-23
(half a turn is pi, rounded at 2^-24; the functions' own two units) and the
products by 4 * 2^-24.  Together below 2^-19 m (|u| + |v|)."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
BATCH, POS, PAGE = 4, 2, 1


def plain(x, w, pos, f, start, paired, mag, eps):
    """(values, bounds without the last rounding) of [tokens, heads, D] in float64."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.double()
    out, room = y.clone(), y.abs() * 2.0 ** -20
    n = f.numel()
    i = torch.arange(n)
    a, b = (start + 2 * i, start + 2 * i + 1) if paired else (start + i, start + n + i)
    # angles by their turns, so that 64 bits hold at any position
    step = f / (2 * math.pi)
    angle = torch.remainder(pos.double()[:, None] * step, 1.0)[:, None] * (2 * math.pi)
    c, s = torch.cos(angle) * mag, torch.sin(angle) * mag
    u, v = y[..., a], y[..., b]
    out[..., a], out[..., b] = u * c - v * s, v * c + u * s
    room[..., a] = room[..., b] = 2.0 ** -19 * abs(mag) * (u.abs() + v.abs())
    return out, room


def check(got, want, dtype, what):
    ref, room = want
    g = got.detach().cpu().double()
    assert g.shape == ref.shape
    bound = room + U[dtype] * (ref.abs() + room) + TINY[dtype]
    bad = ~((g - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}; worst {(g - ref).abs().max():.3e}"


def rows(tokens, Hq, H, D, dtype, g, fused=False):
    x = (torch.randn(tokens, Hq + 2 * H, D, generator=g) * torch.exp2(torch.randint(-3, 4, (Hq + 2 * H, 1), generator=g).float())).to(dtype)
    parts = x.split((Hq, H, H), dim=1)
    if fused:
        dev = x.to(DEV).split((Hq, H, H), dim=1)
    else:
        parts = [p.contiguous() for p in parts]
        dev = [p.to(DEV) for p in parts]
    return parts, dev


CASES = [
    # tokens, Hq, Hkv, D, rotated, start, neighbours, norm, fused, dtype
    (1, 1, 1, 16, 16, 0, False, True, False, torch.bfloat16),
    (1, 32, 8, 128, 128, 0, False, True, False, torch.bfloat16),
    (7, 14, 2, 64, 64, 0, True, False, False, torch.float16),
    (33, 5, 1, 80, 32, 0, False, True, True, torch.float16),
    (5, 3, 3, 96, 96, 0, False, False, False, torch.bfloat16),
    (9, 7, 1, 96, 48, 48, True, True, False, torch.bfloat16),
    (13, 4, 4, 192, 64, 128, False, True, True, torch.bfloat16),
    (6, 6, 2, 192, 128, 8, True, False, False, torch.float16),
    (4, 8, 8, 256, 256, 0, False, True, False, torch.float16),
    (700, 9, 3, 128, 64, 24, False, True, True, torch.bfloat16),
    (1500, 24, 8, 128, 128, 0, True, True, False, torch.bfloat16),
    (3, 32, 8, 128, 0, 0, False, True, False, torch.bfloat16),   # norms alone
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_rotary_rows(case):
    n, Hq, H, D, rd, start, paired, norm, fused, dtype = case
    g = wl.generator(n * 31 + D)
    (q, k, _), (dq, dk, _) = rows(n, Hq, H, D, dtype, g, fused)
    pos = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32)
    f = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64) / max(rd // 2, 1))
    wq, wk = ((torch.randn(D, generator=g) * 0.3 + 1).to(dtype) if norm else None for _ in range(2))
    mag = 1.25 if start else 1.0
    before = (dq.clone(), dk.clone())
    out = pk.paged_rotary(dq, dk, pos.to(DEV), f.to(DEV), rotary_start=start, interleaved=paired, magnitude=mag,
                          query_weight=None if wq is None else wq.to(DEV), key_weight=None if wk is None else wk.to(DEV),
                          eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(dq, before[0]) and torch.equal(dk, before[1])
    for got, x, w, what in ((out[0], q, wq, "query"), (out[1], k, wk, "key")):
        check(got, plain(x, w, pos, f, start, paired, mag, 1e-5), dtype, what)


def test_angles_of_far_and_negative_positions():
    # frequencies of an exact binary fraction of a turn: the float64 product is exact at any position
    pos = torch.tensor([0, 1, -1, 4095, 10 ** 6 + 3, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    turns = torch.tensor([2.0 ** -3, 2.0 ** -9 * 3, 2.0 ** -20 * 77773, 2.0 ** -21, 2.0 ** -5 * 7, 2.0 ** -11, 2.0 ** -4, 2.0 ** -20],
                         dtype=torch.float64)
    f = turns * 2 * math.pi
    g = wl.generator(5)
    (q, k, _), (dq, dk, _) = rows(len(pos), 4, 2, 16, torch.float16, g)
    out = pk.paged_rotary(dq, dk, pos.to(DEV), f.to(DEV))
    y = q.double()
    a = torch.remainder(pos.double()[:, None] * turns, 1.0)[:, None] * 2 * math.pi
    u, v = y[..., :8], y[..., 8:]
    ref = torch.cat((u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()), -1)
    # 2 pi and its reciprocal, each rounded to 53 bits, leave the step off by 2^-52 of itself: at 2^31 positions of
    # steps up to 7 / 32 turns, 2^-52 * 2^31 * 2 pi / 4 < 2^-20 radians
    room = torch.cat((u.abs() + v.abs(),) * 2, -1) * (2.0 ** -19 + 2.0 ** -20)
    check(out[0], (ref, room), torch.float16, "query")


def test_in_place_and_positions_shared():
    g = wl.generator(6)
    (q, k, _), (dq, dk, _) = rows(50, 6, 2, 128, torch.bfloat16, g)
    pos = torch.randint(0, 9000, (50,), generator=g, dtype=torch.int32)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    a = pk.paged_rotary(dq, dk, pos.to(DEV), f.to(DEV))
    b = pk.paged_rotary(dq, dk, pos.to(DEV), f.to(DEV), query_out=dq, key_out=dk)
    assert b[0] is dq and b[1] is dk and torch.equal(a[0], dq) and torch.equal(a[1], dk)


def test_non_finite_rows_stay_apart():
    g = wl.generator(7)
    (q, k, _), (dq, dk, _) = rows(12, 4, 2, 128, torch.bfloat16, g)
    pos = torch.arange(12, dtype=torch.int32)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    w = torch.ones(128, dtype=torch.bfloat16)
    kw = dict(query_weight=w.to(DEV), key_weight=w.to(DEV))
    want = pk.paged_rotary(dq, dk, pos.to(DEV), f.to(DEV), **kw)
    dq[3, 1, 7], dq[5, 0, 100], dk[3, 1, 2] = math.nan, math.inf, -math.inf
    dq[6, 2] = 0
    got = pk.paged_rotary(dq, dk, pos.to(DEV), f.to(DEV), **kw)
    hit = torch.zeros(12, 4, dtype=torch.bool)
    hit[3, 1] = hit[5, 0] = hit[6, 2] = True
    assert torch.equal(got[0][~hit.to(DEV)], want[0][~hit.to(DEV)])
    assert got[0][3, 1].isnan().all() and got[0][5, 0].isnan().any() and (got[0][6, 2] == 0).all()
    assert torch.equal(got[1][:3], want[1][:3]) and torch.equal(got[1][4:], want[1][4:])


def append_case(lens, new, S, Hq, H, D, layout, dtype, seed, rd=None, start=0, paired=False, norm=True, fused=False,
                form="5d", mag=1.0):
    g = wl.generator(seed)
    pt = wl.reserve_pages(lens, S, g, extra=3)
    one = (S, H, D) if layout == wl.NHD else (H, S, D)
    pool = torch.randn((pt.num_pages, 2) + one, generator=g).to(dtype)
    n = sum(new)
    parts, dev = rows(n, Hq, H, D, dtype, g, fused)
    bi = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(torch.int32)
    pos = torch.cat([torch.arange(L - m, L) for L, m in zip(lens, new)]).to(torch.int32)
    rd = D if rd is None else rd
    f = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64) / max(1, rd // 2))
    ws = tuple((torch.randn(D, generator=g) * 0.3 + 1).to(dtype) if norm else None for _ in range(2))
    indices = torch.tensor([p for r in pt.pages for p in r], dtype=torch.int32)
    indptr = torch.tensor([0] + [len(r) for r in pt.pages]).cumsum(0).to(torch.int32)
    last = torch.tensor([L - (len(r) - 1) * S if r else 0 for L, r in zip(lens, pt.pages)], dtype=torch.int32)
    return dict(parts=parts, dev=dev, bi=bi, pos=pos, f=f, ws=ws, pool=pool, idx=indices, ptr=indptr, last=last, S=S,
                layout=layout, dtype=dtype, start=start, paired=paired, mag=mag, form=form, H=H)


def run_append(c, bi=None, pos=None, rot=None, idx=None, **kw):
    pool = c["pool"].to(DEV)
    kv = pool if c["form"] == "5d" else (pool[:, 0].contiguous(), pool[:, 1].contiguous())
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = pk.paged_append_rotary(*c["dev"], (c["bi"] if bi is None else bi).to(DEV), (c["pos"] if pos is None else pos).to(DEV),
                               kv, (c["idx"] if idx is None else idx).to(DEV), c["ptr"].to(DEV), c["last"].to(DEV),
                               c["f"].to(DEV), kv_layout=c["layout"], rotary_start=c["start"], interleaved=c["paired"],
                               magnitude=c["mag"], query_weight=None if c["ws"][0] is None else c["ws"][0].to(DEV),
                               key_weight=None if c["ws"][1] is None else c["ws"][1].to(DEV), eps=1e-6,
                               rotary_positions=rot, err_word=err, **kw)
    torch.cuda.synchronize()
    after = pool if c["form"] == "5d" else torch.stack(kv, 1)
    return q, after.cpu(), int(err.item())


def check_append(c, q, after, skip=(), rot=None):
    pos = c["pos"] if rot is None else rot
    args = (pos, c["f"], c["start"], c["paired"], c["mag"], 1e-6)
    check(q, plain(c["parts"][0], c["ws"][0], *args), c["dtype"], "query")
    want, room = plain(c["parts"][1], c["ws"][1], *args)
    left = c["pool"].clone()
    S = c["S"]
    for i in range(len(c["bi"])):
        if i in skip:
            continue
        p = int(c["pos"][i])
        page, s = int(c["idx"][int(c["ptr"][int(c["bi"][i])]) + p // S]), p % S
        for z in range(2):
            spot = after[page, z, s] if c["layout"] == wl.NHD else after[page, z, :, s]
            old = left[page, z, s] if c["layout"] == wl.NHD else left[page, z, :, s]
            if z == 0:
                check(spot, (want[i], room[i]), c["dtype"], f"key {i}")
            else:
                assert torch.equal(spot, c["parts"][2][i])
            old.copy_(spot)
    assert torch.equal(left.view(torch.int16), after.view(torch.int16))  # nothing else changed


APPENDS = [
    dict(lens=[1], new=[1], S=16, Hq=1, H=1, D=128, layout=wl.HND, dtype=torch.bfloat16, norm=False),
    dict(lens=[5, 40, 17, 64], new=[1, 1, 1, 1], S=16, Hq=32, H=8, D=128, layout=wl.HND, dtype=torch.bfloat16),
    dict(lens=[130, 3, 77], new=[97, 3, 31], S=32, Hq=12, H=4, D=128, layout=wl.NHD, dtype=torch.float16, paired=True, rd=64, start=32),
    dict(lens=[70, 300], new=[70, 211], S=64, Hq=7, H=1, D=64, layout=wl.NHD, dtype=torch.bfloat16, fused=True, form="tuple"),
    dict(lens=[33, 90], new=[33, 5], S=8, Hq=4, H=2, D=192, layout=wl.HND, dtype=torch.bfloat16, rd=64, start=128, fused=True, mag=1.2),
    dict(lens=[20, 0, 9], new=[20, 0, 9], S=1, Hq=3, H=3, D=80, layout=wl.HND, dtype=torch.float16, rd=32),
    dict(lens=[900, 1200], new=[900, 1100], S=128, Hq=5, H=1, D=256, layout=wl.NHD, dtype=torch.float16, paired=True),
]


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append_rotary(i):
    c = append_case(seed=40 + i, **APPENDS[i])
    q, after, err = run_append(c)
    assert err == 0
    check_append(c, q, after)


def test_rotation_by_other_positions():
    c = append_case([50, 20], [50, 4], 16, 4, 2, 128, wl.NHD, torch.bfloat16, 60)
    rot = c["pos"] * 3 + 100000
    q, after, err = run_append(c, rot=rot.to(DEV))
    assert err == 0
    check_append(c, q, after, rot=rot)


def test_without_rotation_it_is_the_append():
    c = append_case([50, 20], [50, 4], 16, 4, 2, 128, wl.HND, torch.bfloat16, 61, rd=0, norm=False)
    q, after, err = run_append(c)
    pool = c["pool"].to(DEV)
    pk.paged_append(c["dev"][1], c["dev"][2], c["bi"].to(DEV), c["pos"].to(DEV), pool, c["idx"].to(DEV), c["ptr"].to(DEV),
                    c["last"].to(DEV), kv_layout=wl.HND)
    assert err == 0 and torch.equal(after, pool.cpu()) and torch.equal(q, c["dev"][0])


def test_entries_without_a_place_are_skipped():
    c = append_case([40, 33, 16], [8, 8, 8], 16, 4, 2, 128, wl.NHD, torch.bfloat16, 62)
    bi, pos, idx = c["bi"].clone(), c["pos"].clone(), c["idx"].clone()
    bi[1], bi[2] = -1, 3
    pos[9], pos[10] = 33, -4
    idx[int(c["ptr"][2])] = c["pool"].shape[0]  # the third request's only page
    q, after, err = run_append(c, bi=bi, pos=pos, rot=c["pos"].to(DEV), idx=idx)
    assert err == BATCH | POS | PAGE
    check_append(c, q, after, skip={1, 2, 9, 10} | set(range(16, 24)))


def test_offsets_past_32_bits():
    # a pool whose last pages lie more than 2^32 elements in
    S, H, D = 256, 8, 128
    pages = (1 << 32) // (2 * S * H * D) + 3
    pool = torch.empty(pages, 2, H, S, D, dtype=torch.float16, device=DEV)
    ids = [pages - 1, 0, pages - 2]
    pool[ids] = 0
    g = wl.generator(63)
    parts, dev = rows(3, 8, H, D, torch.float16, g)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    i32 = dict(dtype=torch.int32, device=DEV)
    pos = torch.tensor([255, 0, 100], **i32)
    pk.paged_append_rotary(*dev, torch.arange(3, **i32), pos, pool, torch.tensor(ids, **i32), torch.arange(4, **i32),
                           torch.full((3,), 256, **i32), f.to(DEV), kv_layout=wl.HND)
    torch.cuda.synchronize()
    want, room = plain(parts[1], None, pos.cpu(), f, 0, False, 1.0, 0.0)
    for i, (page, s) in enumerate(zip(ids, (255, 0, 100))):
        check(pool[page, 0, :, s], (want[i], room[i]), torch.float16, "key")
        assert torch.equal(pool[page, 1, :, s].cpu(), parts[2][i])
        assert pool[page, 0].count_nonzero() <= H * D


def test_no_tokens():
    q = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    i = torch.empty(0, dtype=torch.int32, device=DEV)
    f = torch.ones(64, dtype=torch.float64, device=DEV)
    a, b = pk.paged_rotary(q, k, i, f)
    assert a.shape == q.shape and b.shape == k.shape


def test_graph_replays_follow_the_inputs():
    c = append_case([50, 20], [50, 4], 16, 4, 2, 128, wl.NHD, torch.bfloat16, 64)
    pool = c["pool"].to(DEV)
    dev = [x.clone() for x in c["dev"]]
    tens = [c[n].to(DEV) for n in ("bi", "pos")] + [pool] + [c[n].to(DEV) for n in ("idx", "ptr", "last", "f")]
    out = torch.empty_like(dev[0])
    call = lambda: pk.paged_append_rotary(*dev, *tens, kv_layout=wl.NHD, query_out=out)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x in dev:
        x.mul_(0.5)
    graph.replay()
    got, got_pool = out.clone(), pool.clone()
    call()
    assert torch.equal(got, out) and torch.equal(got_pool, pool)
