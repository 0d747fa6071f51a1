"""Prefill under a window with first tokens, and over E4M3 caches with block
scales, against the definition in 64 bits; and the operators of a long
session run one after another."""
from __future__ import annotations

import math

import pytest
import torch

import _plain
import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
QLEN, PAGE, SCALE = 8, 1, 128


def make(ql, kvl, S, Hq, H, d, layout, dtype, seed, window=-1, first=0, causal=True, G=None, poison=True):
    """Rows that no query of a request sees hold NaN, and pages of only such
    rows have a table entry outside the pool."""
    g = wl.generator(seed)
    pt = wl.reserve_pages(kvl, S, g, extra=2)

    def pool(w):
        x = torch.randn((pt.num_pages,) + ((S, H, w) if layout == wl.NHD else (H, S, w)), generator=g)
        return (x * 112).clamp(-448, 448).to(torch.float8_e4m3fn) if G else x.to(dtype)

    k, v = pool(d), pool(128)
    scales = torch.exp2(torch.randint(-9, -5, (pt.num_pages, 2, H, S // G), generator=g).float()) if G else None
    q = torch.randn(sum(ql), Hq, d, generator=g).to(dtype)
    table, used = pt.block_tables(max(1, pt.max_pages()) + 1), []
    for b, (n, L) in enumerate(zip(ql, kvl)):
        j, p = torch.arange(L), torch.arange(L - n, L)
        u = _plain.visible(j, p, window, first)
        if not causal:
            u |= j[None, :] > p[:, None]
        u = u.any(0)
        used.append(u)
        if poison and n:
            for t in (k, v):
                raw, bad = (t.view(torch.uint8), 0x7F) if G else (t, float("nan"))
                for i in torch.nonzero(~u).flatten().tolist():
                    pg, s = pt.pages[b][i // S], i % S
                    if layout == wl.NHD:
                        raw[pg, s] = bad
                    else:
                        raw[pg, :, s] = bad
            for i in range(len(pt.pages[b])):
                if not u[i * S:(i + 1) * S].any():
                    table[b, i] = wl.POISON
    return dict(pt=pt, k=k, v=v, scales=scales, q=q, table=table, ql=ql, kvl=kvl, S=S, H=H, Hq=Hq, d=d, layout=layout,
                dtype=dtype, window=window, first=first, causal=causal, used=used)


def call(c, scale, err=None, **kw):
    B, mq, mk = len(c["ql"]), max(c["ql"]), max(c["kvl"])
    n = pk.paged_prefill_scaled_workspace_size(B, c["Hq"], c["H"], mq, mk, c["d"], 128) if c["scales"] is not None else \
        pk.paged_prefill_workspace_size(B, c["Hq"], mq, mk)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # (what it holds before the call has no effect)
    out, lse = pk.paged_prefill(c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), scale, ws, mq, mk,
                                torch.tensor(c["ql"], dtype=torch.int32, device=DEV),
                                torch.tensor(c["kvl"], dtype=torch.int32, device=DEV), c["table"].to(DEV),
                                causal=c["causal"], kv_layout=c["layout"], err_word=err, window_left=c["window"],
                                first_tokens=c["first"], kv_scales=None if c["scales"] is None else c["scales"].to(DEV),
                                **kw)
    torch.cuda.synchronize()
    return out, lse


def compare(c, out, lse, scale, skip=()):
    row = 0
    for b, (n, L) in enumerate(zip(c["ql"], c["kvl"])):
        if n and b not in skip:
            kv = []
            for z, pool in enumerate((c["k"], c["v"])):
                x = _plain.tokens(pool.double(), c["pt"].pages[b], L, c["S"], c["layout"], c["used"][b])
                if c["scales"] is not None:
                    x = x * _plain.token_scales(c["scales"][:, z], c["pt"].pages[b], L, c["S"], c["used"][b])
                kv.append(x)
            ro, rl, bo, bl = _plain.attention(c["q"][row:row + n].double(), *kv, L, scale, c["window"], c["first"],
                                              causal=c["causal"], u_p=U[c["dtype"]], u_out=U[c["dtype"]])
            _plain.check(out[row:row + n], ro, bo, f"out of request {b}")
            _plain.check(lse[row:row + n], rl, bl, f"lse of request {b}")
        row += n


WINDOW = [
    # q lens, kv lens, page, Hq, H, d, layout, dtype, window, first, causal
    ([130, 7, 300, 1], [900, 7, 300, 1049], 16, 8, 2, 128, wl.HND, torch.bfloat16, 100, 4, True),
    ([200, 129], [1200, 129], 32, 4, 4, 192, wl.NHD, torch.float16, 95, 1, True),
    ([257, 33], [1300, 600], 8, 6, 2, 128, wl.NHD, torch.bfloat16, 0, 9, True),          # a window of one key
    ([129], [1025], 256, 3, 1, 128, wl.HND, torch.float16, 300, 129, True),              # odd group, big pages
    ([128, 128], [1000, 260], 64, 2, 1, 192, wl.HND, torch.bfloat16, 191, 97, True),
    ([64, 1], [400, 1500], 16, 8, 1, 128, wl.HND, torch.bfloat16, 255, 250, True),       # first tokens near the window
    ([300, 20], [1100, 700], 16, 4, 2, 128, wl.NHD, torch.bfloat16, 130, 0, True),       # no first tokens
    ([100, 50], [800, 50], 32, 4, 2, 128, wl.HND, torch.bfloat16, 200, 5, False),        # keys after the query too
    ([300], [300], 16, 4, 2, 128, wl.HND, torch.float16, 5000, 3, True),                 # longer than the request
    ([40, 0, 70], [30, 20, 600], 16, 4, 2, 128, wl.HND, torch.bfloat16, 60, 2, True),    # more queries than keys
    ([260], [900], 8, 4, 2, 128, wl.HND, torch.bfloat16, 333, 13, True),                 # small boxes, a tile of both parts
    ([130, 257], [2000, 777], 16, 2, 1, 192, wl.NHD, torch.float16, 250, 100, True),     # first tokens end inside a tile
    ([300], [1500], 128, 2, 2, 128, wl.NHD, torch.bfloat16, 129, 127, True),             # first tokens end a key early
    ([150], [700], 64, 4, 1, 192, wl.HND, torch.bfloat16, 40, 200, False),
]


@pytest.mark.parametrize("case", WINDOW, ids=[f"w{i}" for i in range(len(WINDOW))])
def test_window_with_first_tokens(case):
    ql, kvl, S, Hq, H, d, layout, dtype, window, first, causal = case
    c = make(ql, kvl, S, Hq, H, d, layout, dtype, sum(ql) + window, window, first, causal)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 1 / math.sqrt(d), err)
    assert int(err.item()) == (QLEN if any(a > b for a, b in zip(ql, kvl)) else 0)
    compare(c, out, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("scale", [-0.05, 0.0, 2.0])
def test_window_scales(scale):
    c = make([140], [500], 16, 2, 1, 128, wl.HND, torch.bfloat16, 3, 120, 6)
    compare(c, *call(c, scale), scale)


SCALED = [
    # q lens, kv lens, page, block, Hq, H, d, layout, dtype, window, first, causal
    ([130, 7, 300, 1], [400, 7, 300, 1049], 16, 16, 8, 2, 128, wl.HND, torch.bfloat16, -1, 0, True),
    ([200, 129], [900, 129], 32, 8, 4, 4, 192, wl.NHD, torch.float16, -1, 0, True),
    ([100, 50], [800, 50], 64, 32, 6, 2, 128, wl.NHD, torch.bfloat16, -1, 0, False),
    ([129, 40], [1025, 1200], 256, 128, 3, 1, 128, wl.HND, torch.float16, 150, 70, True),
    ([257, 33], [1300, 600], 8, 8, 6, 2, 192, wl.HND, torch.bfloat16, 99, 5, True),
    ([200], [1111], 16, 16, 4, 2, 128, wl.NHD, torch.float16, 333, 77, True),
]


@pytest.mark.parametrize("case", SCALED, ids=[f"s{i}" for i in range(len(SCALED))])
def test_block_scales(case):
    ql, kvl, S, G, Hq, H, d, layout, dtype, window, first, causal = case
    c = make(ql, kvl, S, Hq, H, d, layout, dtype, sum(ql) + G, window, first, causal, G)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.05, err)
    assert int(err.item()) == 0
    compare(c, out, lse, 0.05)


def test_contiguous_keys_and_batch_offsets():
    ql, kvl, window, first = [130, 9, 200], [600, 500, 200], 120, 10
    c = make(ql, kvl, 16, 4, 2, 128, wl.NHD, torch.bfloat16, 5, window, first, poison=False)
    k, v = (torch.cat([_plain.tokens(t, c["pt"].pages[b], L, 16, wl.NHD) for b, L in enumerate(kvl)]) for t in (c["k"], c["v"]))
    ws = torch.empty(pk.paged_prefill_workspace_size(3, 4, 200, 600), dtype=torch.uint8, device=DEV)
    lens = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (ql, kvl)]
    a = pk.paged_prefill(c["q"].to(DEV), k.to(DEV), v.to(DEV), 0.05, ws, 200, 600, *lens, None, window_left=window,
                         first_tokens=first)
    compare(c, *a, 0.05)
    # queries and outputs 5 rows apart
    off = torch.tensor([0, 135, 149], dtype=torch.int32, device=DEV)
    rows = torch.cat([torch.arange(o, o + n) for o, n in zip(off.tolist(), ql)])
    q = torch.full((360, 4, 128), float("nan"), dtype=torch.bfloat16)
    q[rows] = c["q"]
    out = torch.full((360, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((360, 4), 7.0, device=DEV)
    pk.paged_prefill(q.to(DEV), c["k"].to(DEV), c["v"].to(DEV), 0.05, ws, 200, 600, *lens, c["table"].to(DEV),
                     kv_layout="NHD", window_left=window, first_tokens=first, batch_offsets_q=off, batch_offsets_o=off,
                     out=out, lse=lse)
    compare(c, out[rows], lse[rows], 0.05)
    rest = torch.ones(360, dtype=torch.bool)
    rest[rows] = False
    assert (out.cpu()[rest] == 7).all() and (lse.cpu()[rest] == 7).all()


def test_bad_page_and_scale_are_flagged():
    c = make([20, 30], [100, 90], 16, 4, 2, 128, wl.HND, torch.bfloat16, 6, G=16)
    c["table"][0, 3] = -7
    c["scales"][c["pt"].pages[1][2], 0, 1, 0] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    call(c, 0.05, err)
    assert int(err.item()) == PAGE | SCALE
    c = make([20, 30], [100, 90], 16, 4, 2, 128, wl.HND, torch.bfloat16, 6, 40, 3)
    c["table"][0, 5] = 1 << 20
    err.zero_()
    out, lse = call(c, 0.05, err)
    assert int(err.item()) == PAGE
    compare(c, out, lse, 0.05, skip=(0,))


def test_graph_replay_and_another_stream():
    c = make([140, 30], [500, 700], 16, 8, 2, 128, wl.HND, torch.bfloat16, 7, 120, 6, G=16)
    q, k, v, sc, table = (c[n].to(DEV) for n in ("q", "k", "v", "scales", "table"))
    lens = [torch.tensor(c[n], dtype=torch.int32, device=DEV) for n in ("ql", "kvl")]
    ws = torch.empty(pk.paged_prefill_scaled_workspace_size(2, 8, 2, 140, 700, 128, 128), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)

    def step():
        pk.paged_prefill(q, k, v, 0.05, ws, 140, 700, *lens, table, kv_layout="HND", window_left=120, first_tokens=6,
                         kv_scales=sc, out=out, lse=lse)

    step()
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    compare(c, *want, 0.05)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for _ in range(2):
        out.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_refusals():
    c = make([20], [100], 16, 4, 2, 128, wl.HND, torch.bfloat16, 8, G=16)
    e4 = torch.float8_e4m3fn
    for o in (dict(scales=c["scales"].repeat(1, 1, 1, 4)), dict(scales=c["scales"][:-1]), dict(k=c["k"].to(torch.bfloat16)),
              dict(q=c["q"].to(e4)), dict(q=c["q"].half(), k=c["k"].half(), v=c["v"].half()), dict(first=-1), dict(window=-2)):
        with pytest.raises(pk.PagedKVError):
            call(dict(c, **o), 0.05)
    with pytest.raises(pk.PagedKVError):  # E4M3 caches without block scales under a window
        call(dict(c, scales=None, window=10), 0.05)
    with pytest.raises(pk.PagedKVError):
        call(c, 0.05, k_scale=torch.ones(1, device=DEV))
    with pytest.raises(pk.PagedKVError):
        call(c, 0.05, o_data_type=torch.float16)


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_long_session(layout):
    """Prompts appended to a scaled cache and attended over, then tokens one
    at a time, under a window with first tokens; each step's attention against
    the values that the cache then stands for."""
    lay = wl.HND if layout == "HND" else wl.NHD
    S, G, H, Hq, window, first = 16, 16, 2, 8, 60, 5
    g = wl.generator(77)
    prompts, steps = [150, 9], 4
    pt = wl.reserve_pages([n + steps for n in prompts], S, g)
    one = (S, H, 128) if lay == wl.NHD else (H, S, 128)
    cache = torch.zeros((pt.num_pages, 2) + one, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.ones(pt.num_pages, 2, H, S // G, device=DEV)
    table = pt.block_tables().to(DEV)
    lens, scale = [0, 0], 1 / math.sqrt(128)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pages = [torch.tensor(p, dtype=torch.int32) for p in pt.pages]
    kv_indptr = torch.tensor([0, len(pages[0]), len(pages[0]) + len(pages[1])], dtype=torch.int32)
    for step in range(1 + steps):
        new = prompts if step == 0 else [1, 1]
        lens = [a + b for a, b in zip(lens, new)]
        rows = sum(new)
        k, v = (torch.randn(rows, H, 128, generator=g) * 2.0 ** step for _ in range(2))
        q = torch.randn(rows, Hq, 128, generator=g).to(torch.bfloat16)
        # the helpers derive the entries from the lengths so far
        used = [-(-n // S) for n in lens]
        ptr = torch.tensor([0, used[0], sum(used)], dtype=torch.int32)
        idx = torch.cat([p[:n] for p, n in zip(pages, used)])
        last = torch.tensor([n - (u - 1) * S for n, u in zip(lens, used)], dtype=torch.int32)
        ptr, idx, last = ptr.to(DEV), idx.to(DEV), last.to(DEV)
        seq = pk.paged_seq_lens(ptr, last, S)
        bi, pos = pk.paged_batch_indices_positions(torch.tensor([0, new[0], rows], dtype=torch.int32, device=DEV), seq, rows)
        pk.paged_append_scaled(k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), bi, pos, cache, scales, idx,
                               ptr, last, kv_layout=layout, err_word=err)
        if step == 0:
            ws = torch.empty(pk.paged_prefill_scaled_workspace_size(2, Hq, H, max(new), max(lens), 128, 128),
                             dtype=torch.uint8, device=DEV)
            out, lse = pk.paged_prefill(q.to(DEV), cache[:, 0], cache[:, 1], scale, ws, max(new), max(lens),
                                        torch.tensor(new, dtype=torch.int32, device=DEV), seq, table, kv_layout=layout,
                                        window_left=window, first_tokens=first, kv_scales=scales, err_word=err)
        else:
            n = pk.paged_decode_workspace_size(2, 1, Hq, H, 128, max(lens), S, window, first_tokens=first)
            ws = torch.empty(max(1, n), dtype=torch.uint8, device=DEV)
            lse = torch.empty(rows, Hq, device=DEV)
            out = pk.paged_decode(q.to(DEV), cache, ws, table, seq, max(lens), bmm1_scale=scale, window_left=window,
                                  first_tokens=first, kv_scales=scales, kv_layout=layout, lse=lse, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        row = 0
        at = [0, new[0]]
        for b, (n, L) in enumerate(zip(new, lens)):
            kv = []
            for z, src in enumerate((k, v)):
                x = _plain.tokens(cache[:, z].cpu().double(), pt.pages[b], L, S, lay) * \
                    _plain.token_scales(scales[:, z].cpu(), pt.pages[b], L, S)
                kv.append(x)
                # the newest token's values came through within half a step of E4M3 (2^-4) or its smallest step
                want = src[at[b] + n - 1].to(torch.bfloat16).double()
                s = _plain.token_scales(scales[:, z].cpu(), pt.pages[b], L, S)[-1]
                assert ((x[-1] - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * s).all()
            u_p = 2.0 ** -8 if step == 0 else 2.0 ** -11
            ro, rl, bo, bl = _plain.attention(q[row:row + n].double(), *kv, L, scale, window, first, u_p=u_p)
            _plain.check(out[row:row + n], ro, bo, f"step {step} out of request {b}")
            _plain.check(lse[row:row + n], rl, bl, f"step {step} lse of request {b}")
            row += n
