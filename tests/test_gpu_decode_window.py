"""Decode under a window with first tokens, and over an E4M3 cache with block
scales, against the definition in 64 bits."""
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


def make(lens, S, Hq, H, layout, dtype, seed, q=1, q_lens=None, G=None, scaled=False, e4m3=False, sinks=False,
         scale_exp=(-9, -5), form="5d", window=-1, first=0, poison=True):
    """Pages of keys that no query sees get a table entry outside the pool and
    rows that no query sees hold NaN."""
    g = wl.generator(seed)
    pt = wl.reserve_pages(lens, S, g, extra=2)
    one = (S, H, 128) if layout == wl.NHD else (H, S, 128)
    e4m3 = e4m3 or scaled
    if e4m3:
        std = 112.0 if scaled else 1.0
        pool = (torch.randn((pt.num_pages, 2) + one, generator=g) * std).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        pool = torch.randn((pt.num_pages, 2) + one, generator=g).to(dtype)
    scales = None
    if scaled:
        scales = torch.exp2(torch.randint(scale_exp[0], scale_exp[1] + 1, (pt.num_pages, 2, H, S // (G or S)),
                                          generator=g).float())
    ql = [q] * len(lens) if q_lens is None else q_lens
    query = torch.randn(sum(ql), Hq, 128, generator=g).to(dtype)
    table = pt.block_tables(max(1, pt.max_pages()) + 1)
    sk = torch.randn(Hq, generator=g) if sinks else None
    used = []
    for b, (L, n) in enumerate(zip(lens, ql)):
        j = torch.arange(L)
        p = torch.arange(L - n, L)
        u = _plain.visible(j, p, window, first).any(0)
        used.append(u)
        if poison and n:
            raw = pool.view(torch.uint8) if e4m3 else pool
            bad = 0x7F if e4m3 else float("nan")
            for t in torch.nonzero(~u).flatten().tolist():
                pg, s = pt.pages[b][t // S], t % S
                if layout == wl.NHD:
                    raw[pg, :, s] = bad
                else:
                    raw[pg, :, :, s] = bad
            for i in range(len(pt.pages[b])):
                if not u[i * S:(i + 1) * S].any():
                    table[b, i] = wl.POISON
    return dict(pt=pt, pool=pool, scales=scales, query=query, table=table, lens=lens, ql=ql, S=S, H=H, Hq=Hq,
                layout=layout, dtype=dtype, sinks=sk, varlen=q_lens is not None, window=window, first=first,
                used=used, form=form)


def call(c, bmm1, bmm2=1.0, err=None, ws=None, **kw):
    maxq = max(c["ql"])
    L = max(c["lens"])
    n = pk.paged_decode_workspace_size(len(c["lens"]), maxq, c["Hq"], c["H"], 128, L, c["S"], c["window"],
                                       first_tokens=c["first"])
    if ws is None:
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    pool, sc = c["pool"].to(DEV), None if c["scales"] is None else c["scales"].to(DEV)
    if c["form"] == "tuple":
        pool = (pool[:, 0].contiguous(), pool[:, 1].contiguous())
        sc = None if sc is None else (sc[:, 0].contiguous(), sc[:, 1].contiguous())
    lse = torch.empty(c["query"].shape[:2], dtype=torch.float32, device=DEV)
    if c["varlen"]:
        kw.update(cum_seq_lens_q=torch.tensor([0] + c["ql"]).cumsum(0).to(torch.int32).to(DEV), max_q_len=maxq)
    else:
        kw.update(q_len_per_req=maxq)
    out = pk.paged_decode(c["query"].to(DEV), pool, ws, c["table"].to(DEV),
                          torch.tensor(c["lens"], dtype=torch.int32, device=DEV), L, bmm1_scale=bmm1, bmm2_scale=bmm2,
                          window_left=c["window"], sinks=None if c["sinks"] is None else c["sinks"].to(DEV),
                          kv_layout=c["layout"], lse=lse, err_word=err, first_tokens=c["first"], kv_scales=sc, **kw)
    torch.cuda.synchronize()
    return out, lse


def compare(c, out, lse, bmm1, bmm2=1.0, skip=()):
    row = 0
    for b, (L, n) in enumerate(zip(c["lens"], c["ql"])):
        if n and b not in skip:
            kv = []
            for z in range(2):
                x = _plain.tokens(c["pool"][:, z].double(), c["pt"].pages[b], L, c["S"], c["layout"], c["used"][b])
                if c["scales"] is not None:
                    x = x * _plain.token_scales(c["scales"][:, z], c["pt"].pages[b], L, c["S"], c["used"][b])
                kv.append(x)
            u_p = 2.0 ** -11 if c["pool"].dtype == torch.float8_e4m3fn else U[c["dtype"]]
            ro, rl, bo, bl = _plain.attention(c["query"][row:row + n].double(), *kv, L, bmm1, c["window"], c["first"],
                                              c["sinks"], u_p=u_p, u_out=U[c["dtype"]], bmm2=bmm2)
            _plain.check(out[row:row + n], ro, bo, f"out of request {b}")
            _plain.check(lse[row:row + n], rl, bl, f"lse of request {b}")
        row += n


WINDOW = [
    # lens, page, Hq, H, layout, dtype, q, window, first, sinks, e4m3
    ([1, 2, 63, 64, 65, 200], 16, 32, 8, wl.HND, torch.bfloat16, 1, 20, 4, False, False),
    ([700, 130, 129], 8, 8, 8, wl.NHD, torch.float16, 1, 100, 1, True, False),
    ([1000, 500, 300], 64, 16, 2, wl.HND, torch.bfloat16, 2, 63, 65, False, False),    # first tokens cross a tile
    ([1500, 257, 256], 256, 32, 4, wl.NHD, torch.float16, 4, 200, 130, True, False),   # 32 rows, one page holds both
    ([900, 40], 32, 64, 4, wl.HND, torch.bfloat16, 4, 0, 7, False, False),             # 64 rows, a window of one key
    ([170, 110, 111, 175], 8, 4, 1, wl.HND, torch.bfloat16, 1, 70, 100, False, False),  # first tokens reach the window's tile
    ([5000, 9000, 300], 16, 6, 2, wl.NHD, torch.bfloat16, 1, 2500, 700, True, False),  # several splits
    ([700, 131, 64], 16, 32, 8, wl.HND, torch.bfloat16, 1, 90, 10, True, True),        # E4M3 without block scales
    ([900, 300], 32, 32, 2, wl.NHD, torch.float16, 1, 150, 33, False, True),
    ([300, 20], 16, 8, 1, wl.HND, torch.float16, 1, -1, 9, False, False),              # no window: no effect
    ([300, 20], 16, 8, 1, wl.HND, torch.float16, 3, 100000, 1 << 30, False, False),    # everything visible
]


@pytest.mark.parametrize("case", WINDOW, ids=[f"w{i}" for i in range(len(WINDOW))])
def test_window_with_first_tokens(case):
    lens, S, Hq, H, layout, dtype, q, window, first, sinks, e4m3 = case
    c = make(lens, S, Hq, H, layout, dtype, len(lens) + S + window, q=q, sinks=sinks, e4m3=e4m3, window=window, first=first)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    bmm1 = 1 / math.sqrt(128)
    out, lse = call(c, bmm1, 0.75, err)
    assert int(err.item()) == (QLEN if min(lens) < q else 0)
    compare(c, out, lse, bmm1, 0.75)


SCALED = [
    # lens, page, block, Hq, H, layout, dtype, q, window, first, sinks, form
    ([1, 2, 63, 64, 65, 200], 16, 16, 32, 8, wl.HND, torch.bfloat16, 1, -1, 0, False, "5d"),
    ([45, 8, 25, 22], 8, 8, 8, 8, wl.NHD, torch.float16, 1, -1, 0, True, "tuple"),
    ([700, 1111], 32, 8, 8, 1, wl.HND, torch.bfloat16, 1, -1, 0, False, "5d"),
    ([1500, 70], 256, 64, 16, 1, wl.NHD, torch.bfloat16, 1, -1, 0, True, "5d"),        # 16 rows
    ([333, 1000], 64, 32, 40, 8, wl.HND, torch.float16, 4, -1, 0, False, "tuple"),     # 20 rows
    ([600, 129], 128, 128, 32, 2, wl.HND, torch.bfloat16, 4, 100, 5, True, "5d"),      # 64 rows, window
    ([3000, 12000, 5], 16, 16, 8, 2, wl.NHD, torch.bfloat16, 1, -1, 0, True, "5d"),    # several splits
    ([5000, 9000], 8, 8, 7, 1, wl.HND, torch.float16, 1, 4000, 300, False, "5d"),      # splits, window, first tokens
    ([900, 2000, 40], 64, 16, 16, 2, wl.NHD, torch.float16, 2, 300, 70, True, "5d"),
    ([1300, 64, 2500], 16, 16, 24, 8, wl.HND, torch.bfloat16, 3, -1, 0, False, "5d"),  # 9 rows
    ([777, 1500], 32, 16, 8, 1, wl.NHD, torch.bfloat16, 4, 500, 40, True, "5d"),       # 32 rows
    ([900, 100], 16, 8, 17, 1, wl.HND, torch.float16, 1, -1, 0, False, "5d"),          # 17 rows
    ([900, 100], 16, 8, 33, 1, wl.HND, torch.float16, 1, 200, 3, False, "5d"),         # 33 rows
]


@pytest.mark.parametrize("case", SCALED, ids=[f"s{i}" for i in range(len(SCALED))])
def test_block_scales(case):
    lens, S, G, Hq, H, layout, dtype, q, window, first, sinks, form = case
    c = make(lens, S, Hq, H, layout, dtype, len(lens) + S + G, q=q, sinks=sinks, scaled=True, G=G, window=window,
             first=first, form=form)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.05, 1.0, err)
    assert int(err.item()) == (QLEN if min(lens) < q else 0)
    compare(c, out, lse, 0.05)


@pytest.mark.parametrize("Hq", [8, 16])  # swapped and plain operands
def test_scales_of_very_different_sizes(Hq):
    # V blocks 2^60 apart, K blocks 2^20 apart, scales that are no powers of two
    c = make([400, 77], 16, Hq, 1, wl.HND, torch.bfloat16, 31, scaled=True, G=8)
    g = wl.generator(5)
    c["scales"][:, 1] = torch.exp2(torch.randint(-30, 31, c["scales"][:, 1].shape, generator=g).float()) * 1.3
    c["scales"][:, 0] = torch.exp2(torch.randint(-20, -3, c["scales"][:, 0].shape, generator=g).float()) * 0.9
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.02, 1.0, err)
    assert int(err.item()) == 0
    compare(c, out, lse, 0.02)


def test_scale_out_of_range_is_flagged_and_clamped():
    c = make([100], 16, 8, 2, wl.HND, torch.bfloat16, 32, scaled=True, G=16)
    pages = c["pt"].pages[0]
    c["scales"][pages[0], 0, 0, 0] = 0.0
    c["scales"][pages[1], 0, 1, 0] = float("nan")
    c["scales"][pages[2], 1, 0, 0] = -1.0
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.05, 1.0, err)
    assert int(err.item()) == SCALE
    for p, z, h in ((0, 0, 0), (1, 0, 1), (2, 1, 0)):
        c["scales"][pages[p], z, h, 0] = 2.0 ** -48
    compare(c, out, lse, 0.05)


def test_bad_page_is_flagged_and_its_keys_absent():
    c = make([100, 50], 16, 8, 2, wl.NHD, torch.bfloat16, 33, scaled=True, G=8)
    c["table"][0, 2] = -5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.05, 1.0, err)
    assert int(err.item()) == PAGE
    compare(c, out, lse, 0.05, skip=(0,))
    # request 0 without keys 32 .. 47: the same as the 84 other keys in order
    d = dict(c, lens=[84, 50], used=[torch.ones(84, dtype=torch.bool), c["used"][1]])
    pool, sc = c["pool"].clone(), c["scales"].clone()
    pages = [p for i, p in enumerate(c["pt"].pages[0]) if i != 2]
    d["pt"] = wl.PageTable([84, 50], 16, c["pt"].num_pages, [pages, c["pt"].pages[1]])
    d["pool"], d["scales"] = pool, sc
    compare(d, out, lse, 0.05, skip=(1,))


@pytest.mark.parametrize("scaled", [False, True])
def test_variable_length_queries(scaled):
    c = make([700, 3, 40, 1300], 16, 16, 4, wl.HND, torch.bfloat16, 34, q_lens=[2, 3, 0, 4], scaled=scaled, G=16,
             sinks=True, window=250, first=20)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.05, 1.0, err)
    assert int(err.item()) == 0
    compare(c, out, lse, 0.05)


def test_device_scales_and_dependent_launch_give_the_same_bits():
    c = make([700, 3000], 16, 16, 4, wl.HND, torch.bfloat16, 35, scaled=True, G=16, sinks=True, window=2000, first=64)
    a = call(c, 0.05, 0.7)
    b = call(c, torch.tensor([0.05], device=DEV), torch.tensor([0.7], device=DEV), enable_pdl=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_unit_scales_agree_with_the_plain_e4m3_decode():
    c = make([45, 700], 16, 8, 2, wl.HND, torch.bfloat16, 36, e4m3=True)
    compare(c, *call(c, 0.05), 0.05)
    c["scales"] = torch.ones(c["pt"].num_pages, 2, 2, 2)
    compare(c, *call(c, 0.05), 0.05)


@pytest.mark.parametrize("B, lens", [(1, [40000]), (3, [20000, 1, 9000]), (200, None)])
def test_runs_that_span_many_pieces(B, lens):
    """One long run over all CTAs; and more requests than threads, many empty."""
    g = wl.generator(B)
    if lens is None:
        lens = [0 if i % 3 == 0 else int(x) for i, x in enumerate(torch.randint(0, 900, (B,), generator=g))]
    c = make(lens, 16, 4, 1, wl.HND, torch.bfloat16, B, scaled=True, G=16, sinks=True)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.1, 1.0, err)
    assert int(err.item()) == (QLEN if 0 in lens else 0)
    compare(c, out, lse, 0.1)


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("L", [100, 3000])  # one CTA, and parts that are joined
def test_nan_and_infinity_among_the_visible_keys(scaled, L):
    """A visible NaN makes its rows NaN, as the formula does; other heads and requests stay clean."""
    c = make([L, L], 16, 8, 2, wl.HND, torch.bfloat16, 39, scaled=scaled, G=16, poison=False, window=None or -1)
    page = c["pt"].pages[0][3]
    raw = c["pool"].view(torch.uint8) if scaled else c["pool"]
    raw[page, 0, 1, 5, 7] = 0x7F if scaled else float("nan")  # request 0, head 1: a key
    kw = {} if scaled else dict(first=1, window=L)  # (the window path over a 16-bit cache)
    out, lse = call(dict(c, **kw), 0.05)
    assert torch.isnan(out[0, 4:].float()).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(out[0, :4].float()).all() and torch.isfinite(out[1].float()).all()


def test_graph_on_another_stream_follows_its_inputs():
    c = make([700, 300], 16, 16, 4, wl.HND, torch.bfloat16, 37, scaled=True, G=16, window=200, first=8, poison=False)
    pool, sc, table = c["pool"].to(DEV), c["scales"].to(DEV), c["table"].to(DEV)
    q, lens = c["query"].to(DEV), torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    n = pk.paged_decode_workspace_size(2, 1, 16, 4, 128, 700, 16, 200, first_tokens=8)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(2, 16, dtype=torch.float32, device=DEV)

    def step():
        pk.paged_decode(q, pool, ws, table, lens, 700, bmm1_scale=0.05, window_left=200, first_tokens=8, kv_scales=sc,
                        kv_layout="HND", out=out, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for new in ([700, 300], [500, 7], [40, 250]):
        lens.copy_(torch.tensor(new))
        sc.mul_(0.5)
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            g.replay()
        torch.cuda.current_stream().wait_stream(s)
        got = out.clone(), lse.clone()
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        d = dict(c, lens=new, scales=sc.cpu(), used=[_plain.visible(torch.arange(L), torch.tensor([L - 1]), 200, 8).any(0) for L in new])
        compare(d, got[0], got[1], 0.05)


def test_refusals():
    c = make([100], 16, 8, 2, wl.HND, torch.bfloat16, 38, scaled=True, G=16)
    with pytest.raises(pk.PagedKVError):  # scales over a 16-bit cache
        call(dict(c, pool=c["pool"].to(torch.bfloat16)), 0.05)
    with pytest.raises(pk.PagedKVError):
        call(dict(c, scales=c["scales"][:, :, :1]), 0.05)
    with pytest.raises(pk.PagedKVError):
        call(dict(c, scales=c["scales"].repeat(1, 1, 1, 4)), 0.05)  # blocks of 4 tokens
    with pytest.raises(pk.PagedKVError):
        call(dict(c, window=5, first=-3), 0.05)
