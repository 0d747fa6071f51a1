"""paged_append_scaled against the plain implementation: codes and scales
have to be the same bit for bit, and nothing else may be written."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import _plain
import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BATCH, POS, PAGE, SCALE = 4, 2, 1, 128


def case(new, old, S, G, H, D, layout, dtype, seed, form="5d", scale_exp=(-9, -5), mag=4.0):
    g = wl.generator(seed)
    pt = wl.reserve_pages([a + b for a, b in zip(new, old)], S, g, extra=3)
    one = (S, H, D) if layout == wl.NHD else (H, S, D)
    cache = (torch.randn((pt.num_pages, 2) + one, generator=g) * 112).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.randint(scale_exp[0], scale_exp[1] + 1, (pt.num_pages, 2, H, S // G), generator=g).float())
    n = sum(new)
    m = mag ** torch.randint(-2, 3, (n, H, 1), generator=g).float()
    key = (torch.randn(n, H, D, generator=g) * m).to(dtype)
    value = (torch.randn(n, H, D, generator=g) * m).to(dtype)
    bi = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(torch.int32)
    pos = torch.cat([torch.arange(o, o + k) for k, o in zip(new, old)] + [torch.zeros(0, dtype=torch.int64)]).to(torch.int32)
    return dict(pt=pt, cache=cache, scales=scales, key=key, value=value, bi=bi, pos=pos, S=S, layout=layout, form=form)


def run(c, drop=(), expect_err=0, stream=None):
    indptr, indices, last = c["pt"].csr()
    codes = c["cache"].view(torch.uint8).numpy().copy()
    scales = c["scales"].numpy().copy()
    _plain.append_scaled(c["key"], c["value"], c["bi"].numpy(), c["pos"].numpy(), codes, scales, indices.numpy(),
                         indptr.numpy(), c["pt"].lengths, c["S"], c["layout"], drop)
    cache, sc = c["cache"].to(DEV), c["scales"].to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kv, ks = cache, sc
    if c["form"] == "tuple":
        kv = (cache[:, 0].contiguous(), cache[:, 1].contiguous())
        ks = (sc[:, 0].contiguous(), sc[:, 1].contiguous())
    pk.paged_append_scaled(c["key"].to(DEV), c["value"].to(DEV), c["bi"].to(DEV), c["pos"].to(DEV), kv, ks,
                           indices.to(DEV), indptr.to(DEV), last.to(DEV), kv_layout=c["layout"], err_word=err,
                           stream=stream)
    torch.cuda.synchronize()
    if c["form"] == "tuple":
        cache, sc = torch.stack(kv, 1), torch.stack(ks, 1)
    assert int(err.item()) == expect_err
    assert np.array_equal(sc.cpu().numpy().view(np.uint32), scales.view(np.uint32)), "scales differ"
    got = cache.cpu().view(torch.uint8).numpy()
    nan = ((codes & 0x7F) == 0x7F) & ((got & 0x7F) == 0x7F)
    assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, codes)), f"{int((got != codes).sum())} codes differ"


@pytest.mark.parametrize("new, old, S, G, H, D, layout, dtype, form, seed", [
    ([1, 1, 1, 1], [0, 1, 15, 33], 16, 16, 8, 128, wl.HND, torch.bfloat16, "5d", 1),
    ([1], [7], 8, 8, 1, 128, wl.NHD, torch.float16, "5d", 2),
    ([5, 40, 1, 0, 17], [3, 0, 31, 9, 64], 32, 8, 3, 128, wl.NHD, torch.float16, "tuple", 3),
    ([100, 257, 2], [0, 13, 255], 256, 256, 2, 128, wl.HND, torch.bfloat16, "5d", 4),
    ([33, 64, 65], [5, 0, 63], 64, 32, 4, 64, wl.HND, torch.float16, "tuple", 5),
    ([70, 3], [2, 29], 128, 64, 5, 16, wl.NHD, torch.bfloat16, "5d", 6),
    ([50, 9, 8], [6, 8, 0], 16, 8, 2, 272, wl.HND, torch.bfloat16, "5d", 7),
    ([200, 1, 31], [1, 0, 1], 16, 16, 32, 128, wl.NHD, torch.float16, "5d", 8),
])
def test_bits(new, old, S, G, H, D, layout, dtype, form, seed):
    run(case(new, old, S, G, H, D, layout, dtype, seed, form))


def test_many_entries():  # several entries to a warp's share of the work
    run(case([300, 1, 77, 512, 130], [3, 16, 0, 40, 8], 16, 16, 8, 128, wl.HND, torch.bfloat16, 21))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_extreme_values(dtype):
    c = case([40, 24, 3], [5, 0, 9], 16, 8, 2, 128, wl.HND, dtype, 11)
    k, v = c["key"], c["value"]
    k[0, 0, 3], k[1, 0, 5], k[2, 1, 7] = float("nan"), float("inf"), -float("inf")
    k[8:16] = float("nan")
    v[3:20, 0] = 0.0
    v[20:40] = torch.finfo(dtype).tiny / 4 if dtype == torch.float16 else 1e-38
    v[41, 0, 0] = torch.finfo(dtype).max
    k[42, 1, 9], k[43, 1, 9] = 448.0, 449.0 if dtype == torch.float16 else 450.0
    run(c)


def test_scale_that_is_no_power_of_two_and_grows():
    c = case([9, 3], [3, 5], 16, 16, 2, 128, wl.NHD, torch.bfloat16, 12)
    c["scales"] *= 0.7
    run(c)
    c["key"] *= 64
    run(c)


@pytest.mark.parametrize("exp", [-15, -16, -30, 8, 24, 25, 40])
def test_earlier_scale_at_the_ends_of_its_range(exp):
    # fp16 values of every exponent (subnormal ones too) under one held scale
    c = case([11], [5], 16, 16, 2, 128, wl.HND, torch.float16, 22)
    g = wl.generator(23)
    m = torch.exp2(torch.randint(-24, 15, c["key"].shape, generator=g).float())
    c["key"] = (m * (1 + torch.rand(m.shape, generator=g))).half()
    c["value"] = (-m * 1.5 * 2.0 ** -10).half()
    c["scales"][:] = 2.0 ** exp
    run(c)


def test_earlier_scale_out_of_range_is_flagged_and_clamped():
    c = case([2, 2], [3, 5], 16, 16, 2, 128, wl.NHD, torch.bfloat16, 13)
    for b, x in ((0, float("nan")), (1, 0.0)):
        c["scales"][c["pt"].pages[b][0], 0, 1, 0] = x
    run(c, expect_err=SCALE)


def test_appending_twice_is_the_same():
    c = case([20, 1], [3, 15], 16, 16, 4, 128, wl.HND, torch.bfloat16, 14)
    indptr, indices, last = (t.to(DEV) for t in c["pt"].csr())
    cache, sc = c["cache"].to(DEV), c["scales"].to(DEV)
    args = [c[k].to(DEV) for k in ("key", "value", "bi", "pos")]
    got = []
    for _ in range(2):
        pk.paged_append_scaled(*args, cache, sc, indices, indptr, last, kv_layout="HND")
        got.append((cache.clone(), sc.clone()))
    assert torch.equal(got[0][0].view(torch.uint8), got[1][0].view(torch.uint8)) and torch.equal(got[0][1], got[1][1])


def test_bad_entries_are_skipped_and_flagged():
    # request index, position, page and order
    c = case([4, 4, 4, 4], [0, 16, 3, 8], 16, 16, 2, 128, wl.HND, torch.bfloat16, 15)
    c["bi"][0] = 9
    run(c, drop=(0,), expect_err=BATCH)
    c = case([4, 4, 4], [0, 16, 3], 16, 16, 2, 128, wl.HND, torch.bfloat16, 16)
    c["pos"][3], c["pos"][11] = -1, 4000
    run(c, drop=(3, 11), expect_err=POS)
    c = case([4, 4], [0, 16], 16, 16, 2, 128, wl.HND, torch.bfloat16, 17)
    c["pt"].pages[1][1] = 0x7FFFFFFF
    run(c, drop=(4, 5, 6, 7), expect_err=PAGE)
    c = case([4, 4], [0, 17], 16, 16, 2, 128, wl.HND, torch.bfloat16, 18)
    c["pos"][6], c["pos"][7] = 20, 21  # a gap inside the block
    c["pt"].lengths[1] = 22
    run(c, drop=(6, 7), expect_err=POS)


def test_another_stream_and_graph():
    c = case([20, 1], [3, 15], 16, 16, 4, 128, wl.HND, torch.bfloat16, 19)
    s = torch.cuda.Stream()
    run(c, stream=s)
    indptr, indices, last = (t.to(DEV) for t in c["pt"].csr())
    cache, sc = c["cache"].to(DEV), c["scales"].to(DEV)
    want, wsc = cache.clone(), sc.clone()
    args = [c[k].to(DEV) for k in ("key", "value", "bi", "pos")]
    pk.paged_append_scaled(*args, want, wsc, indices, indptr, last, kv_layout="HND")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.paged_append_scaled(*args, cache, sc, indices, indptr, last, kv_layout="HND")
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.view(torch.uint8), want.view(torch.uint8)) and torch.equal(sc, wsc)


def test_refusals():
    c = case([2], [3], 16, 16, 2, 128, wl.NHD, torch.bfloat16, 20)
    indptr, indices, last = (t.to(DEV) for t in c["pt"].csr())
    k, v, bi, pos = (c[n].to(DEV) for n in ("key", "value", "bi", "pos"))
    cache, sc = c["cache"].to(DEV), c["scales"].to(DEV)

    def call(**o):
        a = dict(k=k, v=v, bi=bi, pos=pos, cache=cache, sc=sc, indices=indices, indptr=indptr, last=last)
        a.update(o)
        pk.paged_append_scaled(*a.values())

    for o in (dict(k=k.float()), dict(v=v.half()), dict(k=k[:, :1]), dict(cache=cache.view(torch.uint8)),
              dict(sc=sc.double()), dict(sc=sc[:-1]), dict(sc=sc.cpu()), dict(bi=bi[:1]), dict(pos=pos.long()),
              dict(indptr=indptr[:1]), dict(last=last.long()), dict(k=k.cpu()),
              dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(sc=sc[:, :1].expand(-1, 2, -1, -1))):
        with pytest.raises(pk.PagedKVError):
            call(**o)
    call()
