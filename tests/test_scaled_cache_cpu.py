"""The plain E4M3 arithmetic that the GPU tests rely on, and what the entry
points of the scaled cache and of windows with first tokens refuse (host
checks: the fake pointers are never used)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import _plain
from test_abi_cpu import lib  # noqa: F401  (the built library, a fixture)

GOOD = 0x1000


def test_plain_codes_match_the_type():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_plain.from_codes(codes), want, equal_nan=True)
    x = torch.cat((torch.randn(4000, dtype=torch.float64) * 100, torch.randn(4000, dtype=torch.float64) * 0.02,
                   torch.linspace(-449, 449, 3593, dtype=torch.float64)))
    x = x.clamp(-448, 448).float().double()
    assert np.array_equal(_plain.to_codes(x.numpy()) & 0x7F,
                          x.to(torch.float8_e4m3fn).view(torch.uint8).numpy() & 0x7F)


def _append(lib, **over):  # noqa: F811
    a = dict(key=GOOD, value=GOOD, nnz=4, bi=GOOD, pos=GOOD, k=GOOD, v=GOOD, stride=2 * 8 * 16 * 128, pages=10,
             ks=GOOD, vs=GOOD, ss=16, block=16, idx=GOOD, ptr=GOOD, last=GOOD, B=2, H=8, D=128, S=16, layout=0,
             dtype=1, err=None, stream=None)
    a.update(over)
    return lib.paged_append_scaled(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(layout=2), 2), (dict(dtype=2), 2), (dict(dtype=3), 2), (dict(D=120), 2), (dict(D=0), 2), (dict(H=0), 2),
    (dict(S=24), 3), (dict(S=4), 3), (dict(S=512, stride=1 << 20), 3), (dict(block=4), 2), (dict(block=32), 2),
    (dict(block=12), 2), (dict(block=0), 2), (dict(ss=7), 2), (dict(block=8, ss=15), 2), (dict(stride=100), 2),
    (dict(stride=2 * 8 * 16 * 128 + 8), 2), (dict(nnz=-1), 2), (dict(key=None), 1), (dict(value=None), 1),
    (dict(bi=None), 1), (dict(k=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(idx=None), 1),
    (dict(last=None), 1), (dict(key=0x1008), 2), (dict(k=0x1004), 2), (dict(ks=0x1002), 2),
    (dict(nnz=0, key=None), 0),
])
def test_append_scaled_refuses(lib, over, status):  # noqa: F811
    assert _append(lib, **over) == status


def _decode(lib, **over):  # noqa: F811
    a = dict(q=GOOD, rows=4, k=GOOD, v=GOOD, stride=2 * 8 * 16 * 128, pages=64, ks=GOOD, vs=GOOD, ss=8, block=16,
             ws=GOOD, wsb=1 << 30, bt=GOOD, bts=10000, seq=GOOD, B=4, L=100, s1=0.1, s2=1.0, d1=None, d2=None, win=10,
             first=4, sinks=None, mq=1, cum=None, hq=32, hkv=8, D=128, S=16, layout=1, dtype=4, pdl=0, out=GOOD,
             lse=None, err=None, stream=None)
    a.update(over)
    return lib.paged_decode_window(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(first=-1), 2), (dict(win=-2), 2), (dict(layout=5), 2), (dict(dtype=1), 2), (dict(dtype=2), 2),
    (dict(block=4), 2), (dict(block=32), 2), (dict(block=0), 2), (dict(ss=7), 2), (dict(ks=None), 1),
    (dict(vs=None), 1), (dict(ks=None, vs=None), 1), (dict(rows=3), 2), (dict(mq=0), 2), (dict(D=64), 3),
    (dict(S=24), 3), (dict(mq=17, rows=100), 3), (dict(q=None), 1), (dict(ws=None, L=100000), 1),
    (dict(wsb=16, L=100000, win=-1), 4), (dict(L=(1 << 30) + 1, bts=1 << 28), 3), (dict(bts=2), 2), (dict(stride=2 * 8 * 16 * 128 + 8), 2),
    (dict(ks=None, vs=None, block=0, dtype=0, out=None), 1), (dict(rows=0, B=0), 0),
])
def test_decode_window_refuses(lib, over, status):  # noqa: F811
    if over.get("ws", 1) is None:  # (a window this short takes one split: no workspace)
        over = dict(over, win=-1)
    assert _decode(lib, **over) == status


def test_window_workspace_counts_the_first_tokens(lib):  # noqa: F811
    f, g = lib.paged_decode_window_workspace_size, lib.paged_decode_workspace_size
    a = (64, 1, 32, 8, 128, 65536, 16)
    assert f(*a, -1, 0) == f(*a, -1, 500) == g(*a, -1)
    assert f(*a, 8191, 0) == g(*a, 8191)
    assert f(*a, 8191, 0) <= f(*a, 8191, 4096) <= g(*a, -1)
    assert 0 < g(*a, -1) <= f(*a, 60000, 60000) <= 1.05 * g(*a, -1)  # everything is visible
    assert f(*a, 8191, -1) == 0                   # invalid


def test_binding_refuses_before_the_library():
    import paged_kv_cache_316_gb300 as pk
    from paged_kv_cache_316_gb300.binding import split_scales
    dev = -1  # (the device index of a CPU tensor)
    for bad in (torch.zeros(4, 3, 8, 1), torch.zeros(4, 2, 8), torch.zeros(5, 2, 8, 1), torch.zeros(4, 2, 7, 1),
                torch.zeros(4, 2, 8, 3), torch.zeros(4, 2, 8, 1, dtype=torch.float16),
                torch.zeros(4, 2, 8, 4)[..., ::2], torch.zeros(4, 2, 2, 8).transpose(2, 3),
                (torch.zeros(4, 8, 1), torch.zeros(4, 8, 2))):
        with pytest.raises(pk.PagedKVError):
            split_scales(bad, 4, 8, 16, dev)


def _prefill(lib, **over):  # noqa: F811
    a = dict(q=GOOD, rows=150, k=GOOD, v=GOOD, kst=8 * 32 * 128, vst=8 * 32 * 128, pages=100, ks=GOOD, vs=GOOD, ss=8,
             block=32, scale=0.08, ws=GOOD, wsb=1 << 40, mq=100, mkv=200, lq=GOOD, lkv=GOOD, bt=GOOD, bts=8, B=2,
             causal=1, win=10, first=4, hq=32, hkv=8, dqk=128, dv=128, S=32, layout=1, dtype=4, out=GOOD, lse=GOOD,
             oq=None, oo=None, ok=None, ov=None, err=None, stream=None)
    a.update(over)
    return lib.paged_prefill_window(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(win=-2), 2), (dict(first=-1), 2), (dict(dtype=1), 2), (dict(dtype=2), 2), (dict(layout=7), 2),
    (dict(bt=None), 2), (dict(ok=GOOD), 2), (dict(block=4), 2), (dict(block=64), 2), (dict(ss=7), 2),
    (dict(kst=8 * 32 * 128 + 8), 2), (dict(kst=100), 2), (dict(bts=3), 2), (dict(hkv=5), 2), (dict(dqk=64), 3),
    (dict(dv=64), 3), (dict(S=4), 3), (dict(ks=None), 1), (dict(vs=None), 1), (dict(lse=None), 1), (dict(k=0x1004), 2),
    (dict(wsb=4096), 4), (dict(ws=None), 1), (dict(mkv=-1), 2), (dict(rows=0), 0), (dict(B=0), 0),
    (dict(dtype=1, ks=None, vs=None, block=0, lse=None), 1), (dict(dtype=1, ks=None, vs=None, block=0, wsb=8), 4),
])
def test_prefill_window_refuses(lib, over, status):  # noqa: F811
    assert _prefill(lib, **over) == status


def test_binding_counts_the_columns_of_a_sliced_table(monkeypatch):
    import paged_kv_cache_316_gb300 as pk
    from paged_kv_cache_316_gb300 import binding
    # (tensors on the CPU)
    monkeypatch.setattr(binding, "split_cache", lambda c, layout: (0, 0, c.stride(0), 4, 8, 16, 128, c))
    monkeypatch.setattr(binding, "_same_device", lambda *t: (_ for _ in ()).throw(pk.PagedKVError("past the shapes")))
    cache = torch.zeros(4, 2, 8, 16, 128, dtype=torch.float8_e4m3fn)
    sc = torch.ones(4, 2, 8, 1)
    bt = torch.zeros(2, 8, dtype=torch.int32)[:, 4:]  # 4 columns, rows 8 apart
    lens = torch.tensor([64, 64], dtype=torch.int32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    q = torch.zeros(2, 32, 128, dtype=torch.bfloat16)

    def decode(n):
        return pk.paged_decode(q, cache, ws, bt, lens, n, kv_scales=sc)

    def prefill(n):
        return pk.paged_prefill(q, cache[:, 0], cache[:, 1], 0.1, ws, 1, n, torch.ones_like(lens), lens, bt,
                                kv_scales=sc)
    for call in (decode, prefill):
        with pytest.raises(pk.PagedKVError, match="fewer columns"):
            call(65)
        with pytest.raises(pk.PagedKVError, match="past the shapes"):
            call(64)
