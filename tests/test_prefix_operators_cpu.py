"""What the entry points of rotated appends, decode over shared prefixes and
merged states refuse (host checks: the fake pointers are never used), and the
frequencies of scaled rotations."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from test_abi_cpu import lib  # noqa: F401  (the built library, a fixture)
from test_cache_pair_cpu import _OnGpu0

GOOD = 0x1000


def _rotary(lib, **over):  # noqa: F811
    a = dict(q=GOOD, k=GOOD, qs=32 * 128, ks=8 * 128, n=4, pos=GOOD, f=GOOD, rd=128, start=0, inter=0, mag=1.0, qw=GOOD,
             kw=GOOD, eps=1e-6, hq=32, hk=8, D=128, dtype=1, qo=GOOD, ko=GOOD, stream=None)
    a.update(over)
    return lib.paged_rotary(*a.values())


def _append(lib, **over):  # noqa: F811
    a = dict(q=GOOD, k=GOOD, v=GOOD, qs=32 * 128, ks=8 * 128, vs=8 * 128, n=4, bi=GOOD, pos=GOOD, rp=None, kc=GOOD,
             vc=GOOD, stride=2 * 8 * 16 * 128, pages=10, idx=GOOD, ptr=GOOD, last=GOOD, B=2, f=GOOD, rd=128, start=0,
             inter=0, mag=1.0, qw=None, kw=None, eps=1e-6, hq=32, hk=8, D=128, S=16, layout=0, dtype=1, qo=GOOD,
             err=None, stream=None)
    a.update(over)
    return lib.paged_append_rotary(*a.values())


COMMON = [
    (dict(dtype=2), 2), (dict(dtype=7), 2), (dict(n=-1), 2), (dict(hq=0), 2), (dict(hk=0), 2), (dict(D=120), 2),
    (dict(D=0), 2), (dict(rd=24), 2), (dict(rd=-16), 2), (dict(start=-8), 2), (dict(start=8), 2), (dict(rd=64, start=65), 2),
    (dict(rd=64, start=60), 2), (dict(rd=144), 2), (dict(D=272, qs=32 * 272, ks=8 * 272, vs=8 * 272), 3),
    (dict(qs=32 * 128 - 8), 2), (dict(ks=8 * 128 + 4), 2), (dict(q=0x1008), 2), (dict(k=0x1004), 2), (dict(qo=0x1008), 2),
    (dict(qw=0x1008), 2), (dict(f=0x1004), 2), (dict(eps=-1.0), 2), (dict(eps=math.nan), 2), (dict(q=None), 1),
    (dict(k=None), 1), (dict(pos=None), 1), (dict(f=None), 1), (dict(qo=None), 1), (dict(n=0, q=None), 0),
    (dict(n=1 << 31), 3),
]


def _fits(over):
    return {k: v for k, v in over.items() if k != "vs"}


@pytest.mark.parametrize("over, status", COMMON + [(dict(ko=None), 1), (dict(ko=0x1002), 2)])
def test_rotary_refuses(lib, over, status):  # noqa: F811
    assert _rotary(lib, **_fits(over)) == status


@pytest.mark.parametrize("over, status", COMMON + [
    (dict(layout=2), 2), (dict(S=24), 3), (dict(S=0), 3), (dict(stride=100), 2), (dict(stride=2 * 8 * 16 * 128 + 4), 2),
    (dict(B=-1), 2), (dict(pages=-1), 2), (dict(vs=8), 2), (dict(v=None), 1), (dict(bi=None), 1), (dict(kc=None), 1),
    (dict(vc=None), 1), (dict(idx=None), 1), (dict(ptr=None), 1), (dict(last=None), 1), (dict(vc=0x1008), 2),
])
def test_append_rotary_refuses(lib, over, status):  # noqa: F811
    if over.get("D") == 272:
        over = dict(over, stride=2 * 8 * 16 * 272)
    assert _append(lib, **over) == status


def _shared(lib, **over):  # noqa: F811
    a = dict(q=GOOD, k=GOOD, v=GOOD, stride=2 * 8 * 16 * 128, pages=64, ws=GOOD, wsb=1 << 40, pt=GOOD, pts=10000,
             pl=GOOD, gi=GOOD, G=2, maxp=1000, bt=GOOD, bts=10000, seq=GOOD, B=4, L=100, s1=0.1, s2=1.0, d1=None, d2=None,
             sinks=None, Q=1, hq=32, hkv=8, D=128, S=16, layout=1, dtype=1, out=GOOD, lse=None, err=None, stream=None)
    a.update(over)
    return lib.paged_decode_shared(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(layout=4), 2), (dict(dtype=2), 2), (dict(dtype=4), 2), (dict(G=-1), 2), (dict(maxp=-1), 2), (dict(B=-1), 2),
    (dict(Q=0), 2), (dict(hq=30), 2), (dict(D=64), 3), (dict(S=24), 3), (dict(S=512, stride=1 << 21), 3),
    (dict(Q=9, hq=64), 3), (dict(stride=100), 2), (dict(stride=2 * 8 * 16 * 128 + 4), 2), (dict(pages=-1), 2),
    (dict(bts=2), 2), (dict(pts=2), 2), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(ws=None), 1),
    (dict(pt=None), 1), (dict(pl=None), 1), (dict(gi=None), 1), (dict(bt=None), 1), (dict(seq=None), 1),
    (dict(out=None), 1), (dict(q=0x1008), 2), (dict(k=0x1008), 2), (dict(out=0x1008), 2), (dict(wsb=1000), 4),
    (dict(ws=0x1010), 4), (dict(maxp=(1 << 30) + 1, pts=1 << 27), 3), (dict(B=0, q=None), 0),
])
def test_decode_shared_refuses(lib, over, status):  # noqa: F811
    assert _shared(lib, **over) == status


def test_shared_workspace_follows_sizes(lib):  # noqa: F811
    f = lib.paged_decode_shared_workspace_size
    a = f(64, 1, 32, 8, 128, 1, 8192, 1024, 16)
    assert a > 64 * 32 * 129 * 4 * 2  # a partial of the prefix and one of the own keys for every row
    assert f(64, 1, 32, 8, 128, 0, 0, 1024, 16) <= a
    assert f(64, 1, 32, 8, 64, 1, 8192, 1024, 16) == 0
    assert f(64, 1, 32, 8, 128, -1, 8192, 1024, 16) == 0
    assert f(0, 1, 32, 8, 128, 0, 0, 0, 16) == 0


def _merge(lib, n=2, outs=None, lses=None, **over):  # noqa: F811
    outs = (ctypes.c_void_p * 20)(*(outs or [GOOD] * 20))
    lses = (ctypes.c_void_p * 20)(*(lses or [GOOD] * 20))
    a = dict(outs=ctypes.addressof(outs), lses=ctypes.addressof(lses), n=n, rows=10, D=128, dtype=1, out=GOOD, lse=GOOD,
             stream=None)
    a.update(over)
    return lib.paged_merge_states(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(n=0), 2), (dict(n=17), 3), (dict(rows=-1), 2), (dict(D=0), 2), (dict(D=12), 2), (dict(D=264), 3),
    (dict(dtype=2), 2), (dict(out=None), 1), (dict(lse=None), 1), (dict(outs=None), 1), (dict(out=0x1008), 2),
    (dict(lse=0x1002), 2), (dict(rows=0, out=None), 0), (dict(rows=1 << 40), 3),
])
def test_merge_states_refuses(lib, over, status):  # noqa: F811
    if "outs" in over:
        assert lib.paged_merge_states(None, None, 2, 10, 128, 1, GOOD, GOOD, None) == status
        return
    assert _merge(lib, **over) == status


def test_merge_states_refuses_bad_parts(lib):  # noqa: F811
    assert _merge(lib, outs=[GOOD, None] + [GOOD] * 18) == 1
    assert _merge(lib, lses=[GOOD, 0x1001] + [GOOD] * 18) == 2
    assert _merge(lib, outs=[GOOD, 0x1004] + [GOOD] * 18) == 2


def test_frequencies():
    import paged_kv_cache_316_gb300 as pk
    f, m = pk.rotary_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and m == 1.0
    for i in (0, 1, 31):
        assert f[i].item() == pytest.approx(10000.0 ** (-2 * i / 64), rel=1e-15)
    lin, m = pk.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-15) and m == 1.0
    ntk, _ = pk.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1 and ntk[-1].item() == pytest.approx(f[-1].item() / 4, rel=1e-12)  # the slowest is interpolated
    y, m = pk.rotary_frequencies(64, scaling="yarn", factor=8.0, trained_len=4096, device="cpu")
    assert m == pytest.approx(0.1 * math.log(8) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(y[turns > 32], f[turns > 32]) and torch.allclose(y[turns < 1], f[turns < 1] / 8, rtol=1e-15)
    mid = (turns >= 1) & (turns <= 32)
    assert mid.any() and ((y[mid] <= f[mid]) & (y[mid] >= f[mid] / 8)).all()
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=0.0), dict(rotary_dim=64, factor=0.5),
                dict(rotary_dim=64, scaling="other"), dict(rotary_dim=64, scaling="yarn", factor=2.0),
                dict(rotary_dim=2, scaling="ntk", factor=2.0),
                dict(rotary_dim=64, scaling="yarn", factor=2.0, trained_len=4096, fast=1.0, slow=1.0)):
        with pytest.raises(pk.PagedKVError):
            pk.rotary_frequencies(device="cpu", **bad)


def _gpu(*shape, dtype=torch.bfloat16):
    return _OnGpu0(torch.zeros(*shape, dtype=dtype))


def test_binding_refuses_rotary():
    import paged_kv_cache_316_gb300 as pk
    q, k = torch.zeros(4, 32, 128, dtype=torch.bfloat16), torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.ones(64, dtype=torch.float64)
    for over in (dict(key=k[:3]), dict(key=k.half()), dict(query=q.float()), dict(query=q.transpose(0, 1)),
                 dict(query=q[..., ::2]), dict(positions=pos[:3]), dict(positions=pos.long()), dict(frequencies=f.float()),
                 dict(frequencies=f[::2]), dict(query_weight=torch.ones(64, dtype=torch.bfloat16)),
                 dict(key_weight=torch.ones(128)), dict(query_out=torch.empty(4, 32, 64, dtype=torch.bfloat16)),
                 dict(key_out=torch.empty(4, 8, 128)), dict()):  # (the last: tensors of the CPU)
        a = dict(query=q, key=k, positions=pos, frequencies=f)
        a.update(over)
        with pytest.raises(pk.PagedKVError):
            pk.paged_rotary(**a)


def test_binding_refuses_append_rotary():
    import paged_kv_cache_316_gb300 as pk
    q, k = torch.zeros(4, 32, 128, dtype=torch.bfloat16), torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i, f = torch.zeros(4, dtype=torch.int32), torch.ones(64, dtype=torch.float64)
    base = dict(query=q, key=k, value=k, batch_indices=i, positions=i, paged_kv_cache=_gpu(4, 2, 16, 8, 128), kv_indices=i,
                kv_indptr=i[:3], kv_last_page_len=i[:2], frequencies=f)
    for over in (dict(value=k[:3]), dict(value=k[:, :4]), dict(key=k[:, :4].contiguous()), dict(value=k.half()),
                 dict(paged_kv_cache=_gpu(4, 2, 16, 8, 128, dtype=torch.float16)), dict(kv_layout="HND"),
                 dict(paged_kv_cache=_gpu(4, 2, 16, 8, 128, dtype=torch.float8_e4m3fn)), dict(batch_indices=i[:3]),
                 dict(rotary_positions=i[:2]), dict(rotary_positions=i.long()), dict(kv_indptr=i), dict(kv_indices=i.long()),
                 dict(query=q[..., :64].contiguous()), dict()):
        with pytest.raises(pk.PagedKVError):
            pk.paged_append_rotary(**dict(base, **over))


def test_binding_refuses_decode_shared():
    import paged_kv_cache_316_gb300 as pk
    i32 = dict(dtype=torch.int32)
    base = dict(query=torch.zeros(4, 32, 128, dtype=torch.bfloat16), kv_cache=_gpu(4, 2, 8, 16, 128),
                workspace=torch.zeros(1 << 16, dtype=torch.uint8), prefix_tables=torch.zeros(2, 8, **i32),
                prefix_lens=torch.zeros(2, **i32), group_indptr=torch.zeros(3, **i32), max_prefix_len=100,
                block_tables=torch.zeros(4, 2, **i32), seq_lens=torch.ones(4, **i32), max_seq_len=20)
    q = base["query"]
    for over in (dict(query=q[:3]), dict(query=q.half()), dict(query=q[..., :64].contiguous()),
                 dict(kv_cache=_gpu(4, 2, 8, 16, 128, dtype=torch.float8_e4m3fn)), dict(q_len_per_req=2),
                 dict(group_indptr=torch.zeros(2, **i32)), dict(prefix_lens=torch.zeros(2)), dict(max_prefix_len=129),
                 dict(max_seq_len=33), dict(block_tables=torch.zeros(3, 2, **i32)), dict(seq_lens=torch.ones(4, 1, **i32)),
                 dict(prefix_tables=torch.zeros(2, 16, **i32)[:, ::2]), dict(out=q.float()), dict(lse=torch.zeros(4, 8)),
                 dict(sinks=torch.zeros(8)), dict(bmm1_scale=torch.ones(2)), dict()):
        with pytest.raises(pk.PagedKVError):
            pk.paged_decode_shared(**dict(base, **over))


def test_binding_refuses_merge_states():
    import paged_kv_cache_316_gb300 as pk
    o, l = torch.zeros(4, 32, 128, dtype=torch.bfloat16), torch.zeros(4, 32)
    for states, kw in (([], {}), ([(o, l), (o.half(), l)], {}), ([(o, l), (o[:3], l)], {}), ([(o, l[:3])], {}),
                       ([(o, l.half())], {}), ([(o.float(), l)], {}), ([(o, l)], dict(out=o.float())),
                       ([(o, l)], dict(lse=l[:3])), ([(o, l)], {})):
        with pytest.raises(pk.PagedKVError):
            pk.paged_merge_states(states, **kw)
