"""The operators as a server runs them: a shared prompt appended with its
norms and rotations, requests that go on from it token by token, decoded over
the prefix and their own keys; prompts attended in parts and merged."""
from __future__ import annotations

import math

import pytest
import torch

import _plain
import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_rotary import check, plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = dict(dtype=torch.int32)
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("layout,dtype", [(wl.HND, torch.bfloat16), (wl.NHD, torch.float16)])
def test_a_session(layout, dtype):
    g = wl.generator(77)
    S, Hq, H, P, B, steps = 16, 8, 2, 200, 5, 4
    f, mag = pk.rotary_frequencies(128, 10000.0, "yarn", factor=4.0, trained_len=1024)
    wq, wk = ((torch.randn(128, generator=g) * 0.2 + 1).to(dtype) for _ in range(2))
    pages_prefix, pages_own = -(-P // S), 2
    n_pages = pages_prefix + B * pages_own
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    one = (S, H, 128) if layout == wl.NHD else (H, S, 128)
    pool = torch.full((n_pages, 2) + one, math.nan, dtype=dtype, device=DEV)
    ptab = order[:pages_prefix].view(1, -1).to(DEV)
    btab = order[pages_prefix:].view(B, pages_own).to(DEV)
    kw = dict(kv_layout=layout, magnitude=mag, query_weight=wq.to(DEV), key_weight=wk.to(DEV), eps=1e-6)

    def new(n):
        return [torch.randn(n, h, 128, generator=g).to(dtype) for h in (Hq, H, H)]

    def stored(table, n, ks, vs, pos):
        """The request's keys and values as the pages hold them, the last ones checked against the definition."""
        host = pool.cpu()
        k, v = (_plain.tokens(host[:, z], table, n, S, layout) for z in range(2))
        m = len(ks)
        check(k[n - m:], plain(ks, wk, pos, f.cpu(), 0, False, mag, 1e-6), dtype, "stored keys")
        assert torch.equal(v[n - m:], vs)
        return k.double(), v.double()
    # the prompt
    q, k, v = new(P)
    pos = torch.arange(P, **I32)
    pk.paged_append_rotary(*(x.to(DEV) for x in (q, k, v)), torch.zeros(P, device=DEV, **I32), pos.to(DEV), pool,
                           ptab.flatten(), torch.tensor([0, pages_prefix], device=DEV, **I32),
                           torch.tensor([P - (pages_prefix - 1) * S], device=DEV, **I32), f, **kw)
    keys, values = stored(order[:pages_prefix], P, k, v, pos)
    ws = torch.empty(pk.paged_decode_shared_workspace_size(B, 1, Hq, H, 128, 1, P, pages_own * S, S), dtype=torch.uint8, device=DEV)
    for t in range(steps):
        q, k, v = new(B)
        at = torch.full((B,), t, **I32)
        query = pk.paged_append_rotary(*(x.to(DEV) for x in (q, k, v)), torch.arange(B, device=DEV, **I32), at.to(DEV), pool,
                                       btab.flatten(), torch.arange(B + 1, device=DEV, **I32) * pages_own,
                                       torch.full((B,), S, device=DEV, **I32), f, rotary_positions=(at + P).to(DEV), **kw)
        lse = torch.empty(B, Hq, device=DEV)
        out = pk.paged_decode_shared(query, pool, ws, ptab, torch.tensor([P], device=DEV, **I32),
                                     torch.tensor([0, B], device=DEV, **I32), P, btab, (at + 1).to(DEV), pages_own * S,
                                     bmm1_scale=1 / math.sqrt(128), kv_layout=layout, lse=lse)
        check(query, plain(q, wq, at + P, f.cpu(), 0, False, mag, 1e-6), dtype, "query")
        for b in range(B):
            ko, vo = stored(btab[b].cpu(), t + 1, k[b:b + 1], v[b:b + 1], at[b:b + 1] + P)
            o, l, bo, bl = _plain.attention(query[b:b + 1].cpu().double(), torch.cat((keys, ko)), torch.cat((values, vo)),
                                            P + t + 1, 1 / math.sqrt(128), u_p=U[dtype], u_out=U[dtype])
            _plain.check(out[b:b + 1], o, bo, f"step {t} out {b}")
            _plain.check(lse[b:b + 1], l, bl, f"step {t} lse {b}")


def test_decode_shared_is_decode_over_the_joined_tables():
    g = wl.generator(78)
    S, Hq, H, P, B = 32, 16, 4, 320, 7
    lens = [1, 40, 64, 200, 33, 2, 90]
    pt = wl.reserve_pages([P] + lens, S, g, extra=1)
    pool = torch.randn(pt.num_pages, 2, H, S, 128, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(B, Hq, 128, generator=g).to(torch.bfloat16).to(DEV)
    table = pt.block_tables(pt.max_pages())
    joined = torch.cat((table[:1, :P // S].expand(B, -1), table[1:]), 1).contiguous().to(DEV)
    total = torch.tensor([P + n for n in lens], device=DEV, **I32)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    la, lb = torch.empty(B, Hq, device=DEV), torch.empty(B, Hq, device=DEV)
    a = pk.paged_decode(q, pool, ws, joined, total, P + 200, bmm1_scale=0.09, lse=la).clone()
    b = pk.paged_decode_shared(q, pool, ws, table[:1].to(DEV), torch.tensor([P], device=DEV, **I32),
                               torch.tensor([0, B], device=DEV, **I32), P, table[1:].to(DEV),
                               torch.tensor(lens, device=DEV, **I32), 200, bmm1_scale=0.09, lse=lb)
    # each within its weights' roundings and one of its own of the exact value (values of size about 1)
    assert ((a - b).float().abs() <= 2 * (2.0 ** -8 * a.float().abs() + 2.0 ** -8 * 1.5)).all()
    assert ((la - lb).abs() <= 2.0 ** -14).all()


def test_prompts_in_two_parts_merged():
    g = wl.generator(79)
    S, Hq, H, P, B, n = 16, 8, 2, 160, 3, 37
    pt = wl.reserve_pages([P, n, n, n], S, g, extra=1)
    pool = torch.randn(pt.num_pages, 2, H, S, 128, generator=g).to(torch.float16)
    q = torch.randn(B * n, Hq, 128, generator=g).to(torch.float16)
    table = pt.block_tables(pt.max_pages())
    k, v = pool[:, 0].to(DEV), pool[:, 1].to(DEV)
    ws = torch.empty(pk.paged_prefill_workspace_size(B, Hq, n, P), dtype=torch.uint8, device=DEV)
    new = torch.full((B,), n, device=DEV, **I32)
    first = pk.paged_prefill(q.to(DEV), k, v, 0.09, ws, n, P, new, torch.full((B,), P, device=DEV, **I32),
                             table[:1].expand(B, -1).contiguous().to(DEV), causal=False)
    own = pk.paged_prefill(q.to(DEV), k, v, 0.09, ws, n, n, new, new, table[1:].to(DEV), causal=True)
    out, lse = pk.paged_merge_states([first, own], out=own[0], lse=own[1])
    for b in range(B):
        kv = [torch.cat((_plain.tokens(pool[:, z], table[0], P, S, wl.HND), _plain.tokens(pool[:, z], table[1 + b], n, S, wl.HND))).double()
              for z in range(2)]
        o, l, bo, bl = _plain.attention(q[b * n:(b + 1) * n].double(), *kv, P + n, 0.09, u_p=2.0 ** -11, u_out=2.0 ** -11)
        # the parts' outputs are rounded once more before they are merged
        _plain.check(out[b * n:(b + 1) * n], o, bo + 2.0 ** -11 * (o.abs() + 2 * kv[1].abs().max()), f"out {b}")
        _plain.check(lse[b * n:(b + 1) * n], l, bl, f"lse {b}")
