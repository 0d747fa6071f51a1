"""The ring that the own keys of a shared decode go through: stages whose
records are written again while the warps that read them run apart."""
from __future__ import annotations

import pytest
import torch

import _plain
from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_decode_shared import QLEN, U, check, group_of, make, run

pytestmark = pytest.mark.gpu


def check_short(c, out, lse, b):
    """A request with fewer own keys than tokens: tokens before its own keys see the prefix alone, all of it."""
    g, Q, L = group_of(c, b), c["q"], c["lens"][b]
    k, v = (torch.cat((_plain.tokens(c["pool"][:, z], c["ptab"][g], c["prefix"][g], c["S"], c["layout"]),
                       _plain.tokens(c["pool"][:, z], c["btab"][b], L, c["S"], c["layout"]))).double() for z in range(2))
    for t in range(Q):
        row, n = b * Q + t, c["prefix"][g] + max(0, L - Q + t + 1)
        o, l, bo, bl = _plain.attention(c["query"][row:row + 1].double(), k[:n], v[:n], n, c["scale"], u_p=U[c["dtype"]],
                                        u_out=U[c["dtype"]])
        _plain.check(out[row:row + 1], o, bo, f"out of token {t} of request {b}")
        _plain.check(lse[row:row + 1], l, bl, f"lse of token {t} of request {b}")


@pytest.mark.parametrize("S,layout,q,dtype", [(8, wl.HND, 1, torch.bfloat16), (8, wl.NHD, 4, torch.float16),
                                              (64, wl.HND, 2, torch.bfloat16)])
def test_records_that_are_written_again(S, layout, q, dtype):
    # 800 items of one to ten tiles, V's copies issued box by box (pages of 8: eight to a tile) while the producer runs
    # ahead: the same bits in every run, and right
    lens = [(i * 331) % 600 for i in range(200)]
    c = make([64], [200], lens, Hq=8, H=4, S=S, layout=layout, q=q, dtype=dtype, seed=60 + q)
    out, lse, err = run(c)
    assert err == QLEN
    for b in (0, 1, 2, 50, 77, 120, 198, 199):
        if lens[b] < q:
            check_short(c, out, lse, b)
        else:
            check(c, out, lse, requests=[b])
    for _ in range(10):
        again, again_lse, _ = run(c)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)
