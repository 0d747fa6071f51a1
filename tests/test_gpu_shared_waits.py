"""Shared decode when a wait of its pipelines runs out: every warp waits only
for copies that it issued itself, so that the call ends at once and the next
one is right.  The limit of the waits is one nanosecond here; the wait for
copies in flight before a CTA exits has a limit of its own, one second, so a
call that takes less has waited for nothing that does not come."""
from __future__ import annotations

import time

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_decode_shared import args, make

pytestmark = pytest.mark.gpu

TIMEOUT = 16  # PKV_DEV_ERR_TIMEOUT


@pytest.fixture(autouse=True)
def _default_limit_afterwards():
    yield
    pk.set_wait_limit_ns(0)


@pytest.mark.parametrize("prefix,sizes,lens,S,layout,q", [
    ([64], [200], [4 + (i * 331) % 600 for i in range(200)], 8, wl.HND, 1),     # V in eight boxes a tile, 800 items
    ([64], [200], [4 + (i * 331) % 600 for i in range(200)], 64, wl.NHD, 4),
    ([], [], [1000 + (i * 331) % 2000 for i in range(150)], 16, wl.HND, 1),     # several waves of items, no prefix
    ([9000], [50], [4 + i % 70 for i in range(50)], 16, wl.HND, 1),             # mostly prefix
])
def test_the_call_ends_at_once(prefix, sizes, lens, S, layout, q):
    c = make(prefix, sizes, lens, Hq=8, H=4, S=S, layout=layout, q=q, seed=70 + S + q, poison=False)
    a = args(c)
    good = pk.paged_decode_shared(**a).clone()
    torch.cuda.synchronize()
    for _ in range(5):
        pk.set_wait_limit_ns(1)
        t = time.perf_counter()
        pk.paged_decode_shared(**a)
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        pk.set_wait_limit_ns(0)
        assert t < 0.9, f"{t:.2f} s"
        assert int(a["err_word"].item()) in (0, TIMEOUT)  # (a wait may be met within its first polls)
        a["err_word"].zero_()
        pk.paged_decode_shared(**a)
        torch.cuda.synchronize()
        assert int(a["err_word"].item()) == 0 and torch.equal(a["out"], good)
