"""Merged states out of lists that another thread changes meanwhile: a call
works on the tensors that it found."""
from __future__ import annotations

import threading

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_lists_that_change():
    g = wl.generator(7)
    pairs = [[torch.randn(5, 4, 64, generator=g).to(torch.bfloat16).to(DEV), torch.randn(5, 4, generator=g).to(DEV)]
             for _ in range(3)]
    want = {(i, j): pk.paged_merge_states([tuple(pairs[i]), tuple(pairs[j])])[0] for i in range(3) for j in range(3)}
    states = [list(pairs[0]), list(pairs[1])]
    stop = threading.Event()

    def change():
        i = 0
        while not stop.is_set():
            i += 1
            x = [pairs[i % 3][0].clone(), pairs[i % 3][1].clone()]  # tensors that nothing else holds
            states[i % 2][:] = x
            states[(i + 1) % 2] = list(pairs[i % 3])

    t = threading.Thread(target=change)
    t.start()
    try:
        got = [pk.paged_merge_states(states)[0] for _ in range(300)]
    finally:
        stop.set()
        t.join()
    torch.cuda.synchronize()
    for x in got:
        assert any(torch.equal(x, y) for y in want.values())
