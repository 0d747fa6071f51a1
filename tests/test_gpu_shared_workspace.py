"""One workspace, reserved for the largest of everything, under shared decodes
of many sizes: each is right, and nothing behind the workspace is touched."""
from __future__ import annotations

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_decode_shared import args, check, make

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HEADS = dict(Hq=16, H=2)


def test_one_workspace_for_all_sizes():
    n = pk.paged_decode_shared_workspace_size(70, 4, 16, 2, 128, 12, 5000, 1500, 16)
    room = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    for i, (prefix, sizes, lens, q) in enumerate([
            ([5000], [70], [4 + (j * 37) % 1400 for j in range(70)], 4),
            ([5000], [20], [1 + (j * 37) % 300 for j in range(20)], 1),
            ([90] * 12, [5] * 12, [4 + j % 7 for j in range(60)], 3),
            ([1], [1], [1], 1),
            ([], [], [1 + (j * 91) % 1500 for j in range(70)], 1),
            ([700, 33], [3, 60], [2 + j % 90 for j in range(70)], 2)]):
        c = make(prefix, sizes, lens, q=q, seed=80 + i, layout=wl.NHD if i % 2 else wl.HND, **HEADS)
        a = args(c)
        need = a["workspace"].numel()
        assert need <= n
        for ws in (room[:n], room[:need]):  # as reserved; no more than asked for
            room.fill_(0xFF)
            a["workspace"] = ws
            pk.paged_decode_shared(**a)
            torch.cuda.synchronize()
            assert int(a["err_word"].item()) == 0
            check(c, a["out"], a["lse"], requests=sorted({0, len(lens) // 2, len(lens) - 1}))
            assert (room[ws.numel():] == 0xFF).all()
