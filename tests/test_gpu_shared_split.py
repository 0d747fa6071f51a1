"""How a shared decode divides the SMs between the prefixes and the requests'
own keys: by the work of the whole batch, in whatever order its requests come.
The prefix kernel leaves the steps that each of its teams takes in the last 256
bytes of the workspace, for the kernel that joins the partials."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_cache_316_gb300 as pk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = dict(dtype=torch.int32, device=DEV)


def teams(lens, P, steps):
    """Teams (of one CTA) that the prefix's steps are dealt to: its steps over those of a team."""
    S, Hq, B = 16, 4, len(lens)
    need = [-(-n // S) for n in lens]
    first = -(-P // S)
    g = torch.Generator(device=DEV).manual_seed(5)
    pool = torch.randn(first + sum(need), 2, 1, S, 128, generator=g, device=DEV).to(torch.bfloat16)
    tables = torch.full((B, max(need)), 0x7FFFFFFF, dtype=torch.int32)
    at = first
    for i, n in enumerate(need):
        tables[i, :n] = torch.arange(at, at + n)
        at += n
    n = pk.paged_decode_shared_workspace_size(B, 1, Hq, 1, 128, 1, P, max(lens), S)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = pk.paged_decode_shared(torch.randn(B, Hq, 128, generator=g, device=DEV).to(torch.bfloat16), pool, ws,
                                 torch.arange(first, **I32)[None], torch.tensor([P], **I32), torch.tensor([0, B], **I32), P,
                                 tables.to(DEV), torch.tensor(lens, **I32), max(lens), bmm1_scale=0.09)
    assert out.isfinite().all()
    return steps / int(ws[n - 256:n - 252].view(torch.int32).item())


@pytest.mark.parametrize("B", [200, 256, 257, 300, 511, 700])
def test_the_order_of_the_requests_does_not_matter(B):
    P = 8192
    lens = [16 + 880 * i // (B - 1) for i in range(B)]  # ascending: the long ones come last
    steps = -(-B // 64) * (P // 128)  # tiles of 64 tokens (4 heads to a kv head, two blocks of 128 rows)
    # both kernels end together: C N^2 + (W + A - C S) N - W S = 0 (shared_prefix.cuh), A in steps of 128 own keys
    S, C, A = torch.cuda.get_device_properties(DEV).multi_processor_count, 5.0, sum(lens) / 128
    b = steps + A - C * S
    want = (math.sqrt(b * b + 4 * C * steps * S) - b) / (2 * C)
    for order in (lens, lens[::-1], lens[::2] + lens[1::2]):
        got = teams(order, P, steps)
        # (teams and their steps are whole numbers: n teams take ceil(W / n) steps)
        low, high = steps / math.ceil(steps / math.floor(want * 0.97)), steps / math.ceil(steps / math.ceil(want * 1.03))
        assert low - 1e-6 <= got <= high + 1e-6, (got, want)
