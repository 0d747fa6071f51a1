"""One token's rows cut out of wider ones: the distance to a next token that
is not there refuses nothing."""
from __future__ import annotations

import pytest
import torch

import paged_kv_cache_316_gb300 as pk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("width", [12 * 64, 12 * 64 + 4, 12 * 64 + 1, 1])
def test_rows_of_one_token(width):
    g = torch.Generator(device=DEV).manual_seed(3)
    row = torch.randn(12 * 64, generator=g, device=DEV).to(torch.bfloat16)
    parts = row.view(1, 12, 64).split((8, 2, 2), dim=1)
    far = [p.as_strided(p.shape, (width, 64, 1)) for p in parts]  # the stride of a row of `width`
    pos, f = torch.tensor([5], dtype=torch.int32, device=DEV), torch.full((32,), 0.1, dtype=torch.float64, device=DEV)
    a, b = pk.paged_rotary(*parts[:2], pos, f), pk.paged_rotary(*far[:2], pos, f)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    i = torch.zeros(1, dtype=torch.int32, device=DEV)
    caches = [torch.zeros(2, 2, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for (q, k, v), c in zip((parts, far), caches):
        pk.paged_append_rotary(q, k, v, i, pos, c, torch.arange(2, dtype=torch.int32, device=DEV),
                               torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                               torch.tensor([16], dtype=torch.int32, device=DEV), f)
    assert torch.equal(caches[0], caches[1]) and (caches[0][0, 1, 5] == parts[2][0]).all()
