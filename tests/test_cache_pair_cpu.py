"""What the binding refuses in a (K, V) tuple of caches before the library is
called (host checks)."""
from __future__ import annotations

import pytest
import torch


class _OnGpu0:
    """A tensor of the CPU that says it is on GPU 0 (host checks: never used)."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.mark.parametrize("v", [
    torch.zeros(4, 8, 16, 128, dtype=torch.float8_e4m3fn),            # on the CPU
    _OnGpu0(torch.zeros(4, 8, 16, 128, dtype=torch.bfloat16)),        # twice the bytes
    _OnGpu0(torch.zeros(4, 8, 16, 128, dtype=torch.uint8)),
])
def test_a_value_cache_unlike_the_key_cache_is_refused(v):
    import paged_kv_cache_316_gb300 as pk
    k = _OnGpu0(torch.zeros(4, 8, 16, 128, dtype=torch.float8_e4m3fn))
    new = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    bt, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    q, ws = torch.zeros(2, 32, 128, dtype=torch.bfloat16), torch.zeros(1 << 16, dtype=torch.uint8)
    sc = torch.ones(4, 2, 8, 1)
    for call in (lambda: pk.paged_append_scaled(new, new, i, i, (k, v), sc, i, torch.zeros(3, dtype=torch.int32), i,
                                                kv_layout="HND"),
                 lambda: pk.paged_append(new, new, i, i, (k, v), i, torch.zeros(3, dtype=torch.int32), i, kv_layout="HND"),
                 lambda: pk.paged_decode(q, (k, v), ws, bt, lens, 16, kv_scales=sc),
                 lambda: pk.paged_decode(q, (k, v), ws, bt, lens, 16)):
        with pytest.raises(pk.PagedKVError, match="same type on the same device"):
            call()
