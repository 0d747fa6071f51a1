"""The frequencies of rotations scaled for contexts longer than the trained
one, pair by pair: the ramp of "yarn" is linear in the pair's index between
rounded ends, which is what models trained with it were given."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_cache_316_gb300 as pk


def yarn(rotary_dim, base, factor, trained_len, fast=32.0, slow=1.0):
    """The definition, one pair at a time."""
    def pair_that_turns(r):
        return rotary_dim * math.log(trained_len / (r * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(pair_that_turns(fast)), 0), min(math.ceil(pair_that_turns(slow)), rotary_dim - 1)
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2 * i / rotary_dim)
        ramp = min(max((i - low) / (high - low if high != low else 0.001), 0.0), 1.0)
        out.append(f / factor * ramp + f * (1 - ramp))
    return out


@pytest.mark.parametrize("rotary_dim,base,factor,trained_len", [
    (128, 1e6, 4.0, 32768), (64, 1e4, 40.0, 4096), (128, 1e4, 8.0, 4096), (128, 5e5, 8.0, 8192), (96, 1e4, 32.0, 2048),
    (16, 1e4, 2.0, 1024), (2, 1e4, 2.0, 1024), (64, 1e4, 1.0, 4096), (64, 10.0, 4.0, 100), (64, 1e4, 4.0, 7),
])
def test_yarn(rotary_dim, base, factor, trained_len):
    f, m = pk.rotary_frequencies(rotary_dim, base, "yarn", factor=factor, trained_len=trained_len, device="cpu")
    want = yarn(rotary_dim, base, factor, trained_len)
    assert m == pytest.approx(0.1 * math.log(factor) + 1) and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor(want, dtype=torch.float64), rtol=1e-13, atol=0)


def test_yarn_in_numbers():
    # 64 pairs, base 10^6: 32 turns over 32768 positions between pairs 23 and 24, one turn between 39 and 40
    f, _ = pk.rotary_frequencies(128, 1e6, "yarn", factor=4.0, trained_len=32768, device="cpu")
    plain, _ = pk.rotary_frequencies(128, 1e6, device="cpu")
    got = f / plain
    assert (got[:24] == 1).all() and torch.allclose(got[40:], torch.tensor(0.25, dtype=torch.float64), rtol=1e-15)
    for i in range(23, 41):
        assert got[i].item() == pytest.approx(1 - 0.75 * (i - 23) / 17, rel=1e-12)


def test_other_ends():
    f, _ = pk.rotary_frequencies(128, 1e4, "yarn", factor=4.0, trained_len=4096, fast=64.0, slow=4.0, device="cpu")
    assert torch.allclose(f, torch.tensor(yarn(128, 1e4, 4.0, 4096, 64.0, 4.0), dtype=torch.float64), rtol=1e-13, atol=0)
    for bad in (dict(base=1.0), dict(base=0.5), dict(slow=0.0), dict(slow=-1.0), dict(trained_len=0)):
        with pytest.raises(pk.PagedKVError):
            pk.rotary_frequencies(64, **{**dict(base=1e4, scaling="yarn", factor=2.0, trained_len=4096, device="cpu"), **bad})
