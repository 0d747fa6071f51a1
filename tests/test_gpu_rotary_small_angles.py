"""Rotations by small angles: an element that the rotation alone brings in,
x sin a beside a zero, is right in itself, not just beside its partner.

Bound: the angle in 2^-64 turns is off by at most 2^-65 turn a step, its fp32
form by 2^-24 of itself, sine and magnitude by 3 * 2^-23, then one rounding."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_cache_316_gb300 as pk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("f0", [1e-3, 1e-6, 3e-7, 1e-8, -2e-8])
def test_sines_of_small_angles(f0, paired):
    pos = torch.tensor([1, 2, 3, 7, -1, -5, 1000], dtype=torch.int32)
    f = f0 * (1 + torch.arange(8, dtype=torch.float64) / 7)
    x = torch.zeros(len(pos), 2, 16, dtype=torch.bfloat16)
    u, v = (slice(0, None, 2), slice(1, None, 2)) if paired else (slice(0, 8), slice(8, 16))
    x[:, 0, u], x[:, 1, v] = 1.0, 1.0
    out, _ = pk.paged_rotary(x.to(DEV), x.to(DEV), pos.to(DEV), f.to(DEV), interleaved=paired, magnitude=1.5)
    out = out.cpu().double()
    a = pos.double()[:, None] * f
    room = (2.0 ** -8 + 2.0 ** -20) * 1.5 * a.abs() + 2 * math.pi * 1.5 * 2.0 ** -65 * pos.double().abs()[:, None]
    for got, want in ((out[:, 0, v], 1.5 * torch.sin(a)), (out[:, 1, u], -1.5 * torch.sin(a))):
        assert ((got - want).abs() <= room).all(), ((got - want).abs() / want.abs()).max()
    assert ((out[:, 0, u] - 1.5 * torch.cos(a)).abs() <= 1.5 * 2.0 ** -8).all()


def test_small_angles_of_far_positions():
    # whole turns and a little: 2^-30 of a turn beyond, of a frequency that float64 and the 2^-64 count hold exactly
    f = torch.full((8,), 2 * math.pi * 2.0 ** -30, dtype=torch.float64)
    turns = f * (1 / (2 * math.pi))
    assert (turns == 2.0 ** -30).all()
    pos = torch.tensor([2 ** 30 + 1, 2 ** 30 - 1, -2 ** 30 + 3], dtype=torch.int32)
    x = torch.zeros(3, 1, 16, dtype=torch.bfloat16)
    x[:, :, :8] = 1.0
    out, _ = pk.paged_rotary(x.to(DEV), x.to(DEV), pos.to(DEV), f.to(DEV))
    want = torch.sin(2 * math.pi * 2.0 ** -30 * torch.tensor([1.0, -1.0, 3.0], dtype=torch.float64))[:, None]
    got = out[:, 0, 8:].cpu().double()
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all()
