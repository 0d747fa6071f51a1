"""Scales that are not on a float's boundary are refused by every entry point
that reads them (host checks: the fake pointers are never used)."""
from __future__ import annotations

import pytest

import test_scaled_cache_cpu as sc
from test_abi_cpu import lib  # noqa: F401  (the built library, a fixture)


@pytest.mark.parametrize("call", [sc._append, sc._decode, sc._prefill])
@pytest.mark.parametrize("over", [dict(ks=0x1002), dict(vs=0x1001)])
def test_scales_off_a_float_boundary_are_refused(lib, call, over):  # noqa: F811
    assert call(lib, **over) == 2
