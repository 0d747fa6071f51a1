"""Rotated appends, decode over shared prefixes and merged states under the
range-checking build of the library: every offset that their kernels derive is
checked before the access, and none may be out of range."""
from __future__ import annotations

import pytest
import torch

import test_gpu_decode_shared as shared
import test_gpu_rotary as rotary
import test_gpu_shared_paths as paths
from paged_kv_cache_316_gb300 import binding
from paged_kv_cache_316_gb300 import build as pk_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def debug_library():
    binding.load_library(pk_build.build(debug_bounds=True))
    assert binding.debug_bounds()
    yield
    binding.load_library(binding.library_path())
    assert not binding.debug_bounds()


@pytest.mark.parametrize("i", range(len(shared.CASES)))
def test_decode_shared(i):
    shared.test_decode_shared(i)  # (asserts the error word)


@pytest.mark.parametrize("S", [8, 16, 64, 256])
def test_pages_with_gaps(S):
    paths.test_pages_with_gaps(S, 0 if S == 16 else 1, 8)


def test_long_prefixes_in_teams():
    paths.test_long_prefixes_in_teams(70, 1, 64, [33])


def test_own_keys_in_splits():
    paths.test_own_keys_in_splits(64, 16, 2, 8, torch.bfloat16)


def test_pools_past_32_bits():
    paths.test_pools_past_32_bits()


@pytest.mark.parametrize("i", range(len(rotary.APPENDS)))
def test_append_rotary(i):
    rotary.test_append_rotary(i)
