"""More of decode over shared prefixes under the range-checking build: more
than 32 groups, more items than CTAs, records that are written again, values
that some tokens do not see, workspaces and batches of other sizes."""
from __future__ import annotations

import math

import pytest
import torch

import test_gpu_shared_errors as errors
import test_gpu_shared_hidden as hidden
import test_gpu_shared_paths as paths
import test_gpu_shared_ring as ring
import test_gpu_shared_workspace as workspace
from paged_kv_cache_316_gb300 import binding
from paged_kv_cache_316_gb300 import build as pk_build
from paged_kv_cache_316_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def debug_library():
    binding.load_library(pk_build.build(debug_bounds=True))
    assert binding.debug_bounds()
    yield
    binding.load_library(binding.library_path())
    assert not binding.debug_bounds()


def test_more_than_32_groups():
    paths.test_more_than_32_groups()  # (all of these assert the error word)


def test_more_items_than_ctas():
    paths.test_more_items_than_ctas()


def test_long_prefixes_in_teams_of_several_groups():
    paths.test_long_prefixes_in_teams(70, 1, 64, [3, 60, 7])


@pytest.mark.parametrize("S,q,dtype", [(8, 4, torch.float16), (64, 2, torch.bfloat16)])
def test_records_that_are_written_again(S, q, dtype):
    ring.test_records_that_are_written_again(S, wl.NHD if S == 8 else wl.HND, q, dtype)


@pytest.mark.parametrize("i", range(len(hidden.CASES)))
def test_values_that_some_tokens_do_not_see(i):
    hidden.test_values_that_some_tokens_do_not_see(*hidden.CASES[i], math.nan)


def test_one_workspace_for_all_sizes():
    workspace.test_one_workspace_for_all_sizes()


def test_no_prefix_has_a_key():
    errors.test_no_prefix_has_a_key(40)
