"""Groups that are wrong are flagged in every call of a shared decode, also in
one that says that no prefix has a key."""
from __future__ import annotations

import pytest
import torch

from test_gpu_decode_shared import BATCH, DEV, I32, LEN, PAGE, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [1, 2, 40])
def test_no_prefix_has_a_key(groups):
    sizes = [1] * groups
    c = make([0] * groups, sizes, [1 + i % 30 for i in range(groups + 2)], seed=groups)
    out, lse, err = run(c)
    assert err == 0
    check(c, out, lse, requests=[0, groups, groups + 1])

    def same(want, **over):
        got = run(c, **{k: torch.tensor(v, device=DEV, **I32) for k, v in over.items()})
        assert got[2] == want and torch.equal(got[0], out) and torch.equal(got[1], lse), over

    at = [int(x) for x in c["indptr"]]
    same(BATCH, group_indptr=[1] + at[1:])
    same(BATCH, group_indptr=at[:-1] + [groups + 3])
    same(BATCH, group_indptr=at[:-1] + [-1])
    same(LEN, prefix_lens=[0] * (groups - 1) + [5])
    same(LEN, prefix_lens=[-2] + [0] * (groups - 1))


def test_a_prefix_has_keys():
    c = make([30, 0], [2, 2], [3, 4, 5, 6, 7], seed=1)
    # (31 is clamped to 30 keys, for which the second group's table has no pages)
    for over, want in ((dict(prefix_lens=[30, 31]), LEN | PAGE), (dict(prefix_lens=[30, -1]), LEN),
                       (dict(group_indptr=[0, 5, 4]), BATCH)):
        assert run(c, **{k: torch.tensor(v, device=DEV, **I32) for k, v in over.items()})[2] == want
