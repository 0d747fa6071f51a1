"""What rotated appends, decode over shared prefixes and the merge refuse, with
tensors of the GPU; and that results handed in are the ones handed back."""
from __future__ import annotations

import sys

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from test_gpu_decode_shared import args, check, make

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = dict(dtype=torch.int32, device=DEV)


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def append_args():
    i = torch.zeros(4, **I32)
    return dict(query=zeros(4, 32, 128), key=zeros(4, 8, 128), value=zeros(4, 8, 128), batch_indices=i,
                positions=torch.arange(4, **I32), paged_kv_cache=zeros(4, 2, 16, 8, 128), kv_indices=torch.arange(4, **I32),
                kv_indptr=torch.tensor([0, 4], **I32), kv_last_page_len=torch.tensor([16], **I32),
                frequencies=torch.ones(64, dtype=torch.float64, device=DEV))


@pytest.mark.parametrize("over", [
    lambda a: dict(kv_layout="HND"), lambda a: dict(value=a["value"][:3]), lambda a: dict(value=a["value"].half()),
    lambda a: dict(paged_kv_cache=a["paged_kv_cache"].half()), lambda a: dict(paged_kv_cache=a["paged_kv_cache"][:, :1]),
    lambda a: dict(paged_kv_cache=a["paged_kv_cache"].transpose(2, 3)),
    lambda a: dict(paged_kv_cache=(zeros(4, 16, 8, 128), zeros(4, 16, 8, 64))),
    lambda a: dict(paged_kv_cache=(zeros(4, 16, 8, 128), zeros(4, 16, 8, 128, dtype=torch.half))),
    lambda a: dict(paged_kv_cache=(zeros(4, 16, 8, 128),)), lambda a: dict(positions=a["positions"].cpu()),
    lambda a: dict(query=a["query"].cpu()), lambda a: dict(kv_indptr=a["kv_indptr"][:1]),
    lambda a: dict(rotary_positions=a["positions"][:3]), lambda a: dict(err_word=torch.zeros(1, dtype=torch.int32)),
    lambda a: dict(query_weight=zeros(64)), lambda a: dict(key_weight=zeros(128, dtype=torch.half)),
    lambda a: dict(query_out=zeros(4, 32, 64)), lambda a: dict(rotary_start=8), lambda a: dict(eps=-1.0),
    lambda a: dict(frequencies=a["frequencies"].float()),
])
def test_append_rotary(over):
    a = append_args()
    pk.paged_append_rotary(**a)  # as it is, it runs
    with pytest.raises(pk.PagedKVError):
        pk.paged_append_rotary(**dict(a, **over(a)))


@pytest.mark.parametrize("over", [
    lambda a: dict(query=a["query"][1:]), lambda a: dict(query=a["query"].half()), lambda a: dict(query=a["query"].cpu()),
    lambda a: dict(kv_layout="NHD"), lambda a: dict(kv_cache=a["kv_cache"].half()), lambda a: dict(q_len_per_req=2),
    lambda a: dict(group_indptr=a["group_indptr"][:1]), lambda a: dict(prefix_lens=a["prefix_lens"].long()),
    lambda a: dict(max_prefix_len=1 << 20), lambda a: dict(max_seq_len=1 << 20), lambda a: dict(block_tables=a["block_tables"][:1]),
    lambda a: dict(prefix_tables=a["prefix_tables"].float()), lambda a: dict(workspace=a["workspace"][:256]),
    lambda a: dict(workspace=a["workspace"][1:]), lambda a: dict(out=a["out"].float()), lambda a: dict(lse=a["lse"].half()),
    lambda a: dict(sinks=torch.zeros(3, device=DEV)), lambda a: dict(bmm1_scale=torch.ones(2, device=DEV)),
    lambda a: dict(bmm2_scale=torch.ones(1)), lambda a: dict(max_prefix_len=-1), lambda a: dict(seq_lens=a["seq_lens"].long()),
])
def test_decode_shared(over):
    a = args(make([40], [2], [3, 5], H=4, Hq=8, seed=51))
    pk.paged_decode_shared(**a)
    with pytest.raises(pk.PagedKVError):
        pk.paged_decode_shared(**dict(a, **over(a)))


def test_merge_states():
    o, l = zeros(4, 32, 128), torch.zeros(4, 32, device=DEV)
    pk.paged_merge_states([(o, l)])
    for states, kw in (([(o, l), (o.half(), l)], {}), ([(o, l.cpu())], {}), ([(o, l), (o, l.half())], {}), ([(o, l)] * 17, {}),
                       ([(o, l)], dict(out=o.cpu())), ([(o, l)], dict(lse=l[:3])), ([(o[..., ::2], l)], {})):
        with pytest.raises(pk.PagedKVError):
            pk.paged_merge_states(states, **kw)


def test_results_and_references():
    c = make([40], [2], [3, 5], seed=52)
    a = args(c)
    count = sys.getrefcount(a["out"])
    same = all([pk.paged_decode_shared(**a) is a["out"] for _ in range(20)])  # (an assert in a loop holds its last operand)
    now = sys.getrefcount(a["out"])
    assert same and now == count
    del a["out"]
    out = pk.paged_decode_shared(**a)
    now = sys.getrefcount(out)
    assert now == 2 and out.device == DEV
    check(c, out, a["lse"])
    q, k = zeros(3, 8, 64), zeros(3, 2, 64)
    f, pos = torch.ones(32, dtype=torch.float64, device=DEV), torch.zeros(3, **I32)
    x, y = pk.paged_rotary(q, k, pos, f, query_out=q, key_out=k)
    assert x is q and y is k
    x, y = pk.paged_rotary(q, k, pos, f)
    now = sys.getrefcount(x)
    assert now == 2 and x.shape == q.shape and y.shape == k.shape and x.dtype == q.dtype


def test_the_stream_of_the_context():
    c = make([600], [10], [1 + i * 9 for i in range(10)], seed=53)
    a = args(c)
    want = pk.paged_decode_shared(**a).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a["out"].zero_()
        pk.paged_decode_shared(**a)
    side.synchronize()
    assert torch.equal(a["out"], want)
    a["out"].zero_()
    torch.cuda.synchronize()
    pk.paged_decode_shared(**a, stream=side.cuda_stream)  # a handle
    side.synchronize()
    assert torch.equal(a["out"], want)
