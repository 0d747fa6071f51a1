"""The scaled cache's append, decode and prefill and the windowed attention under
conditions that cut across them: the range-checking debug build, caches whose
offsets pass 32 bits, calls on two streams at once, empty batches and lengths,
waits that run out."""
from __future__ import annotations

import pytest
import torch

import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import binding
from paged_kv_cache_316_gb300 import build as pk_build
from paged_kv_cache_316_gb300 import workloads as wl
import test_gpu_append_scaled as ta
import test_gpu_decode_window as td
import test_gpu_prefill_window as tp

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TIMEOUT = 16


@pytest.fixture
def debug_library():
    binding.load_library(pk_build.build(debug_bounds=True))
    assert binding.debug_bounds()
    yield
    binding.load_library(binding.library_path())
    assert not binding.debug_bounds()


def test_debug_build_finds_nothing_out_of_range(debug_library):
    # (each of these requires the error word to be 0, or only the named bit)
    ta.test_bits([5, 40, 1, 0, 17], [3, 0, 31, 9, 64], 32, 8, 3, 128, wl.NHD, torch.float16, "tuple", 3)
    ta.test_bits([100, 257, 2], [0, 13, 255], 256, 256, 2, 128, wl.HND, torch.bfloat16, "5d", 4)
    ta.test_bits([70, 3], [2, 29], 128, 64, 5, 16, wl.NHD, torch.bfloat16, "5d", 6)
    for c in td.WINDOW:
        td.test_window_with_first_tokens(c)
    for c in td.SCALED:
        td.test_block_scales(c)
    for scaled in (False, True):
        td.test_variable_length_queries(scaled)
    for c in tp.WINDOW:
        tp.test_window_with_first_tokens(c)
    for c in tp.SCALED:
        tp.test_block_scales(c)
    tp.test_contiguous_keys_and_batch_offsets()


def _session(P, first_page, k, v, q):
    """Append 40 tokens of two requests, then decode and prefill over them, on
    the pages first_page .. of a pool of P pages."""
    S, H, G = 64, 8, 16
    cache = torch.empty(P, 2, H, S, 128, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.ones(P, 2, H, S // G, device=DEV)  # (blocks that no call writes are compared too)
    idx = torch.tensor([first_page + 1, first_page], dtype=torch.int32, device=DEV)
    ptr, last = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1, 2], [30, 10]))
    seq = pk.paged_seq_lens(ptr, last, S)
    bi, pos = pk.paged_batch_indices_positions(torch.tensor([0, 30, 40], dtype=torch.int32, device=DEV), seq, 40)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.paged_append_scaled(k, v, bi, pos, cache, scales, idx, ptr, last, kv_layout="HND", err_word=err)
    table = idx.view(2, 1).contiguous()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = [pk.paged_decode(q[:2], cache, ws, table, seq, 30, bmm1_scale=0.1, kv_scales=scales, first_tokens=2,
                           window_left=20, err_word=err)]
    n = pk.paged_prefill_scaled_workspace_size(2, 16, H, 30, 30, 128, 128)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out += pk.paged_prefill(q, cache[:, 0], cache[:, 1], 0.1, ws, 30, 30, seq, seq, table, kv_scales=scales,
                            window_left=9, first_tokens=3, err_word=err)
    out.append(scales[first_page:first_page + 2].clone())
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def test_offsets_beyond_32_bits():
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    k, v = (torch.randn(40, 8, 128, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(40, 16, 128, device=DEV, generator=g).to(torch.bfloat16)
    small = _session(4, 1, k, v, q)
    P = 40000  # 131072 bytes a page: 5.2 GB
    large = _session(P, P - 2, k, v, q)
    for a, b in zip(small, large):
        assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    cs = [td.make([3000, 700], 16, 16, 2, wl.HND, torch.bfloat16, 50 + i, scaled=True, G=16, window=2000, first=8)
          for i in range(2)]
    want = [td.call(c, 0.05) for c in cs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = pk.paged_decode_workspace_size(2, 1, 16, 2, 128, 3000, 16, 2000, first_tokens=8)
    args = []
    for c in cs:
        args.append([c["query"].to(DEV), c["pool"].to(DEV), torch.empty(max(1, n), dtype=torch.uint8, device=DEV),
                     c["table"].to(DEV), torch.tensor(c["lens"], dtype=torch.int32, device=DEV), c["scales"].to(DEV),
                     torch.empty_like(c["query"], device=DEV), torch.empty(2, 16, device=DEV)])
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (q, pool, ws, table, lens, sc, out, lse) in zip(streams, args):
            pk.paged_decode(q, pool, ws, table, lens, 3000, bmm1_scale=0.05, window_left=2000, kv_layout="HND",
                            first_tokens=8, kv_scales=sc, out=out, lse=lse, stream=s)
    torch.cuda.synchronize()
    for (o, l), a in zip(want, args):
        assert torch.equal(o, a[6]) and torch.equal(l, a[7])


@pytest.mark.parametrize("B", [0, 3])
def test_no_keys_and_no_requests(B):
    S, H = 16, 2
    cache = torch.zeros(2, 2, H, S, 128, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.ones(2, 2, H, 1, device=DEV)
    zeros = torch.zeros(B, dtype=torch.int32, device=DEV)
    table = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    q = torch.randn(B, 4, 128, device=DEV).to(torch.bfloat16)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    lse = torch.zeros(B, 4, device=DEV)
    sinks = torch.randn(4, device=DEV)
    for kw in (dict(kv_scales=scales), dict(kv_scales=scales, window_left=5, first_tokens=2)):
        out = pk.paged_decode(q, cache, ws, table, zeros, 0, kv_layout="HND", lse=lse, **kw)
        assert (out == 0).all() and torch.isneginf(lse).all()
        out = pk.paged_decode(q, cache, ws, table, zeros, 0, kv_layout="HND", lse=lse, sinks=sinks, **kw)
        assert (out == 0).all() and ((lse - sinks).abs() <= 2.0 ** -20 * (1 + sinks.abs())).all()
    pk.paged_append_scaled(torch.empty(0, H, 128, dtype=torch.bfloat16, device=DEV),
                           torch.empty(0, H, 128, dtype=torch.bfloat16, device=DEV), zeros[:0], zeros[:0], cache, scales,
                           zeros[:0], torch.zeros(B + 1, dtype=torch.int32, device=DEV), zeros, kv_layout="HND")
    if B:
        ones = torch.ones(B, dtype=torch.int32, device=DEV)
        n = pk.paged_prefill_scaled_workspace_size(B, 4, H, 1, 0, 128, 128)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        out, lse = pk.paged_prefill(q, cache[:, 0], cache[:, 1], 0.1, ws, 1, 0, ones, zeros, table, kv_scales=scales)
        assert (out == 0).all() and torch.isneginf(lse).all()
    torch.cuda.synchronize()


def test_a_wait_that_runs_out_in_a_windowed_prefill():
    c = tp.make([300], [900], 16, 4, 2, 128, wl.HND, torch.bfloat16, 60, 200, 6)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.set_wait_limit_ns(1)
    try:
        tp.call(c, 0.05, err)
    finally:
        pk.set_wait_limit_ns(0)
    assert int(err.item()) & TIMEOUT
    tp.compare(c, *tp.call(c, 0.05), 0.05)
