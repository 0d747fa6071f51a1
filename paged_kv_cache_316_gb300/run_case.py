"""Run one operation of the library on its named synthetic workload.

    python -m paged_kv_cache_316_gb300.run_case --op prefill [--d-qk 128] [--iters 3] [--kv-dtype e4m3]
                                                [--contiguous]
    python -m paged_kv_cache_316_gb300.run_case --op decode_llama | decode_long | decode_varlen | append
                                                [--batch N] [--iters 3] [--kv-dtype e4m3]
    python -m paged_kv_cache_316_gb300.run_case --op append_scaled | decode_scaled | decode_window | prefill_window
                                                [--batch N] [--iters 3] [--d-qk 128] [--q-len 1]

    python -m paged_kv_cache_316_gb300.run_case --op append_rotary | decode_shared | merge_states
                                                [--batch N] [--iters 3] [--q-len 1] [--prefix 8192]

The third line's operators on the same workloads: the append sweep into an
E4M3 cache with a scale for each 16 tokens and head; the Llama-shaped decode
over such a cache (--q-len tokens a request); the long-context decode with 64
first tokens that stay visible; the ragged prefill under a window of 1024 keys
with 4 first tokens.  The fourth's: the append sweep with 32 query heads,
norms and rotations; a decode of requests with up to 1024 keys of their own
behind one shared prefix; 8192 rows from two parts of their keys.

Used to drive profilers (ncu) on one kernel at a size that keeps a capture
short; it prints the mean CUDA-event time per call, which is informational
only (the benchmark is bench.py).
"""
from __future__ import annotations

import argparse
import json

import torch

from . import binding as pk
from . import workloads as wl


def long_session_op(a, dev):
    """The append, decode and prefill of long sessions on the named workloads."""
    g = wl.generator(9, dev)

    def scales(c):  # about 2^-7, as N(0, 1) values filling E4M3's range have
        p = c.pool
        return torch.exp2(torch.randint(-8, -5, (p.num_pages, 2, p.num_heads, 1), generator=g, device=dev).float())

    if a.op == "append_scaled":
        c = wl.append_sweep(a.batch or 4096, seed=1, layout=wl.NHD, device=dev, fill="empty", dtype=wl.BF16)
        cache = torch.zeros(c.pool.storage[0].shape, dtype=torch.float8_e4m3fn, device=dev)
        kvi, kvp, last = (x.to(dev) for x in (c.kv_indices, c.kv_indptr, c.kv_last_page_len))
        bi, pos = pk.paged_batch_indices_positions(c.append_indptr.to(dev), pk.paged_seq_lens(kvp, last, 16),
                                                   c.append_key.shape[0])
        sc = scales(c)
        return lambda: pk.paged_append_scaled(c.append_key, c.append_value, bi, pos, cache, sc, kvi, kvp, last,
                                              kv_layout="NHD")
    if a.op == "prefill_window":
        c = wl.ragged_prefill(d_qk=a.d_qk, device=dev)
        ws = torch.empty(pk.paged_prefill_workspace_size(16, 32, c.max_q, c.max_kv), dtype=torch.uint8, device=dev)
        lq, lkv, bt = c.seq_lens_q.to(dev), c.seq_lens_kv.to(dev), c.block_tables.to(dev)
        return lambda: pk.paged_prefill(c.q, c.pool.k, c.pool.v, c.scale, ws, c.max_q, c.max_kv, lq, lkv, bt,
                                        kv_layout="HND", window_left=1023, first_tokens=4)
    if a.op == "decode_scaled":
        L = wl.uniform_lengths(wl.generator(0), 64, 512, 8192)[:a.batch or 64]
        c = wl.decode_case(L, 16, 32, 8, 128, wl.HND, wl.BF16, device=dev, bt_width=512, kv_dtype=wl.E4M3,
                           q_len_per_req=a.q_len)
        kw = dict(kv_scales=scales(c), first_tokens=0)
    else:
        L = wl.lognormal_lengths(wl.generator(0), 256, 4096.0, 1.0, 4, 32768)[:a.batch or 256]
        c = wl.decode_case(L, 64, 64, 8, 128, wl.HND, wl.BF16, q_len_per_req=4, window_left=4095, with_sinks=True,
                           device=dev, bt_width=512)
        kw = dict(first_tokens=64)
    n = pk.paged_decode_workspace_size(len(L), c.q_len_per_req, c.num_qo_heads, c.num_kv_heads, 128, c.max_seq_len,
                                       c.pool.page_size, c.window_left, first_tokens=kw["first_tokens"])
    ws = torch.empty(max(1, n), dtype=torch.uint8, device=dev)
    bt, sl, sinks = (None if x is None else x.to(dev) for x in (c.block_tables, c.seq_lens, c.sinks))
    return lambda: pk.paged_decode(c.query, c.pool.storage[0], ws, bt, sl, c.max_seq_len, bmm1_scale=c.bmm1_scale,
                                   window_left=c.window_left, sinks=sinks, kv_layout=c.pool.layout,
                                   q_len_per_req=c.q_len_per_req, **kw)


def prefix_op(a, dev):
    """Rotated append, decode over a shared prefix, merged states."""
    g = wl.generator(10, dev)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    if a.op == "append_rotary":
        c = wl.append_sweep(a.batch or 1024, seed=1, layout=wl.NHD, device=dev, fill="empty", dtype=wl.BF16)
        kvi, kvp, last = (x.to(dev) for x in (c.kv_indices, c.kv_indptr, c.kv_last_page_len))
        n = c.append_key.shape[0]
        bi, pos = pk.paged_batch_indices_positions(c.append_indptr.to(dev), pk.paged_seq_lens(kvp, last, 16), n)
        q, w = rand(n, 32, 128), rand(2, 128)
        f, magnitude = pk.rotary_frequencies(128, 500000.0, device=dev)
        return lambda: pk.paged_append_rotary(q, c.append_key, c.append_value, bi, pos, c.pool.storage[0], kvi, kvp, last,
                                              f, kv_layout="NHD", magnitude=magnitude, query_weight=w[0], key_weight=w[1])
    if a.op == "merge_states":
        parts = [(rand(8192, 32, 128), torch.randn(8192, 32, generator=g, device=dev)) for _ in range(2)]
        return lambda: pk.paged_merge_states(parts)
    B, P, S, Q = a.batch or 64, a.prefix, 16, a.q_len
    L = wl.uniform_lengths(wl.generator(0), B, 64, 1024)
    need = [-(-n // S) for n in [P] + L]
    ids = torch.randperm(sum(need), generator=g, device=dev).to(torch.int32)
    table, at = torch.zeros(1 + B, max(need), dtype=torch.int32, device=dev), 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    cache, q = rand(sum(need), 2, 8, S, 128), rand(B * Q, 32, 128)
    i32 = dict(dtype=torch.int32, device=dev)
    ws = torch.empty(pk.paged_decode_shared_workspace_size(B, Q, 32, 8, 128, 1, P, 1024, S), dtype=torch.uint8, device=dev)
    plen, groups, lens = torch.tensor([P], **i32), torch.tensor([0, B], **i32), torch.tensor(L, **i32)
    return lambda: pk.paged_decode_shared(q, cache, ws, table[:1], plen, groups, P, table[1:], lens, 1024,
                                          bmm1_scale=128 ** -0.5, q_len_per_req=Q)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", required=True,
                    choices=["prefill", "decode_llama", "decode_long", "decode_varlen", "append", "append_scaled",
                             "decode_scaled", "decode_window", "prefill_window", "append_rotary", "decode_shared",
                             "merge_states"])
    ap.add_argument("--q-len", type=int, default=1, help="decode_scaled, decode_shared: query tokens per request")
    ap.add_argument("--prefix", type=int, default=8192, help="decode_shared: keys of the shared prefix")
    ap.add_argument("--d-qk", type=int, default=128)
    ap.add_argument("--batch", type=int, default=0, help="override the workload's batch")
    ap.add_argument("--iters", type=int, default=3)
    ap.add_argument("--kv-dtype", choices=["same", "e4m3"], default="same",
                    help="the cache in the query's dtype, or E4M3 (FP8; prefill: query and caches)")
    ap.add_argument("--contiguous", action="store_true",
                    help="prefill: the same keys as contiguous (non-paged) K/V, no block table")
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    from . import build
    build.build()

    if a.op in ("append_scaled", "decode_scaled", "decode_window", "prefill_window"):
        run = long_session_op(a, dev)
    elif a.op in ("append_rotary", "decode_shared", "merge_states"):
        run = prefix_op(a, dev)
    elif a.op == "prefill":
        e4 = a.kv_dtype == "e4m3"  # E4M3 query and caches, unit device scales
        kw = dict(q_dtype=wl.E4M3, kv_dtype=wl.E4M3) if e4 else {}
        c = wl.ragged_prefill(d_qk=a.d_qk, device=dev, **kw)
        B = c.seq_lens_q.shape[0]
        nbytes = (pk.paged_prefill_fp8_workspace_size(B, c.num_qo_heads, c.num_kv_heads, c.max_q, c.max_kv,
                                                      c.q.shape[0], c.d_qk, c.d_vo, c.q.dtype, c.pool.k.dtype)
                  if e4 else pk.paged_prefill_workspace_size(B, c.num_qo_heads, c.max_q, c.max_kv))
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        lq, lkv, bt = c.seq_lens_q.to(dev), c.seq_lens_kv.to(dev), c.block_tables.to(dev)
        scales = dict(q_scale=torch.ones(1, device=dev), k_scale=torch.ones(1, device=dev),
                      v_scale=torch.ones(1, device=dev)) if e4 else {}

        if a.contiguous:  # each request's keys gathered into [rows, Hkv, d] tensors
            ks, vs = zip(*(wl.read_tokens(c.pool, c.pt, b) for b in range(B)))
            kc, vc = torch.cat(ks).contiguous(), torch.cat(vs).contiguous()

            def run():
                pk.paged_prefill(c.q, kc, vc, c.scale, ws, c.max_q, c.max_kv, lq, lkv, None, causal=True,
                                 **scales)
        else:
            def run():
                pk.paged_prefill(c.q, c.pool.k, c.pool.v, c.scale, ws, c.max_q, c.max_kv, lq, lkv,
                                 bt, causal=True, kv_layout="HND", **scales)
    elif a.op in ("decode_llama", "decode_long", "decode_varlen"):
        kvd = dict(kv_dtype=wl.E4M3) if a.kv_dtype == "e4m3" else {}
        if a.op == "decode_varlen":  # (batch: the first requests of the same draws)
            c = wl.long_decode_varlen(device=dev, batch=a.batch or 256, **kvd)
        elif not a.batch:
            c = (wl.llama_decode(device=dev, **kvd) if a.op == "decode_llama"
                 else wl.long_decode(device=dev, **kvd))
        elif a.op == "decode_llama":  # the first `batch` requests of the same length draw
            L = wl.uniform_lengths(wl.generator(0), 64, 512, 8192)[:a.batch]
            c = wl.decode_case(L, 16, 32, 8, 128, wl.HND, wl.BF16, device=dev, bt_width=512, **kvd)
        else:
            L = wl.lognormal_lengths(wl.generator(0), 256, 4096.0, 1.0, 4, 32768)[:a.batch]
            c = wl.decode_case(L, 64, 64, 8, 128, wl.HND, wl.BF16, q_len_per_req=4,
                               window_left=4095, with_sinks=True, device=dev, bt_width=512, **kvd)
        B = len(c.pt.lengths)
        ws = torch.zeros(max(1, pk.paged_decode_workspace_size(
            B, c.q_len_per_req, c.num_qo_heads, c.num_kv_heads, c.head_dim, c.max_seq_len,
            c.pool.page_size, c.window_left)), dtype=torch.uint8, device=dev)
        bt, sl = c.block_tables.to(dev), c.seq_lens.to(dev)
        sinks = None if c.sinks is None else c.sinks.to(dev)
        kv = c.pool.storage[0]

        cum = None if c.cum_seq_lens_q is None else c.cum_seq_lens_q.to(dev)
        vl = {} if cum is None else dict(cum_seq_lens_q=cum, max_q_len=c.q_len_per_req)

        def run():
            pk.paged_decode(c.query, kv, ws, bt, sl, c.max_seq_len, bmm1_scale=c.bmm1_scale,
                            window_left=c.window_left, sinks=sinks, kv_layout=c.pool.layout,
                            q_len_per_req=c.q_len_per_req, **vl)
    else:
        c = wl.append_sweep(a.batch or 4096, seed=1, layout=wl.NHD, device=dev, fill="empty",
                            **(dict(dtype=wl.E4M3) if a.kv_dtype == "e4m3" else {}))
        kvi, kvp, last = (x.to(dev) for x in (c.kv_indices, c.kv_indptr, c.kv_last_page_len))
        seq = pk.paged_seq_lens(kvp, last, 16)
        nnz = c.append_key.shape[0]
        bi, pos = pk.paged_batch_indices_positions(c.append_indptr.to(dev), seq, nnz)
        pool = c.pool.storage[0]

        def run():
            pk.paged_append(c.append_key, c.append_value, bi, pos, pool, kvi, kvp, last,
                            kv_layout="NHD")

    run()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(a.iters):
        run()
    e1.record()
    torch.cuda.synchronize()
    print(json.dumps({"op": a.op, "d_qk": a.d_qk, "batch": a.batch, "iters": a.iters,
                      "ms_per_call": e0.elapsed_time(e1) / max(1, a.iters)}))


if __name__ == "__main__":
    main()
