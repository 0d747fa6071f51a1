"""Prefill over E4M3 caches with block scales whose products leave a 16-bit
type's range: fp16 values at the end of theirs, scales far from one and
different from head to head, and scales that are no powers of two."""
from __future__ import annotations

import pytest
import torch

import _plain
import paged_kv_cache_316_gb300 as pk
from paged_kv_cache_316_gb300 import workloads as wl
from test_gpu_prefill_window import DEV, U, call, make

pytestmark = pytest.mark.gpu


def values(c, b, L):
    return [_plain.tokens(pool.double(), c["pt"].pages[b], L, c["S"], c["layout"], c["used"][b]) *
            _plain.token_scales(c["scales"][:, z], c["pt"].pages[b], L, c["S"], c["used"][b])
            for z, pool in enumerate((c["k"], c["v"]))]


def compare(c, out, lse, scale, u_kv=0.0):
    """As in test_gpu_prefill_window, with two terms more.  u_kv: a key or
    value off by u_kv of itself shifts a logit by dz = u_kv scale sum |q||k|,
    a weight by 2 dz of itself, and the output by (2 dz + u_kv) sum w |v|.
    And an output below fp16's normal numbers is off by half a step, 2^-25."""
    row = 0
    for b, (n, L) in enumerate(zip(c["ql"], c["kvl"])):
        if n:
            u = U[c["dtype"]]
            q = c["q"][row:row + n].double()
            k, v = values(c, b, L)
            a = (L, scale, c["window"], c["first"])
            kw = dict(causal=c["causal"], u_p=u, u_out=u)
            ro, rl, bo, bl = _plain.attention(q, k, v, *a, **kw)
            A = _plain.attention(q, k, v.abs(), *a, **kw)[0]
            g = c["Hq"] // c["H"]
            dz = u_kv * abs(scale) * torch.einsum("nhd,lhd->nhl", q.abs(), k.abs().repeat_interleave(g, 1)).amax(-1)
            half = 2.0 ** -25 if c["dtype"] == torch.float16 else 0.0
            _plain.check(out[row:row + n], ro, bo + (2 * dz[..., None] + u_kv) * A * 1.01 + half, f"out of request {b}")
            _plain.check(lse[row:row + n], rl, bl + dz, f"lse of request {b}")
        row += n


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("window, first", [(-1, 0), (40, 3)])
def test_fp16_tokens_at_the_end_of_the_range(layout, window, first):
    """Tokens of 63488 to 65504 (and an infinity) take the scale 2^8 and the
    code 256: 65536, beyond fp16.  Appended, attended over as a prompt, then
    by one more token."""
    lay = wl.HND if layout == "HND" else wl.NHD
    S, H, Hq, lens = 16, 2, 4, [150, 61]
    g = wl.generator(5)
    pt = wl.reserve_pages([n + 1 for n in lens], S, g)
    one = (S, H, 128) if lay == wl.NHD else (H, S, 128)
    cache = torch.zeros((pt.num_pages, 2) + one, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.ones(pt.num_pages, 2, H, 1, device=DEV)
    rows = sum(lens)
    key, value = (torch.randn(rows, H, 128, generator=g).half() for _ in range(2))
    big = torch.tensor([63488.0, -64504.0, 65504.0, -65504.0, float("inf")]).half()
    for i in range(5):  # (behind enough other tokens that no output leaves fp16's range)
        key[30 + 7 * i, 0, 11 * i] = big[i]
        key[170 + 5 * i, 1, 3 + 20 * i] = big[4 - i]
        value[30 + 7 * i, 1, 11 * i] = big[i]
        value[170 + 5 * i, 0, 3 + 20 * i] = big[4 - i]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pages = [torch.tensor(p, dtype=torch.int32) for p in pt.pages]

    def append(k, v, new, total):
        used = [-(-n // S) for n in total]
        ptr = torch.tensor([0, used[0], sum(used)], dtype=torch.int32, device=DEV)
        idx = torch.cat([p[:n] for p, n in zip(pages, used)]).to(DEV)
        last = torch.tensor([n - (u - 1) * S for n, u in zip(total, used)], dtype=torch.int32, device=DEV)
        seq = pk.paged_seq_lens(ptr, last, S)
        bi, pos = pk.paged_batch_indices_positions(torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device=DEV), seq,
                                                   sum(new))
        pk.paged_append_scaled(k.to(DEV), v.to(DEV), bi, pos, cache, scales, idx, ptr, last, kv_layout=layout, err_word=err)
        return seq

    scale = 2.0 ** -20
    table = pt.block_tables().to(DEV)
    seq = append(key, value, lens, lens)
    q = (torch.randn(rows, Hq, 128, generator=g) * 8).half()
    ws = torch.empty(pk.paged_prefill_scaled_workspace_size(2, Hq, H, 150, 150, 128, 128), dtype=torch.uint8, device=DEV)
    out, lse = pk.paged_prefill(q.to(DEV), cache[:, 0], cache[:, 1], scale, ws, 150, 150, seq, seq, table, kv_layout=layout,
                                kv_scales=scales, err_word=err, window_left=window, first_tokens=first)
    torch.cuda.synchronize()
    c = dict(pt=pt, k=cache[:, 0].cpu(), v=cache[:, 1].cpu(), scales=scales.cpu(), q=q, ql=lens, kvl=lens, S=S, H=H, Hq=Hq,
             layout=lay, dtype=torch.float16, window=window, first=first, causal=True, used=[None, None])
    assert c["scales"].max() == 256 and max(values(c, 0, 150)[0].abs().max(), values(c, 1, 61)[1].abs().max()) >= 65536
    compare(c, out, lse, scale)
    # one more token each
    now = [n + 1 for n in lens]
    seq = append(key[:2], value[:2], [1, 1], now)
    n = pk.paged_decode_workspace_size(2, 1, Hq, H, 128, 151, S, window, first_tokens=first)
    q, dlse = q[:2], torch.empty(2, Hq, device=DEV)
    out = pk.paged_decode(q.to(DEV), cache, torch.empty(max(1, n), dtype=torch.uint8, device=DEV), table, seq, 151,
                          bmm1_scale=scale, kv_layout=layout, lse=dlse, err_word=err, window_left=window,
                          first_tokens=first, kv_scales=scales)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    c.update(k=cache[:, 0].cpu(), v=cache[:, 1].cpu(), scales=scales.cpu(), q=q, ql=[1, 1], kvl=now)
    compare(c, out, dlse, scale)


RANGE = [
    # q lens, kv lens, page, block, Hq, H, d, layout, dtype, window, first
    ([130, 7], [400, 90], 16, 16, 4, 4, 128, wl.HND, torch.float16, -1, 0),
    ([200, 129], [900, 129], 32, 8, 8, 4, 192, wl.NHD, torch.float16, 150, 20),
    ([100, 50, 0, 3], [800, 50, 40, 3], 64, 32, 6, 2, 128, wl.NHD, torch.bfloat16, -1, 0),
    ([33], [500], 256, 128, 3, 1, 192, wl.HND, torch.bfloat16, 60, 9),
]
IDS = [f"r{i}" for i in range(len(RANGE))]


@pytest.mark.parametrize("case", RANGE, ids=IDS)
@pytest.mark.parametrize("k_exp, scale", [(-40, 2.0 ** 30), (24, 2.0 ** -34)])
def test_scales_far_from_one(case, k_exp, scale):
    """K products below fp16's smallest number and beyond its largest; V
    scales 2^16 apart; each head of each request in a range of its own."""
    ql, kvl, S, G, Hq, H, d, layout, dtype, window, first = case
    c = make(ql, kvl, S, Hq, H, d, layout, dtype, sum(ql) + G, window, first, G=G)
    g = wl.generator(S)
    shape = c["scales"][:, 0].shape
    head = torch.arange(H)[None, :, None] * 3.0
    c["scales"][:, 0] = torch.exp2(torch.randint(-2, 1, shape, generator=g) + head + k_exp)
    c["scales"][:, 1] = torch.exp2(torch.randint(-16, 1, shape, generator=g) - head)
    for b, pages in enumerate(c["pt"].pages):  # (the logits of every request and head of one size)
        c["scales"][pages, 0] *= 2.0 ** (-2 * b)
        at = sum(ql[:b])
        c["q"][at:at + ql[b]] *= 2.0 ** (2 * b)
        for i, page in enumerate(pages):  # blocks that no query sees: any scale
            for n in range(S // G):
                seen = c["used"][b][i * S + n * G:i * S + (n + 1) * G]
                if ql[b] and not seen.any():
                    c["scales"][page, :, :, n] = 2.0 ** 48
    for h in range(H):
        c["q"][:, h * (Hq // H):(h + 1) * (Hq // H)] *= 2.0 ** (-3 * h)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, scale, err)
    assert int(err.item()) == 0
    compare(c, out, lse, scale)


@pytest.mark.parametrize("case", RANGE, ids=IDS)
def test_scales_that_are_no_powers_of_two(case):
    """The dequantised keys and values are rounded once to 16 bits."""
    ql, kvl, S, G, Hq, H, d, layout, dtype, window, first = case
    c = make(ql, kvl, S, Hq, H, d, layout, dtype, sum(ql) + G, window, first, G=G)
    c["scales"] *= 1 + torch.rand(c["scales"].shape, generator=wl.generator(9))
    out, lse = call(c, 0.05)
    compare(c, out, lse, 0.05, u_kv=U[dtype])


def test_scale_out_of_range_is_flagged_and_clamped():
    c = make([20, 30], [100, 90], 16, 4, 2, 128, wl.HND, torch.float16, 6, G=16)
    pages = c["pt"].pages
    bad = {(pages[0][0], 0, 0): (0.0, 2.0 ** -48), (pages[0][2], 0, 1): (float("nan"), 2.0 ** -48),
           (pages[1][1], 1, 0): (-1.0, 2.0 ** -48)}
    for at, (was, _) in bad.items():
        c["scales"][at] = was
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = call(c, 0.05, err)
    assert int(err.item()) == 128
    for at, (_, now) in bad.items():
        c["scales"][at] = now
    compare(c, out, lse, 0.05)
