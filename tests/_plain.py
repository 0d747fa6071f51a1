"""Plain 64-bit implementations, on the CPU, of the append to an E4M3 cache
with block scales and of attention under a window with first tokens, and the
bounds that the kernels' roundings allow.  Written from the definitions in
include/pagedkv.h; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

NHD, HND = 0, 1

# the finite non-negative E4M3 values in the order of their codes 0x00 .. 0x7e
GRID = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def to_codes(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 codes of float64 values: ties to the even code, beyond
    448 the largest code, NaN 0x7f."""
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), GRID[-1])
    hi = np.clip(np.searchsorted(GRID, a), 0, GRID.size - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def from_codes(c: np.ndarray) -> np.ndarray:
    mag = np.append(GRID, np.nan)[c & 0x7F]
    return np.where(c & 0x80, -mag, mag)


def slot_view(cache: np.ndarray, page: int, which: int, head: int, slot: int, layout: int):
    """The row of one token and head in a [P, 2, ..] array of codes."""
    return cache[page, which, slot, head] if layout == NHD else cache[page, which, head, slot]


def append_scaled(key, value, batch_indices, positions, cache, scales, kv_indices, kv_indptr, lens, page_size,
                  layout, drop=()):
    """In place on numpy arrays: cache uint8 [P, 2, ..], scales float32
    [P, 2, H, nb].  `drop`: entries that the call has to skip."""
    H = key.shape[1]
    G = page_size // scales.shape[3]
    src = [key.double().numpy(), value.double().numpy()]
    i = 0
    n_all = len(batch_indices)
    while i < n_all:
        b, pos = int(batch_indices[i]), int(positions[i])
        if i in drop:
            i += 1
            continue
        j = i + 1
        while j < n_all and j not in drop and batch_indices[j] == b and positions[j] == pos + j - i \
                and (pos + j - i) // G == pos // G:
            j += 1
        page, slot = int(kv_indices[kv_indptr[b] + pos // page_size]), pos % page_size
        for z in range(2):
            for h in range(H):
                x = src[z][i:j, h]
                fin = np.abs(x[np.isfinite(x)])
                a = float(fin.max()) if fin.size else 0.0
                e = -40
                while e < 40 and a > 448.0 * 2.0 ** e:
                    e += 1
                s = np.float32(2.0 ** e)
                was = s
                if slot % G:
                    was = scales[page, z, h, slot // G]
                    was = np.float32(min(max(was, 2.0 ** -48), 2.0 ** 48)) if was == was else np.float32(2.0 ** -48)
                    s = max(s, was)
                scales[page, z, h, slot // G] = s
                if s > was:
                    r = np.float32(was / s)
                    for t in range(slot // G * G, slot):
                        row = slot_view(cache, page, z, h, t, layout)
                        row[:] = to_codes((from_codes(row).astype(np.float32) * r).astype(np.float64))
                for t in range(j - i):
                    with np.errstate(over="ignore"):
                        q = (x[t].astype(np.float32) / s).astype(np.float64)
                    slot_view(cache, page, z, h, slot + t, layout)[:] = to_codes(q)
        i = j


def visible(j, p, window, first):
    """[len(p), len(j)]: which keys j each query position p sees."""
    seen = j[None, :] <= p[:, None]
    if window >= 0:
        seen &= (j[None, :] >= p[:, None] - window) | (j[None, :] < first)
    return seen


def attention(q, k, v, L, scale, window=-1, first=0, sinks=None, causal=True, u_p=2.0 ** -8, u_out=2.0 ** -8,
              bmm2=1.0):
    """One request: q [n, Hq, d], k [L, H, d], v [L, H, dv] (float64, CPU; rows
    that no query sees may hold anything), queries at the last n of L
    positions.  Returns (out, lse, out bound, lse bound).

    Bounds, for weights w_j = e^z_j / total and A = sum w_j |v_j|: a logit is
    off by at most dz = (d 2^-22) scale sum |q||k| (fp32 products accumulated
    in any order, each step off by at most 2^-22 of the running sum of
    magnitudes) + 2^-20 (1 + |z|) (scaling, the exponent's fp32 argument, the
    2^x and log2 approximations); the weights in the product with V are
    rounded (u_p), the denominator is summed from unrounded ones; the output
    is rounded once (u_out).  So |err| <= u_out |o| + (u_p + 2 dz) A (1 + small),
    and the log-sum-exp is off by at most dz."""
    n, Hq, d = q.shape
    g = Hq // k.shape[1]
    p = torch.arange(L - n, L)
    j = torch.arange(L)
    seen = visible(j, p, window, first) if causal else \
        (torch.ones(n, L, dtype=torch.bool) if window < 0 else
         ((j[None, :] >= p[:, None] - window) | (j[None, :] < first)))
    used = seen.any(0)
    k = torch.where(used[:, None, None], k, torch.zeros((), dtype=torch.float64))
    v = torch.where(used[:, None, None], v, torch.zeros((), dtype=torch.float64))
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    z = torch.einsum("nhd,lhd->hnl", q, k) * scale
    mag = torch.einsum("nhd,lhd->hnl", q.abs(), k.abs()) * abs(scale)
    dz = torch.where(seen, d * 2.0 ** -22 * mag + 2.0 ** -20 * (1 + z.abs()), torch.zeros((), dtype=torch.float64))
    dz = dz.amax(-1) if L else torch.zeros(Hq, n, dtype=torch.float64)
    z = z.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, -1) if L else torch.full((Hq, n), -math.inf, dtype=torch.float64)
    if sinks is not None:
        lse = torch.logaddexp(lse, sinks.double()[:, None].expand_as(lse))
    w = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("hnl,lhd->nhd", w, v) * bmm2
    A = torch.einsum("hnl,lhd->nhd", w, v.abs()) * abs(bmm2)
    dz_t = dz.T
    bound = u_out * out.abs() + (u_p + 2 * dz_t[..., None] + 2.0 ** -20) * A * 1.01 + 2.0 ** -24 * 6e-2
    return out, lse.T, bound, dz_t + 2.0 ** -20 * (1 + torch.where(torch.isinf(lse.T), torch.zeros_like(lse.T), lse.T).abs())


def tokens(pool, table, L, page_size, layout, used=None):
    """Rows [L, H, d] of one request out of a [P, ..] CPU tensor; rows that
    `used` leaves out are zeros and their pages are not looked up."""
    H = pool.shape[2] if layout == NHD else pool.shape[1]
    out = torch.zeros(L, H, pool.shape[3], dtype=pool.dtype)
    for j in range(L):
        if used is None or used[j]:
            pg, s = int(table[j // page_size]), j % page_size
            out[j] = pool[pg, s] if layout == NHD else pool[pg, :, s]
    return out


def token_scales(scales, table, L, page_size, used=None):
    """Scales [L, H, 1] (float64) of one request out of [P, H, nb]."""
    G = page_size // scales.shape[2]
    out = torch.ones(L, scales.shape[1], 1, dtype=torch.float64)
    for j in range(L):
        if used is None or used[j]:
            out[j, :, 0] = scales[int(table[j // page_size]), :, j % page_size // G].double()
    return out


def check(got, ref, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (g.shape, ref.shape)
    ninf = torch.isneginf(ref)
    assert torch.equal(torch.isneginf(g), ninf), f"{what}: -inf pattern differs"
    assert torch.isfinite(g[~ninf]).all(), f"{what}: non-finite values"
    err = torch.where(ninf, torch.zeros_like(ref), (g - torch.where(ninf, g, ref)).abs())
    bad = err > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; worst {err.max():.3e} where "
                           f"{bound.flatten()[err.argmax()]:.3e} is allowed")
