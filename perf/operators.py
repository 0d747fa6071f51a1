"""Cases, plain forms and exact values of the operators that serve long sessions from a compact paged cache:

- appending 16-bit keys and values to a cache held in E4M3 with one power-of-two scale for each block of tokens and head;
- attention of the newest tokens (decode) and of whole prompts (prefill) over that cache;
- attention with a sliding window and a few first tokens that stay visible, for decode and for prompts.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) unless `own` is true; then it
calls the library.  `exact` is the definition in 64 bits, request by request.
"""
import math

import torch

own = False

POISON = 0x7FFFFFFF  # block-table entries past a request's pages: never read
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -40, 40  # exponents of the scales that an append writes


def _case(name, op, **kw):
    base = dict(
        name=name, op=op, batch=1, lo=1, hi=1, q_lo=1, q_hi=1, heads=32, kv_heads=8, d=128, page=16, block=16,
        layout="HND", dtype="bf16", window=-1, first=0, sinks=False)
    base.update(kw)
    return base


def listed():
    return [
        # one new token for each of 64 running requests: what every decode step of a server appends (latency counts)
        _case("append step 64", "append", batch=64, lo=16, hi=4096, q_lo=1, q_hi=1),
        # a few prompts of mixed lengths, token-major pages and fp16, blocks smaller than a page
        _case("append prompts 16", "append", batch=16, lo=0, hi=0, q_lo=1, q_hi=2048, page=32, block=8, layout="NHD", dtype="fp16"),
        # the append sweep's shape: 1024 requests with a cached prefix append up to 128 tokens, 32 kv heads
        _case("append sweep 1024", "append", batch=1024, lo=0, hi=256, q_lo=1, q_hi=128, kv_heads=32, layout="NHD"),
        # four short requests: the smallest decode step (latency counts)
        _case("decode8 short 4", "decode8", batch=4, lo=8, hi=45),
        # 64 requests with contexts up to 8192, four query heads to a kv head, one token each
        _case("decode8 64x8k", "decode8", batch=64, lo=512, hi=8192),
        # long sessions checked four tokens at a time (speculative decoding) under a window with first tokens and sinks
        _case("decode8 stream q4", "decode8", batch=96, lo=3, hi=16384, q_lo=4, q_hi=4, heads=64, page=64, block=64, layout="NHD", dtype="fp16", window=4095, first=64, sinks=True),
        # one chunk of a long prompt over what is cached already
        _case("prefill8 chunk", "prefill8", batch=2, lo=3000, hi=6000, q_lo=512, q_hi=512, page=16),
        # ragged prompts behind cached prefixes
        _case("prefill8 ragged 8", "prefill8", batch=8, lo=0, hi=2048, q_lo=128, q_hi=2048, page=32, block=32, layout="NHD", dtype="fp16"),
        # a few streaming chats: a short window and four first tokens (latency counts)
        _case("window decode 8", "window", batch=8, lo=5, hi=12000, window=1023, first=4),
        # a full batch of long streaming sessions, one token each
        _case("window decode 128", "window", batch=128, lo=700, hi=24000, heads=64, page=64, window=4095, first=128, layout="NHD"),
        # the last chunk of a long document under a window
        _case("window prefill 32k", "window_prefill", batch=1, lo=30700, hi=30700, q_lo=2048, q_hi=2048, page=32, window=4095, first=4),
        # ragged prompts, 192-wide keys, fp16, odd window and first tokens
        _case("window prefill ragged 8", "window_prefill", batch=8, lo=0, hi=2048, q_lo=100, q_hi=2048, page=64, d=192, window=777, first=33, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode8", "prefill8", "window", "window_prefill"))
    page = rng.choice((8, 16, 32, 64, 128))
    kv = rng.choice((1, 2, 4, 8))
    c = dict(_case("", op, page=page, kv_heads=kv, block=rng.choice([b for b in (8, 16, 32, 64, 128) if b <= page]),
                   layout=rng.choice(("HND", "NHD")), dtype=rng.choice(("bf16", "fp16"))))
    del c["name"]
    c["heads"] = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    window, first = _log(rng, 1, 4096), rng.choice((0, 1, 4, 17, 64, 100))
    if op == "append":
        c["batch"], c["lo"] = _log(rng, 1, 256), rng.randrange(0, 40)
        c["hi"], c["q_hi"] = c["lo"] + _log(rng, 1, 500), _log(rng, 1, 300)
        c["q_lo"] = rng.randrange(1, c["q_hi"] + 1)
        return c
    if op in ("decode8", "window"):
        c["q_lo"] = c["q_hi"] = rng.choice((1, 1, 1, 2, 3, 4))
        c["batch"], c["lo"] = _log(rng, 1, 64), rng.randrange(4, 100)
        c["hi"] = c["lo"] + _log(rng, 1, 8000)
        c["sinks"] = rng.random() < 0.3
        if op == "window" or rng.random() < 0.4:
            c["window"], c["first"] = window, first
        return c
    c["batch"], c["lo"] = rng.randrange(1, 7), rng.randrange(0, 50)
    c["hi"], c["q_hi"] = c["lo"] + _log(rng, 1, 2500), _log(rng, 1, 1500)
    c["q_lo"] = rng.randrange(1, c["q_hi"] + 1)
    if op == "window_prefill":
        c["d"] = rng.choice((128, 128, 192))
    if op == "window_prefill" or rng.random() < 0.4:
        c["window"], c["first"] = window, first
    return c


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _spread(n, lo, hi, ratio):
    """n whole numbers over [lo, hi], the same for a case whatever the seed (work() depends on them)."""
    return [lo + int((hi - lo + 1) * (((i + 0.5) * ratio) % 1.0)) for i in range(n)]


def _lengths(c):
    """(tokens already cached or seen, new tokens) of each request, in an order that prepare() permutes."""
    new = _spread(c["batch"], c["q_lo"], c["q_hi"], 0.7548776662466927)
    old = _spread(c["batch"], c["lo"], c["hi"], 0.6180339887498949)
    if c["op"] in ("decode8", "window"):  # lo..hi counts the new tokens too
        old = [max(0, x - n) for x, n in zip(old, new)]
    return old, new


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    old, new = _lengths(c)
    order = torch.randperm(c["batch"], generator=g, device=dev).tolist()
    old, new = [old[i] for i in order], [new[i] for i in order]
    total = [a + b for a, b in zip(old, new)]
    S, H, G = c["page"], c["kv_heads"], c["block"]
    need = [-(-n // S) for n in total]
    pages = sum(need) + sum(need) // 16 + 1
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    start = [0]
    for n in need:
        start.append(start[-1] + n)
    width = max(need)
    kv_indptr = torch.tensor(start, dtype=torch.int32, device=dev)
    col = torch.arange(width, device=dev)
    count = (kv_indptr[1:] - kv_indptr[:-1]).long()
    tables = torch.where(col < count[:, None], ids[(kv_indptr[:-1, None] + col).long().clamp(max=pages - 1)], POISON).to(torch.int32)
    s = dict(case=c, tables=tables, max_len=max(total), max_new=max(new), pages=pages,
             lens=torch.tensor(total, dtype=torch.int32, device=dev), new=torch.tensor(new, dtype=torch.int32, device=dev))

    def rand(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    one = (lambda d: (S, H, d)) if c["layout"] == "NHD" else (lambda d: (H, S, d))
    eight = c["op"] in ("append", "decode8", "prefill8")
    rows = sum(new)
    if eight:  # E4M3 values filled as a block's largest one nearly fills their range, and scales about 2^-7
        cache = torch.empty((pages, 2) + one(c["d"]), dtype=torch.float8_e4m3fn, device=dev)
        step = max(1, (1 << 28) // cache[0].numel())
        for at in range(0, pages, step):
            n = min(step, pages - at)
            cache[at:at + n] = rand(n, *cache.shape[1:]).mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        e = torch.randint(-8, -5, (pages, 2, H, S // G), generator=g, device=dev)
        s["cache"], s["scales"] = cache, torch.exp2(e.float())
    else:
        s["k"] = rand(pages, *one(c["d"]), dtype=_dtype(c))
        s["v"] = rand(pages, *one(128), dtype=_dtype(c))
    if c["op"] == "append":
        # keys and values of a few different magnitudes: some blocks outgrow the scale they have
        mag = torch.exp2(torch.randint(-2, 3, (rows, H, 1), generator=g, device=dev).float())
        s["key"] = (rand(rows, H, c["d"]) * mag).to(_dtype(c))
        s["value"] = (rand(rows, H, c["d"]) * mag).to(_dtype(c))
        s["kv_indptr"], s["kv_indices"] = kv_indptr, ids[:start[-1]].contiguous()
        s["last"] = torch.tensor([n - (p - 1) * S if p else 0 for n, p in zip(total, need)], dtype=torch.int32, device=dev)
        b = torch.repeat_interleave(torch.arange(c["batch"], device=dev), s["new"].long())
        first = torch.cumsum(s["new"].long(), 0) - s["new"].long()
        s["batch_indices"] = b.to(torch.int32)
        s["positions"] = (torch.arange(rows, device=dev) - first[b] + (s["lens"] - s["new"]).long()[b]).to(torch.int32)
        return s
    s["query"] = rand(rows, c["heads"], c["d"]).to(_dtype(c))
    s["scale"] = 1.0 / math.sqrt(c["d"])
    s["sinks"] = rand(c["heads"]) if c["sinks"] else None
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] in ("decode8", "window"):
        return _plain_decode(s)
    return _plain_prefill(s)


def _own(s):
    import paged_kv_cache_316_gb300 as pk

    c = s["case"]
    if c["op"] == "append":
        pk.paged_append_scaled(s["key"], s["value"], s["batch_indices"], s["positions"], s["cache"], s["scales"],
                               s["kv_indices"], s["kv_indptr"], s["last"], kv_layout=c["layout"])
        return s["cache"], s["scales"]
    eight = c["op"] in ("decode8", "prefill8")
    scales = s["scales"] if eight else None
    if c["op"] in ("decode8", "window"):
        if "workspace" not in s:  # kept between calls, as a serving loop does
            n = pk.paged_decode_workspace_size(c["batch"], c["q_hi"], c["heads"], c["kv_heads"], c["d"], s["max_len"],
                                               c["page"], c["window"], first_tokens=c["first"])
            s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        lse = torch.empty(s["query"].shape[:2], dtype=torch.float32, device="cuda")
        out = pk.paged_decode(s["query"], s["cache"] if eight else (s["k"], s["v"]), s["workspace"], s["tables"],
                              s["lens"], s["max_len"], bmm1_scale=s["scale"], window_left=c["window"], sinks=s["sinks"],
                              kv_layout=c["layout"], q_len_per_req=c["q_hi"], lse=lse, first_tokens=c["first"],
                              kv_scales=scales)
        return out, lse
    if "workspace" not in s:
        n = (pk.paged_prefill_scaled_workspace_size(c["batch"], c["heads"], c["kv_heads"], s["max_new"], s["max_len"],
                                                    c["d"], 128) if eight else
             pk.paged_prefill_workspace_size(c["batch"], c["heads"], s["max_new"], s["max_len"]))
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    k, v = (s["cache"][:, 0], s["cache"][:, 1]) if eight else (s["k"], s["v"])
    return pk.paged_prefill(s["query"], k, v, s["scale"], s["workspace"], s["max_new"], s["max_len"], s["new"],
                            s["lens"], s["tables"], causal=True, kv_layout=c["layout"], window_left=c["window"],
                            first_tokens=c["first"], kv_scales=scales)


def _plain_append(s):
    """Every block that gets new tokens takes the larger of its scale (where it holds earlier tokens) and the smallest
    power of two under which its new finite values reach at most 448; earlier values are rounded again where it grew."""
    c, cache, scales = s["case"], s["cache"], s["scales"]
    S, H, G, d = c["page"], c["kv_heads"], c["block"], c["d"]
    P, nb = s["pages"], S // G
    pos = s["positions"].long()
    page = s["kv_indices"][s["kv_indptr"][s["batch_indices"].long()].long() + pos // S].long()
    slot = pos % S
    block = page * nb + slot // G
    x = torch.stack((s["key"], s["value"]), 1).float()  # [rows, 2, H, d]
    size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)  # [rows, 2, H]
    most = torch.zeros(P * nb, 2, H, device=x.device).index_reduce_(0, block, size, "amax")
    low = torch.full((P * nb,), S, dtype=torch.long, device=x.device).index_reduce_(0, block, slot, "amin")
    m, e = torch.frexp(most)  # most = m 2^e with m in [1/2, 1); 448 = 7/8 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(MIN_EXP, MAX_EXP)
    wanted = torch.exp2(torch.where(most > 0, e, torch.full_like(e, MIN_EXP)).float())
    was = scales.permute(0, 3, 1, 2).reshape(P * nb, 2, H)  # a copy
    kept = (low % G != 0) & (low < S)  # blocks with earlier tokens
    now = torch.where((low < S)[:, None, None], torch.where(kept[:, None, None], torch.maximum(was, wanted), wanted), was)
    # earlier values, on the blocks whose scale grew
    at = torch.nonzero(kept & (now > was).flatten(1).any(1)).squeeze(1)
    view = cache.view(P, 2, nb, G, H, d).permute(0, 2, 1, 4, 3, 5) if c["layout"] == "NHD" else \
        cache.view(P, 2, H, nb, G, d).permute(0, 3, 1, 2, 4, 5)  # [P, nb, 2, H, G, d]
    held = view[at // nb, at % nb].float()
    again = (held * (was[at] / now[at])[..., None, None]).to(torch.float8_e4m3fn)
    early = torch.arange(G, device=x.device) < (low[at] % G)[:, None]
    grew = (now[at] > was[at])[..., None, None] & early[:, None, None, :, None]
    view[at // nb, at % nb] = torch.where(grew, again.float(), held).to(torch.float8_e4m3fn)
    # the new values
    q = (x / now[block][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    view[page, slot // G, :, :, slot % G] = q
    scales.copy_(now.view(P, nb, 2, H).permute(0, 2, 3, 1))
    return cache, scales


def _rows(s, which, tables, keys, ok):
    """Keys or values [B, N, H, d] of token indices keys [B, N] in 32 bits; zeros where not ok."""
    c = s["case"]
    S = c["page"]
    page = torch.where(ok, tables.gather(1, (keys // S).clamp(0, tables.shape[1] - 1)), 0).long()
    slot = torch.where(ok, keys % S, 0)
    if "cache" in s:
        pool, scale = s["cache"][:, which], s["scales"][:, which]
    else:
        pool, scale = s["kv"[which]], None
    x = (pool[page, slot] if c["layout"] == "NHD" else pool.transpose(1, 2)[page, slot]).float()
    if scale is not None:
        x = x * scale.transpose(1, 2)[page, slot // c["block"]][..., None]
    return torch.where(ok[..., None, None], x, 0.0)


def _visible(c, keys, at):
    """Which keys a query at position `at` sees."""
    seen = keys <= at
    if c["window"] >= 0:
        seen = seen & ((keys >= at - c["window"]) | (keys < c["first"]))
    return seen


def _attend(score, seen, v, sinks):
    """softmax and its product with v; score, seen [B, H, g, Q, N], v [B, N, H, d] -> [B, Q, H g, d], lse [B, Q, H g]."""
    B, H, g, Q, N = score.shape
    score = score.masked_fill_(~seen, -math.inf)
    m = score.amax(-1)
    if sinks is not None:
        m = torch.maximum(m, sinks.view(1, H, g, 1))
    base = torch.where(torch.isinf(m), 0.0, m)
    p = score.sub_(base[..., None]).exp_()
    total = p.sum(-1)
    if sinks is not None:
        total = total + torch.exp(sinks.view(1, H, g, 1) - base)
    out = torch.matmul(p.reshape(B, H, g * Q, N), v.transpose(1, 2)).view(B, H, g, Q, -1)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = base + torch.log(total)
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)


def _score(s, q, k):
    """scale <q, k>: q [B, Q, heads, d], k [B, N, H, d] -> [B, H, g, Q, N]."""
    B, Q, heads, d = q.shape
    H = k.shape[2]
    q = q.float().view(B, Q, H, heads // H, d).permute(0, 2, 3, 1, 4)
    return torch.matmul(q.reshape(B, H, -1, d), k.permute(0, 2, 3, 1)).view(B, H, heads // H, Q, -1).mul_(s["scale"])


def _plain_decode(s):
    c, dev = s["case"], s["query"].device
    B, Q, W, F = c["batch"], c["q_hi"], c["window"], c["first"]
    L = s["lens"].long()[:, None]
    if W >= 0:  # the first tokens before the window, then the window of all the request's queries
        lo = (L - Q - W).clamp(min=0)
        first = torch.arange(F, device=dev).expand(B, F)
        near = lo + torch.arange(min(W + Q, s["max_len"]), device=dev)
        keys, ok = torch.cat((first, near), 1), torch.cat(((first < lo) & (first < L), near < L), 1)
    else:
        keys = torch.arange(s["max_len"], device=dev).expand(B, -1)
        ok = keys < L
    tables = s["tables"]
    k = _rows(s, 0, tables, keys, ok)
    score = _score(s, s["query"].view(B, Q, c["heads"], -1), k)
    del k
    at = L - Q + torch.arange(Q, device=dev)  # [B, Q]
    seen = _visible(c, keys[:, None, :], at[..., None]) & ok[:, None, :]
    out, lse = _attend(score, seen[:, None, None], _rows(s, 1, tables, keys, ok), s["sinks"])
    return out.flatten(0, 1).to(_dtype(c)), lse.flatten(0, 1)


def _plain_prefill(s):
    c, dev = s["case"], s["query"].device
    new, L = s["new"].long(), s["lens"].long()
    row = torch.arange(s["max_new"], device=dev)
    real = row < new[:, None]  # [B, Q]
    place = (torch.cumsum(new, 0) - new)[:, None] + row
    q = s["query"][torch.where(real, place, 0)]
    keys = torch.arange(s["max_len"], device=dev).expand(c["batch"], -1)
    ok = keys < L[:, None]
    k = _rows(s, 0, s["tables"], keys, ok)
    score = _score(s, q, k)
    del k
    at = (L - new)[:, None] + row
    seen = _visible(c, keys[:, None, :], at[..., None]) & ok[:, None, :]
    out, lse = _attend(score, seen[:, None, None], _rows(s, 1, s["tables"], keys, ok), None)
    return out[real].to(_dtype(c)), lse[real]


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(c):
    old, new = _lengths(c)
    H, d, S, G, W, F = c["kv_heads"], c["d"], c["page"], c["block"], c["window"], c["first"]
    rows = sum(new)
    if c["op"] == "append":  # keys and values read in 16 bits and written in 8, touched scales written
        blocks = sum((a + n - 1) // G - a // G + 1 for a, n in zip(old, new))
        return {"bytes": rows * H * d * 2 * 3 + 8 * rows + blocks * H * 2 * 4, "flops": rows * H * d * 2 * 2}
    read, pairs, blocks, pages = 0, 0, 0, 0
    for a, n in zip(old, new):
        L = a + n
        lo = max(0, a - W) if W >= 0 else 0
        span = L - lo + min(F, lo)  # keys that some query of the request sees
        read += span
        blocks += -(-span // G)
        pages += -(-span // S)
        for t in range(n):
            pairs += a + t + 1 if W < 0 else _seen_by(a + t, W, F)
    eight = c["op"] in ("decode8", "prefill8")
    size = 1 if eight else 2
    dv = 128
    moved = read * H * (d + dv) * size + (blocks * H * 8 if eight else 0) + 4 * pages
    return {"bytes": moved + rows * c["heads"] * ((d + dv) * 2 + 4), "flops": 2.0 * pairs * c["heads"] * (d + dv)}


def _seen_by(p, W, F):
    lo = max(0, p - W)
    return p + 1 - lo + min(F, lo)


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return _exact_append(s) if c["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    c = s["case"]
    S, H, G = c["page"], c["kv_heads"], c["block"]
    nhd = c["layout"] == "NHD"
    cache, scales = s["cache"], s["scales"]
    grid = torch.tensor([x for x in _e4m3_grid()], dtype=torch.float64, device=cache.device)
    ptr, ids, pos_all = s["kv_indptr"].tolist(), s["kv_indices"].tolist(), s["positions"].tolist()
    runs, i, who = [], 0, s["batch_indices"].tolist()
    while i < len(who):  # new tokens that share a block
        j = i + 1
        while j < len(who) and who[j] == who[i] and pos_all[j] // G == pos_all[i] // G:
            j += 1
        runs.append((i, j - i, ids[ptr[who[i]] + pos_all[i] // S], pos_all[i] % S))
        i = j
    if len(runs) > 40000:
        return None
    lut = {}
    for r in runs:
        lut.setdefault(r[1], []).append(r)
    for n, some in lut.items():  # runs of one length at a time
        for at in range(0, len(some), 2048):
            part = some[at:at + 2048]
            row, page, slot = (torch.tensor([r[k] for r in part], device=cache.device) for k in (0, 2, 3))
            span = torch.arange(n, device=cache.device)
            x = torch.stack([t[row[:, None] + span].double() for t in (s["key"], s["value"])], 1)  # [r, 2, n, H, d]
            size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax((2, 4))  # [r, 2, H]
            e = torch.ceil(torch.log2(torch.clamp(size, min=2.0 ** -200) / E4M3_MAX) - 1e-12).clamp(MIN_EXP, MAX_EXP)
            e = torch.where(size > E4M3_MAX * torch.exp2(e), e + 1, e).clamp(MIN_EXP, MAX_EXP)
            want = torch.exp2(e)
            was = scales[page, :, :, slot // G].double()
            held = (slot % G > 0)[:, None, None]
            now = torch.where(held, torch.maximum(was, want), want)
            scales[page, :, :, slot // G] = now.float()
            for t in range(G):  # earlier tokens of the block
                on = slot % G > t
                here = torch.where(on, slot // G * G + t, 0)
                old = (cache[page, :, here] if nhd else cache[page, :, :, here]).double()  # [r, 2, H, d]
                redo = _nearest(old * (was / now)[..., None], grid)
                redo = torch.where((now > was)[..., None], redo, old).to(torch.float8_e4m3fn)
                if nhd:
                    cache[page[on], :, here[on]] = redo[on]
                else:
                    cache[page[on], :, :, here[on]] = redo[on]
            for t in range(n):
                put = _nearest(x[:, :, t] / now[..., None], grid).to(torch.float8_e4m3fn)
                if nhd:
                    cache[page, :, slot + t] = put
                else:
                    cache[page, :, :, slot + t] = put
    return cache.to(torch.float64), scales.double()


def _e4m3_grid():
    """The finite non-negative values of an 8-bit float with 4 exponent bits (bias 7) and 3 mantissa bits."""
    return sorted([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])


def _nearest(x, grid):
    """The grid value nearest to each |x| with x's sign; ties to the even mantissa; the largest value beyond the range."""
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    take = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take, grid[hi], grid[lo]).copysign(x)


def _exact_attention(s):
    c = s["case"]
    S, H, heads, W, F = c["page"], c["kv_heads"], c["heads"], c["window"], c["first"]
    outs, lses, row = [], [], 0
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        lo = max(0, L - n - W) if W >= 0 else 0
        j = torch.arange(L, device=s["query"].device)
        j = j[(j >= lo) | (j < F)] if W >= 0 else j
        page, slot = s["tables"][b, (j // S)].long(), j % S
        kv = []
        for which in (0, 1):
            pool = s["cache"][:, which] if "cache" in s else s["kv"[which]]
            x = (pool[page, slot] if c["layout"] == "NHD" else pool[page, :, slot]).double()
            if "cache" in s:
                x = x * s["scales"][page, which, :, slot // c["block"]].double()[..., None]
            kv.append(x)
        p = torch.arange(L - n, L, device=j.device)
        hidden = j[None, :] > p[:, None]
        if W >= 0:
            hidden |= (j[None, :] < p[:, None] - W) & (j[None, :] >= F)
        q = s["query"][row:row + n].double()
        out = torch.empty(n, heads, kv[1].shape[-1], dtype=torch.float64, device=j.device)
        lse = torch.empty(n, heads, dtype=torch.float64, device=j.device)
        for h in range(heads):
            z = (q[:, h] @ kv[0][:, h // (heads // H)].T) * s["scale"]
            z[hidden] = -math.inf
            if s["sinks"] is not None:
                z = torch.cat((z, s["sinks"][h].double().expand(n, 1)), 1)
            lse[:, h] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[:, h, None])[:, :j.numel()]
            out[:, h] = torch.nan_to_num(w) @ kv[1][:, h // (heads // H)]
        outs.append(out)
        lses.append(lse)
        row += n
    return torch.cat(outs), torch.cat(lses)
