"""Cases, plain forms and exact values of the operators around attention over prefixes that requests share:

- normalising the heads of queries and keys, rotating them by their positions and appending keys and values to the
  pages, in one pass (and the same onto rows, for what follows without a 16-bit paged cache);
- decode of a batch whose requests share long prefixes (system prompts, documents, examples), each prefix read once for
  all of its requests;
- merging attention over separate parts of the keys by their log-sum-exp.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64) unless `own` is
true; then it calls the library.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

POISON = 0x7FFFFFFF  # block-table entries past a request's pages: never read


def _rope(name, op, **kw):
    """One rotation case.  lo..hi tokens are cached already, q_lo..q_hi are new; the dimensions start .. start + part of
    every head are rotated; norm: RMS norm of each head of queries and keys first."""
    base = dict(name=name, op=op, batch=1, lo=0, hi=0, q_lo=1, q_hi=1, heads=32, kv_heads=8, d=128, part=128, start=0,
                page=16, layout="NHD", dtype="bf16", norm=True, interleaved=False, base=10000.0, stretch=1.0,
                magnitude=1.0, fused=False)
    base.update(kw)
    return base


def _shared(name, **kw):
    """One decode over shared prefixes: `groups` prefixes of p_lo..p_hi tokens, the requests divided among them unevenly,
    lo..hi tokens of each request's own (the q newest among them)."""
    base = dict(name=name, op="shared", batch=4, groups=1, p_lo=512, p_hi=512, lo=1, hi=64, q=1, heads=32, kv_heads=8,
                page=16, layout="HND", dtype="bf16", sinks=False)
    base.update(kw)
    return base


def _merge(name, **kw):
    base = dict(name=name, op="merge", states=2, rows=1, heads=32, d=128, dtype="bf16", empty=0.0)
    base.update(kw)
    return base


def listed():
    return [
        # one new token for each of 64 running requests: what every decode step does before attention (latency counts)
        _rope("append rotary step 64", "append_rotary", batch=64, lo=16, hi=4096, layout="HND"),
        # a chunk of a long document whose positions are stretched over the trained length, rows of one fused projection
        _rope("append rotary chunk 120k", "append_rotary", lo=120000, hi=120000, q_lo=4096, q_hi=4096, page=32,
              base=500000.0, stretch=8.0, magnitude=1.2079441541679836, fused=True),
        # ragged prompts in fp16, half of each head rotated, neighbouring elements paired, no norms
        _rope("append rotary prompts 16", "append_rotary", batch=16, q_lo=1, q_hi=2048, page=64, layout="HND",
              dtype="fp16", norm=False, interleaved=True, part=64),
        # the append sweep's shape: 1024 requests with a cached prefix append up to 128 tokens
        _rope("append rotary sweep 1024", "append_rotary", batch=1024, lo=0, hi=256, q_lo=1, q_hi=128),
        # seven tokens of small heads onto rows (latency counts)
        _rope("rotary rows 7", "rotary", q_lo=7, q_hi=7, heads=14, kv_heads=2, d=64, part=64, dtype="fp16",
              interleaved=True),
        # prompts with 192-wide queries and keys, of which the last 64 dimensions hold positions, onto rows
        _rope("rotary rows 8k d192", "rotary", batch=4, q_lo=1500, q_hi=2500, heads=32, kv_heads=32, d=192, part=64,
              start=128, norm=False),
        # four requests behind a short system prompt: the smallest decode step (latency counts)
        _shared("shared decode 4"),
        # 64 requests with the context of a long document in common and up to 1024 tokens of their own
        _shared("shared decode 64x8k", batch=64, p_lo=8192, p_hi=8192, lo=64, hi=1024),
        # three prompts of odd lengths, four tokens checked at a time (speculative decoding), sinks
        _shared("shared decode groups q4", batch=45, groups=3, p_lo=1001, p_hi=16001, lo=4, hi=333, q=4, heads=28,
                kv_heads=4, page=64, layout="NHD", dtype="fp16", sinks=True),
        # many samples over one long context: as much arithmetic as a prefill
        _shared("shared decode 256x32k", batch=256, p_lo=32768, p_hi=32768, lo=16, hi=512, heads=64),
        # one step's rows from two parts of the context (latency counts)
        _merge("merge 2x64", rows=64),
        # prompts attended in four parts of the context, some rows with nothing visible in a part, fp16
        _merge("merge 4x8k", states=4, rows=8192, dtype="fp16", empty=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append_rotary", "append_rotary", "rotary", "shared", "shared", "shared", "merge"))
    dtype = rng.choice(("bf16", "fp16"))
    kv = rng.choice((1, 2, 4, 8))
    if op == "merge":
        c = _merge("", states=rng.randrange(2, 9), rows=_log(rng, 1, 3000), heads=rng.randrange(1, 41),
                   d=rng.choice((64, 128, 192, 256)), dtype=dtype, empty=rng.choice((0.0, 0.1, 0.5)))
    elif op == "shared":
        c = _shared("", batch=_log(rng, 1, 128), kv_heads=kv, q=rng.choice((1, 1, 1, 2, 3, 4)), dtype=dtype,
                    page=rng.choice((8, 16, 32, 64, 128)), layout=rng.choice(("HND", "NHD")), sinks=rng.random() < 0.3)
        c["heads"] = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
        c["groups"] = rng.randrange(1, min(c["batch"], 6) + 1)
        c["p_lo"] = rng.randrange(1, 300)
        c["p_hi"] = c["p_lo"] + _log(rng, 1, 14000)
        c["lo"] = rng.randrange(4, 40)
        c["hi"] = c["lo"] + _log(rng, 1, 1500)
    else:
        d = rng.choice((64, 80, 96, 128, 128, 128, 192, 256))
        part = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= d])
        c = _rope("", op, kv_heads=kv, d=d, part=part, start=rng.choice((0, 0, (d - part) // 8 * 8)), dtype=dtype,
                  page=rng.choice((8, 16, 32, 64, 128)), layout=rng.choice(("HND", "NHD")), norm=rng.random() < 0.6,
                  interleaved=rng.random() < 0.5, base=rng.choice((10000.0, 500000.0, 1000000.0)),
                  stretch=rng.choice((1.0, 1.0, 4.0)), magnitude=rng.choice((1.0, 1.0, 1.1386294361119891)),
                  fused=rng.random() < 0.3)
        c["heads"] = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
        c["batch"], c["lo"] = _log(rng, 1, 100), rng.randrange(0, 40)
        c["hi"], c["q_hi"] = c["lo"] + _log(rng, 1, 3000), _log(rng, 1, 300)
        c["q_lo"] = rng.randrange(1, c["q_hi"] + 1)
    del c["name"]
    return c


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _spread(n, lo, hi, ratio):
    """n whole numbers over [lo, hi], the same for a case whatever the seed (work() depends on them)."""
    return [lo + int((hi - lo + 1) * (((i + 0.5) * ratio) % 1.0)) for i in range(n)]


def _lengths(c):
    """(tokens already cached, new tokens) of each request of a rotation case."""
    return (_spread(c["batch"], c["lo"], c["hi"], 0.6180339887498949),
            _spread(c["batch"], c["q_lo"], c["q_hi"], 0.7548776662466927))


def _parts(c):
    """(requests, prefix length) of each group, and each request's own length, of a shared decode."""
    weight = _spread(c["groups"], 1, 9, 0.6180339887498949)
    left, sizes = c["batch"] - c["groups"], []
    for i, w in enumerate(weight):
        n = left if i == c["groups"] - 1 else min(left, left * w // sum(weight[i:]))
        sizes.append(1 + n)
        left -= n
    prefix = _spread(c["groups"], c["p_lo"], c["p_hi"], 0.7548776662466927)
    return sizes, prefix, [max(n, c["q"]) for n in _spread(c["batch"], c["lo"], c["hi"], 0.5698402909980532)]


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def _frequencies(c):
    """Angle of a step of one position, for each rotated pair: base^(-2 i / part), the slower ones (fewer than 4 turns
    over 8192 positions, ramping from 32 turns) divided by `stretch`."""
    n = c["part"] // 2
    f = c["base"] ** (-torch.arange(n, dtype=torch.float64) / n)
    if c["stretch"] != 1.0:
        keep = ((8192 * f / (2 * math.pi) - 4) / 28).clamp(0, 1)
        f = f * (keep + (1 - keep) / c["stretch"])
    return f


def _table(ids, count):
    """Rows of page ids, `count` pages each taken from `ids` in turn, padded with POISON."""
    out = torch.full((len(count), max(max(count), 1)), POISON, dtype=torch.int32, device=ids.device)
    at = 0
    for i, n in enumerate(count):
        out[i, :n] = ids[at:at + n]
        at += n
    return out


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rand(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    t = _dtype(c)
    s = dict(case=c)
    if c["op"] == "merge":
        shape = (c["rows"], c["heads"])
        s["states"] = []
        for _ in range(c["states"]):
            lse = rand(*shape) * 2 + 6
            if c["empty"]:
                gone = torch.rand(shape, generator=g, device=dev) < c["empty"]
                lse = torch.where(gone, -math.inf, lse)
            s["states"].append((rand(*shape, c["d"], dtype=t), lse))
        return s
    H, d, S = c["kv_heads"], c.get("d", 128), c["page"]
    one = (S, H, d) if c["layout"] == "NHD" else (H, S, d)
    if c["op"] == "shared":
        sizes, prefix, lens = _parts(c)
        order = torch.randperm(c["batch"], generator=g, device=dev).tolist()
        lens = [lens[i] for i in order]
        first = [-(-n // S) for n in prefix]
        rest = [-(-n // S) for n in lens]
        pages = sum(first) + sum(rest)
        pages += pages // 16 + 1
        ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["prefix_tables"], s["tables"] = _table(ids, first), _table(ids[sum(first):], rest)
        s["sizes"], s["prefix"], s["own_lens"] = sizes, prefix, lens
        indptr = [0]
        for n in sizes:
            indptr.append(indptr[-1] + n)
        s["group_indptr"] = torch.tensor(indptr, dtype=torch.int32, device=dev)
        s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["max_prefix"], s["max_len"] = max(prefix), max(lens)
        s["cache"] = rand(pages, 2, *one, dtype=t)
        s["query"] = rand(c["batch"] * c["q"], c["heads"], d).to(t)
        s["scale"] = 1.0 / math.sqrt(d)
        s["sinks"] = rand(c["heads"]) if c["sinks"] else None
        return s
    old, new = _lengths(c)
    order = torch.randperm(c["batch"], generator=g, device=dev).tolist()
    old, new = [old[i] for i in order], [new[i] for i in order]
    rows = sum(new)
    batch_indices = torch.repeat_interleave(torch.arange(c["batch"], device=dev), torch.tensor(new, device=dev))
    before = torch.tensor(new, device=dev).cumsum(0) - torch.tensor(new, device=dev)
    at = torch.arange(rows, device=dev) - before[batch_indices] + torch.tensor(old, device=dev)[batch_indices]
    s["positions"] = at.to(torch.int32)
    # what a projection gives: heads of different sizes
    size = torch.exp2(torch.randint(-2, 3, (c["heads"] + 2 * H, 1), generator=g, device=dev).float())
    rows_of = (rand(rows, c["heads"] + 2 * H, d) * size).to(t)
    parts = rows_of.split((c["heads"], H, H), dim=1)
    s["query"], s["key"], s["value"] = parts if c["fused"] else (x.contiguous() for x in parts)
    s["query_weight"], s["key_weight"] = ((1 + 0.2 * rand(d)).to(t) if c["norm"] else None for _ in range(2))
    s["frequencies"] = _frequencies(c).to(dev)
    if c["op"] == "append_rotary":
        need = [-(-(a + n) // S) for a, n in zip(old, new)]
        pages = sum(need) + sum(need) // 16 + 1
        start = [0]
        for n in need:
            start.append(start[-1] + n)
        s["batch_indices"] = batch_indices.to(torch.int32)
        s["kv_indptr"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["kv_indices"] = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[:start[-1]].contiguous()
        s["last"] = torch.tensor([a + n - (p - 1) * S for a, n, p in zip(old, new, need)], dtype=torch.int32, device=dev)
        s["cache"] = rand(pages, 2, *one, dtype=t)
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "merge":
        return _plain_merge(s)
    if c["op"] == "shared":
        return _plain_shared(s)
    return _plain_rotary(s)


def _own(s):
    import paged_kv_cache_316_gb300 as pk

    c = s["case"]
    if c["op"] == "merge":
        return pk.paged_merge_states(s["states"])
    if c["op"] == "shared":
        if "workspace" not in s:  # kept between calls, as a serving loop does
            n = pk.paged_decode_shared_workspace_size(c["batch"], c["q"], c["heads"], c["kv_heads"], 128, c["groups"],
                                                      s["max_prefix"], s["max_len"], c["page"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        lse = torch.empty(s["query"].shape[:2], dtype=torch.float32, device="cuda")
        out = pk.paged_decode_shared(s["query"], s["cache"], s["workspace"], s["prefix_tables"], s["prefix_lens"],
                                     s["group_indptr"], s["max_prefix"], s["tables"], s["lens"], s["max_len"],
                                     bmm1_scale=s["scale"], sinks=s["sinks"], kv_layout=c["layout"],
                                     q_len_per_req=c["q"], lse=lse)
        return out, lse
    kw = dict(rotary_start=c["start"], interleaved=c["interleaved"], magnitude=c["magnitude"],
              query_weight=s["query_weight"], key_weight=s["key_weight"], eps=1e-6)
    if c["op"] == "rotary":
        return pk.paged_rotary(s["query"], s["key"], s["positions"], s["frequencies"], **kw)
    query = pk.paged_append_rotary(s["query"], s["key"], s["value"], s["batch_indices"], s["positions"], s["cache"],
                                   s["kv_indices"], s["kv_indptr"], s["last"], s["frequencies"],
                                   kv_layout=c["layout"], **kw)
    return query, s["cache"]


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos = (torch.cos(angle) * c["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * c["magnitude"]).float()[:, None]
    out = []
    for x, w in ((s["query"], s["query_weight"]), (s["key"], s["key_weight"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        else:
            x = x.clone()
        part = x[..., c["start"]:c["start"] + c["part"]]
        half = c["part"] // 2
        a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :half], part[..., half:])
        u, v = a * cos - b * sin, b * cos + a * sin
        part.copy_(torch.stack((u, v), -1).flatten(-2) if c["interleaved"] else torch.cat((u, v), -1))
        out.append(x.to(_dtype(c)))
    if c["op"] == "rotary":
        return out[0], out[1]
    S = c["page"]
    at = s["positions"].long()
    page = s["kv_indices"][s["kv_indptr"][s["batch_indices"].long()].long() + at // S].long()
    for which, x in ((0, out[1]), (1, s["value"])):
        pool = s["cache"][:, which]
        if c["layout"] == "NHD":
            pool[page, at % S] = x
        else:
            pool[page, :, at % S] = x
    return out[0], s["cache"]


def _plain_merge(s):
    lse = torch.stack([l for _, l in s["states"]])
    m = lse.amax(0)
    base = torch.where(torch.isinf(m), 0.0, m)
    w = torch.exp(lse - base)
    total = w.sum(0)
    out = torch.zeros_like(s["states"][0][0], dtype=torch.float32)
    for i, (x, _) in enumerate(s["states"]):
        out += torch.where(w[i] > 0, w[i] / torch.where(total > 0, total, 1.0), 0.0)[..., None] * x.float()
    return out.to(_dtype(s["case"])), base + torch.log(total)


def _gather(s, which, tables, n):
    """Keys or values [rows of the table, n, H, d] of the first n tokens in 32 bits; zeros past a row's pages."""
    c = s["case"]
    S = c["page"]
    at = torch.arange(n, device=tables.device)
    page = tables[:, at // S]
    ok = page < s["cache"].shape[0]
    page = torch.where(ok, page, 0).long()
    pool = s["cache"][:, which] if c["layout"] == "NHD" else s["cache"][:, which].transpose(1, 2)
    return torch.where(ok[..., None, None], pool[page, at % S].float(), 0.0)


def _plain_shared(s):
    c, dev = s["case"], s["query"].device
    Q, H, heads = c["q"], c["kv_heads"], c["heads"]
    g = heads // H
    out = torch.empty(s["query"].shape, dtype=_dtype(c), device=dev)
    lse = torch.empty(s["query"].shape[:2], dtype=torch.float32, device=dev)
    row = 0
    for i, (n, P) in enumerate(zip(s["sizes"], s["prefix"])):
        L = s["lens"][row:row + n].long()
        q = s["query"][row * Q:(row + n) * Q].float().view(n, Q, H, g, 128).mul(s["scale"])
        # the prefix: all of the group's rows against one set of keys
        k = _gather(s, 0, s["prefix_tables"][i:i + 1], P)[0]
        z = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(H, n * Q * g, 128), k.permute(1, 2, 0))
        z = z.view(H, n, Q, g, P)
        # each request's own keys, the newest Q of them hidden from the tokens before them
        ko = _gather(s, 0, s["tables"][row:row + n], s["max_len"])
        zo = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(H, n, Q * g, 128), ko.permute(2, 0, 3, 1))
        zo = zo.view(H, n, Q, g, -1)
        at = L[:, None] - Q + torch.arange(Q, device=dev)
        hidden = torch.arange(s["max_len"], device=dev) > at[..., None]  # [n, Q, N]
        zo.masked_fill_(hidden[None, :, :, None], -math.inf)
        m = torch.maximum(z.amax(-1), zo.amax(-1))
        sinks = None if s["sinks"] is None else s["sinks"].view(H, 1, 1, g)
        if sinks is not None:
            m = torch.maximum(m, sinks)
        z.sub_(m[..., None]).exp_()
        zo.sub_(m[..., None]).exp_()
        total = z.sum(-1) + zo.sum(-1)
        if sinks is not None:
            total = total + torch.exp(sinks - m)
        v = _gather(s, 1, s["prefix_tables"][i:i + 1], P)[0]
        o = torch.matmul(z.view(H, n * Q * g, P), v.transpose(0, 1)).view(H, n, Q, g, 128)
        vo = _gather(s, 1, s["tables"][row:row + n], s["max_len"])
        o = o + torch.matmul(zo.view(H, n, Q * g, -1), vo.permute(2, 0, 1, 3)).view(H, n, Q, g, 128)
        o = o / total[..., None]
        out[row * Q:(row + n) * Q] = o.permute(1, 2, 0, 3, 4).reshape(n * Q, heads, 128).to(out.dtype)
        lse[row * Q:(row + n) * Q] = (m + torch.log(total)).permute(1, 2, 0, 3).reshape(n * Q, heads)
        row += n
    return out, lse


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(c):
    if c["op"] == "merge":
        n = c["rows"] * c["heads"]
        return {"bytes": n * (c["states"] + 1) * (2 * c["d"] + 4), "flops": 2.0 * n * c["d"] * c["states"]}
    if c["op"] == "shared":
        sizes, prefix, lens = _parts(c)
        H, Q, S = c["kv_heads"], c["q"], c["page"]
        keys = sum(prefix) + sum(lens)
        tables = sum(-(-n // S) for n in prefix + lens)
        pairs = Q * (sum(n * p for n, p in zip(sizes, prefix)) + sum(lens)) - len(lens) * Q * (Q - 1) // 2
        rows = c["batch"] * Q
        return {"bytes": keys * H * 512 + 4 * tables + rows * c["heads"] * (512 + 4),
                "flops": 2.0 * pairs * c["heads"] * 256}
    _, new = _lengths(c)
    rows, d, H = sum(new), c["d"], c["kv_heads"]
    moved = rows * (c["heads"] + H) * d * 4 + 4 * rows
    if c["op"] == "append_rotary":
        moved += rows * H * d * 4 + 4 * rows
    return {"bytes": moved, "flops": rows * (c["heads"] + H) * (3.0 * c["part"] + (4.0 * d if c["norm"] else 0.0))}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "merge":
        return _exact_merge(s)
    return _exact_shared(s) if c["op"] == "shared" else _exact_rotary(s)


def _exact_rotary(s):
    """Every rotated pair as a complex number times magnitude e^(i angle)."""
    c = s["case"]
    turn = torch.polar(torch.full((len(s["positions"]), c["part"] // 2), c["magnitude"], dtype=torch.float64,
                                  device=s["positions"].device),
                       torch.outer(s["positions"].to(torch.float64), s["frequencies"]))
    pair = torch.arange(c["part"] // 2, device=turn.device)
    re, im = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + c["part"] // 2)
    re, im = re + c["start"], im + c["start"]
    done = []
    for x, w in ((s["query"], s["query_weight"]), (s["key"], s["key_weight"])):
        y = x.to(torch.float64)
        if w is not None:
            y = y / (y.pow(2).sum(-1) / c["d"] + 1e-6).sqrt().unsqueeze(-1) * w.to(torch.float64)
        z = torch.complex(y[:, :, re], y[:, :, im]) * turn.unsqueeze(1)
        y = y.clone()
        y[:, :, re], y[:, :, im] = z.real, z.imag
        done.append(y)
    if c["op"] == "rotary":
        return done[0], done[1]
    cache = s["cache"].to(torch.float64)
    S, N = c["page"], cache.shape[0]
    spot = s["kv_indices"].long()[s["kv_indptr"].long()[s["batch_indices"].long()] + s["positions"].long() // S]
    slot = s["positions"].long() % S
    for which, x in ((0, done[1]), (1, s["value"].to(torch.float64))):
        if c["layout"] == "NHD":
            cache.view(N * 2 * S, c["kv_heads"], c["d"])[(spot * 2 + which) * S + slot] = x
        else:
            for h in range(c["kv_heads"]):
                cache.view(N * 2 * c["kv_heads"] * S, c["d"])[((spot * 2 + which) * c["kv_heads"] + h) * S + slot] = x[:, h]
    return done[0], cache


def _exact_merge(s):
    parts = [(x.double(), l.double()) for x, l in s["states"]]
    lse = torch.logsumexp(torch.stack([l for _, l in parts]), 0)
    out = sum(torch.where(l.isinf(), 0.0, torch.exp(l - lse))[..., None] * x for x, l in parts)
    return torch.where(lse.isinf()[..., None], 0.0, out), lse


def _exact_shared(s):
    c = s["case"]
    S, H, Q, heads = c["page"], c["kv_heads"], c["q"], c["heads"]
    g = heads // H
    out = torch.empty(s["query"].shape, dtype=torch.float64, device=s["query"].device)
    lse = torch.empty(s["query"].shape[:2], dtype=torch.float64, device=out.device)

    def rows_of(table, n, h, which):
        j = torch.arange(n, device=out.device)
        page = table[j // S].long()
        return (s["cache"][page, which, j % S, h] if c["layout"] == "NHD" else s["cache"][page, which, h, j % S]).double()

    r = 0
    for i, (n, P) in enumerate(zip(s["sizes"], s["prefix"])):
        for h in range(H):
            q = s["query"][r * Q:(r + n) * Q, h * g:(h + 1) * g].double()  # [n Q, g, 128]
            kp, vp = (rows_of(s["prefix_tables"][i], P, h, w) for w in (0, 1))
            near = (q.reshape(-1, 128) @ kp.T).view(n, Q, g, P) * s["scale"]
            for b in range(n):
                L = s["own_lens"][r + b]
                ko, vo = (rows_of(s["tables"][r + b], L, h, w) for w in (0, 1))
                z = torch.cat((near[b], torch.einsum("qgd,jd->qgj", q[b * Q:(b + 1) * Q], ko) * s["scale"]), -1)
                for t in range(Q):
                    z[t, :, P + L - Q + t + 1:] = -math.inf
                top = torch.logsumexp(z, -1)
                if s["sinks"] is not None:
                    top = torch.logaddexp(top, s["sinks"][h * g:(h + 1) * g].double())
                p = torch.exp(z - top[..., None])
                at = slice((r + b) * Q, (r + b + 1) * Q)
                out[at, h * g:(h + 1) * g] = p @ torch.cat((vp, vo))
                lse[at, h * g:(h + 1) * g] = top
        r += n
    return out, lse
