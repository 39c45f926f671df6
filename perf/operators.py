"""The operators over key/value caches, as they are measured.

Three operators: the E4M3 cache (tokens quantised as they are written, and
read back), cross attention of queries to cached states of another length,
and attention of a batch to one shared prefix and to each element's own keys.

``run`` computes them in plain form (elementary torch operations in 32 bits)
where ``own`` is false, and calls the package's operators where it is true.
``exact`` states them again from their definitions in 64 bits.
"""

import math

import torch

own = False

DEVICE = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # --- the cache --------------------------------------------------------
        # one new token for each of 16 sequences, appended at 16 positions: the write of a decoding step
        {"name": "write one token", "op": "write", "type": "bf16", "batch": 16, "tokens": 1, "kv_heads": 1,
         "dim": 256, "capacity": 1024, "start": True, "ragged": False},
        # the caches of 64 observations (816 tokens: three views and the text, some with fewer), as a prefill leaves them
        {"name": "write prefixes", "op": "write", "type": "bf16", "batch": 64, "tokens": 816, "kv_heads": 8,
         "dim": 128, "capacity": 1024, "start": False, "ragged": True},
        # the same caches read back to be attended to in bf16 (18 layers of an observation and more)
        {"name": "read prefixes", "op": "read", "type": "bf16", "batch": 72, "tokens": 816, "kv_heads": 4,
         "dim": 256, "capacity": 960, "first": 0, "ragged": True},
        # --- cross attention --------------------------------------------------
        # a single query token over one observation's states: the smallest call
        {"name": "cross one token", "op": "cross", "type": "bf16", "cache": "bf16", "batch": 1, "queries": 1,
         "keys": 816, "heads": 8, "kv_heads": 1, "dim": 256, "ragged": False, "masked": False, "lse": False},
        # the suffix (a state and 50 actions) of 16 observations over their states, some views missing
        {"name": "cross suffix", "op": "cross", "type": "bf16", "cache": "bf16", "batch": 16, "queries": 51,
         "keys": 816, "heads": 8, "kv_heads": 1, "dim": 256, "ragged": True, "masked": True, "lse": False},
        # single tokens of 32 sequences over long quantised caches of different lengths
        {"name": "cross decode quantised", "op": "cross", "type": "bf16", "cache": "fp8", "batch": 32, "queries": 1,
         "keys": 16384, "heads": 8, "kv_heads": 2, "dim": 128, "ragged": True, "masked": False, "lse": True},
        # many queries over long states: the largest product
        {"name": "cross long", "op": "cross", "type": "bf16", "cache": "bf16", "batch": 4, "queries": 2050,
         "keys": 4001, "heads": 16, "kv_heads": 4, "dim": 128, "ragged": False, "masked": False, "lse": False},
        # the fp32 expert's heads, an odd number of keys
        {"name": "cross fp32", "op": "cross", "type": "f32", "cache": "f32", "batch": 8, "queries": 51,
         "keys": 561, "heads": 4, "kv_heads": 1, "dim": 64, "ragged": True, "masked": True, "lse": True},
        # --- shared prefix ----------------------------------------------------
        # 64 sequences decode one token each behind one long prefix
        {"name": "shared decode", "op": "shared", "type": "bf16", "cache": "bf16", "batch": 64, "queries": 1,
         "prefix": 8192, "own": 130, "heads": 8, "kv_heads": 1, "dim": 128, "ragged": True, "masked": False,
         "lse": True},
        # 16 candidate chunks of one observation: each suffix sees the prefix and itself
        {"name": "shared suffixes", "op": "shared", "type": "bf16", "cache": "bf16", "batch": 16, "queries": 51,
         "prefix": 816, "own": 51, "heads": 8, "kv_heads": 1, "dim": 256, "ragged": False, "masked": False,
         "lse": False},
        # 8 suffixes over a long quantised prefix with parts masked
        {"name": "shared quantised", "op": "shared", "type": "bf16", "cache": "fp8", "batch": 8, "queries": 50,
         "prefix": 5000, "own": 70, "heads": 8, "kv_heads": 1, "dim": 256, "ragged": True, "masked": True,
         "lse": False},
        # the fp32 expert's verification: three suffixes of nine tokens over 64 tokens
        {"name": "shared fp32", "op": "shared", "type": "f32", "cache": "f32", "batch": 3, "queries": 9,
         "prefix": 64, "own": 9, "heads": 4, "kv_heads": 1, "dim": 64, "ragged": False, "masked": False,
         "lse": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; odd ones as often as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "cross", "cross", "cross", "shared", "shared", "shared"])
        c = {"op": op, "type": "bf16" if rng.random() < 0.75 else "f32"}
        if op in ("write", "read"):
            c.update(batch=_spread(rng, 1, 72), tokens=_spread(rng, 1, 2048), kv_heads=rng.choice([1, 2, 4, 8]),
                     dim=rng.choice([64, 128, 256]))
            if op == "write":
                c.update(start=rng.random() < 0.5, ragged=rng.random() < 0.5)
            else:
                c.update(first=rng.choice([0, rng.randrange(1, 100)]), ragged=rng.random() < 0.5)
            c["capacity"] = c["tokens"] + rng.randrange(100, 400)
        else:
            f32 = c["type"] == "f32"
            kv_heads = rng.choice([1, 1, 2, 4, 8])
            c.update(cache=c["type"] if f32 or rng.random() < 0.6 else "fp8", batch=_spread(rng, 1, 64),
                     queries=1 if rng.random() < 0.3 else _spread(rng, 1, 400 if f32 else 2050), kv_heads=kv_heads,
                     heads=kv_heads * rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 256]))
            if op == "cross":
                c["keys"] = _spread(rng, 1, 16384)
            else:
                c.update(prefix=_spread(rng, 1, 16384), own=_spread(rng, 1, 400))
            c.update(ragged=rng.random() < 0.5, masked=rng.random() < 0.4, lse=rng.random() < 0.4)
        if _cost(c) <= _most(c):
            return c


def _cost(c):
    """(seconds, about) of the plain form: its fp32 products and its passes over the scores or the cache."""
    if c["op"] in ("write", "read"):
        return 2 * c["batch"] * c["tokens"] * c["kv_heads"] * c["dim"]
    keys = c["keys"] if c["op"] == "cross" else c["prefix"] + c["own"]
    return c["batch"] * (c["heads"] * c["queries"] * (4 * c["dim"] + 200) * keys +
                         (40 * c["kv_heads"] * c["dim"] * c.get("keys", c.get("own"))))


def _most(c):
    alike = [x for x in listed() if x["op"] == c["op"] and x["type"] == c["type"]] or \
        [x for x in listed() if x["op"] == c["op"]]
    most = max(_cost(x) for x in alike)
    return 8 * most if c["type"] == "f32" and c["op"] in ("cross", "shared") else most


def work(c):
    """Bytes: each input and output once, of the tokens that count.  Flops: the products with the visible keys."""
    b, d = c["batch"], c["dim"]
    if c["op"] in ("write", "read"):
        rows = 2 * sum(_lens(b, c["tokens"], c["ragged"])) * c["kv_heads"]
        dense = 2 * b * c["tokens"] * c["kv_heads"] * d * BYTES[c["type"]]
        if c["op"] == "write":   # the real tokens in, their codes and scales out
            return {"bytes": rows * (d * BYTES[c["type"]] + d + 4), "flops": 0}
        return {"bytes": rows * (d + 4) + dense, "flops": 0}   # codes and scales in, every row out
    e, ce = BYTES[c["type"]], BYTES[c["cache"]]
    row = d * ce + (4 if c["cache"] == "fp8" else 0)
    io = b * c["queries"] * c["heads"] * (2 * d * e + (4 if c["lse"] else 0))
    if c["op"] == "cross":
        keys = sum(_visible(n, i, c["masked"]) for i, n in enumerate(_lens(b, c["keys"], c["ragged"])))
        return {"bytes": io + 2 * keys * c["kv_heads"] * row, "flops": 4 * keys * c["queries"] * c["heads"] * d}
    pre = _visible(c["prefix"], 0, c["masked"])
    mine = sum(_lens(b, c["own"], c["ragged"]))
    return {"bytes": io + 2 * c["kv_heads"] * (pre * row + mine * d * e),
            "flops": 4 * (pre * b + mine) * c["queries"] * c["heads"] * d}


def _lens(batch, n, ragged):
    """Valid tokens of each element: all of them, or between a half and all."""
    return [n - (((17 * i) % batch) * (n // 2)) // batch if ragged else n for i in range(batch)]


def _hidden(t, b):
    """Masked keys: one view of 256 tokens in four is missing, another one in each element."""
    return (t // 256 + b) % 4 == 3


def _visible(n, b, masked):
    return n if not masked else sum(not _hidden(t, b) for t in range(n))


# ---------------------------------------------------------------------------
# inputs


def prepare(c, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))

    def normal(*shape, dtype):
        return torch.randn(shape, generator=g, device=DEVICE).to(dtype)

    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEVICE)  # noqa: E731
    t = TYPES[c["type"]]
    b, h, d = c["batch"], c["kv_heads"], c["dim"]
    s = {"case": c}
    if c["op"] == "write":
        n, cap = c["tokens"], c["capacity"]
        s["k"], s["v"] = normal(b, n, h, d, dtype=t), normal(b, n, h, d, dtype=t)
        s["start"] = torch.randint(0, cap - n + 1, (b,), generator=g, device=DEVICE, dtype=torch.int32) \
            if c["start"] else None
        s["count"] = ints(_lens(b, n, True)) if c["ragged"] else None
        s["cache"] = _empty(b, h, cap, d)
        return s
    if c["op"] == "read":
        s["cache"] = _filled(normal, b, h, c["capacity"], d)
        s["lens"] = ints([c["first"] + x for x in _lens(b, c["tokens"], True)]) if c["ragged"] else None
        return s
    s["q"] = normal(b, c["queries"], c["heads"], d, dtype=t)
    if c["op"] == "cross":
        n = c["keys"]
        s["lens"] = ints(_lens(b, n, True)) if c["ragged"] else None
        s["mask"] = ~_hidden(torch.arange(n, device=DEVICE)[None, :], torch.arange(b, device=DEVICE)[:, None]) \
            if c["masked"] else None
        s["kv"] = _filled(normal, b, h, n, d) if c["cache"] == "fp8" else \
            (normal(b, n, h, d, dtype=t), normal(b, n, h, d, dtype=t))
        return s
    n = c["prefix"]
    s["mask"] = ~_hidden(torch.arange(n, device=DEVICE), 0) if c["masked"] else None
    s["kv"] = _filled(normal, 1, h, n, d) if c["cache"] == "fp8" else \
        (normal(n, h, d, dtype=t), normal(n, h, d, dtype=t))
    s["own"] = (normal(b, c["own"], h, d, dtype=t), normal(b, c["own"], h, d, dtype=t))
    s["lens"] = ints(_lens(b, c["own"], True)) if c["ragged"] else None
    return s


def _empty(b, h, cap, d):
    """An E4M3 cache: codes of keys and values [b][h][cap][d], a scale for each token and head [b][h][cap]."""
    return {n: torch.zeros((b, h, cap, d), dtype=torch.uint8, device=DEVICE).view(torch.float8_e4m3fn)
            if n in "kv" else torch.zeros((b, h, cap), device=DEVICE) for n in ("k", "v", "ks", "vs")}


def _filled(normal, b, h, cap, d):
    k, ks = _quantise(normal(b, h, cap, d, dtype=torch.bfloat16).float())
    v, vs = _quantise(normal(b, h, cap, d, dtype=torch.bfloat16).float())
    return {"k": k, "v": v, "ks": ks, "vs": vs}


# ---------------------------------------------------------------------------
# one pass


_handle = []


def _ops():
    from flow_matching_action_dm0_b200 import CacheOps
    if not _handle:
        _handle.append(CacheOps(device=0))
    return _handle[0]


def _cache(kv):
    from flow_matching_action_dm0_b200 import QuantizedKV
    return QuantizedKV(kv["k"], kv["v"], kv["ks"], kv["vs"])


def run(s):
    if own:
        return _run_own(s)
    return {"write": _write, "read": _read, "cross": _cross, "shared": _shared}[s["case"]["op"]](s)


def _run_own(s):
    c, ops = s["case"], _ops()
    if c["op"] == "write":
        ops.write(_cache(s["cache"]), s["k"], s["v"], start=s["start"], count=s["count"])
        return s["cache"]
    if c["op"] == "read":
        return ops.read(_cache(s["cache"]), first=c["first"], n=c["tokens"], lens=s["lens"], dtype=c["type"])
    kv = _cache(s["kv"]) if c["cache"] == "fp8" else s["kv"]
    if c["op"] == "cross":
        return ops.cross_attention(s["q"], kv, lens=s["lens"], mask=s["mask"], lse=c["lse"])
    return ops.shared_attention(s["q"], kv, s["own"], prefix_mask=s["mask"], own_lens=s["lens"], lse=c["lse"])


def _quantise(x):
    """E4M3 codes of the rows x [..., d] and their scales: the least power of two (not under 2^-126) that
    brings the row's largest magnitude to 448 or less."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, -126, torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126))
    scale = ((e + 127) << 23).view(torch.float32)   # 2^e, exactly
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _write(s):
    cache, b, n = s["cache"], s["k"].shape[0], s["k"].shape[1]
    t = torch.arange(n, device=DEVICE)[None, :].expand(b, n)
    if s["count"] is not None:   # tokens behind the last real one repeat it, at its place
        t = torch.minimum(t, s["count"].long()[:, None] - 1)
    at = t if s["start"] is None else t + s["start"].long()[:, None]
    for x, codes, scales in ((s["k"], cache["k"], cache["ks"]), (s["v"], cache["v"], cache["vs"])):
        h, d = x.shape[2], x.shape[3]
        c, f = _quantise(x.float())
        if s["count"] is not None:
            c = c.view(torch.uint8).gather(1, t[:, :, None, None].expand(b, n, h, d))
            f = f.gather(1, t[:, :, None].expand(b, n, h))
        codes.view(torch.uint8).scatter_(2, at[:, None, :, None].expand(b, h, n, d),
                                         c.view(torch.uint8).transpose(1, 2))
        scales.scatter_(2, at[:, None, :].expand(b, h, n), f.transpose(1, 2))
    return cache


def _values(kv, n=None, first=0):
    n = kv["k"].shape[2] if n is None else n
    part = slice(first, first + n)
    return (kv["k"][:, :, part].float() * kv["ks"][:, :, part, None],
            kv["v"][:, :, part].float() * kv["vs"][:, :, part, None])


def _read(s):
    c = s["case"]
    k, v = _values(s["cache"], c["tokens"], c["first"])
    if s["lens"] is not None:
        at = torch.arange(c["first"], c["first"] + c["tokens"], device=DEVICE)
        real = (at[None, :] < s["lens"][:, None])[:, None, :, None]
        k, v = torch.where(real, k, 0.0), torch.where(real, v, 0.0)
    t = TYPES[c["type"]]
    return k.permute(0, 2, 1, 3).to(t).contiguous(), v.permute(0, 2, 1, 3).to(t).contiguous()


def _scores(q, k, visible):
    """Scaled scores [b][kv head][query, head of the group][key] of q [b][t][heads][d] with k [b or 1][kv head][n][d]."""
    b, t, h, d = q.shape
    hk = k.shape[1]
    rows = q.float().reshape(b, t, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, t * (h // hk), d)
    x = torch.matmul(rows, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    return x if visible is None else torch.where(visible[:, None, None, :], x, -math.inf)


def _finish(top, total, weighted, q, lse):
    """The output [b][t][heads][d] in q's type from each row's maximum, sum and weighted values; empty rows give 0."""
    b, t, h, d = q.shape
    hk = weighted.shape[1]

    def rows(x):
        return x.reshape(b, hk, t, h // hk, -1).permute(0, 2, 1, 3, 4).reshape(b, t, h, -1)

    out = rows(weighted / torch.where(total == 0, 1.0, total)).to(q.dtype)
    if not lse:
        return out
    return out, rows(torch.where(total == 0, -math.inf, top + total.log()))[..., 0]


def _cross(s):
    c = s["case"]
    k, v = _values(s["kv"]) if c["cache"] == "fp8" else (x.float().transpose(1, 2) for x in s["kv"])
    x = _scores(s["q"], k, _seen(s["lens"], s["mask"], k.shape[2]))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    return _finish(top, p.sum(-1, keepdim=True), torch.matmul(p, v), s["q"], c["lse"])


def _seen(lens, mask, n):
    seen = None if lens is None else torch.arange(n, device=DEVICE)[None, :] < lens[:, None]
    if mask is None:
        return seen
    return mask if seen is None else mask & seen


def _shared(s):
    c = s["case"]
    pk, pv = _values(s["kv"]) if c["cache"] == "fp8" else (x.float().transpose(0, 1)[None] for x in s["kv"])
    ok, ov = (x.float().transpose(1, 2) for x in s["own"])
    x = _scores(s["q"], pk, None if s["mask"] is None else s["mask"][None])
    y = _scores(s["q"], ok, _seen(s["lens"], None, ok.shape[2]))
    top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, 0.0, top)
    p, r = torch.exp(x - top), torch.exp(y - top)
    total = p.sum(-1, keepdim=True) + r.sum(-1, keepdim=True)
    return _finish(top, total, torch.matmul(p, pv) + torch.matmul(r, ov), s["q"], c["lse"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "write":
        return _exact_write(s)
    if c["op"] == "read":
        out = []
        for codes, scales in (("k", "ks"), ("v", "vs")):
            x = _decode(s["cache"][codes]) * s["cache"][scales].double()[..., None]
            x = x[:, :, c["first"]:c["first"] + c["tokens"]]
            for i, n in enumerate(s["lens"].tolist() if s["lens"] is not None else []):
                x[i, :, max(0, n - c["first"]):] = 0
            out.append(x.transpose(1, 2).contiguous())
        return tuple(out)
    return _exact_attention(s)


def _decode(codes):
    """The values of E4M3 codes from the format: a sign, four exponent bits of bias 7, three mantissa bits."""
    x = codes.contiguous().view(torch.uint8).long()
    e, m = (x >> 3) & 15, (x & 7).double()
    size = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _two(e - 10))
    return torch.where(x >= 128, -size, size)


def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_write(s):
    c, out = s["case"], {}
    starts = s["start"].tolist() if s["start"] is not None else [0] * c["batch"]
    counts = s["count"].tolist() if s["count"] is not None else [c["tokens"]] * c["batch"]
    for name, scales in (("k", "ks"), ("v", "vs")):
        x = s[name].double().transpose(1, 2)
        big = x.abs().amax(-1)
        f = _two(torch.ceil(torch.log2(big / 448)).clamp(min=-126))
        f = torch.where(big > 448 * f, 2 * f, torch.where(big <= 224 * f, f / 2, f)).clamp(min=2.0 ** -126)
        y = x / f[..., None]
        step = _two(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
        codes = torch.zeros(s["cache"][name].shape, dtype=torch.float64, device=DEVICE)
        size = torch.zeros(s["cache"][scales].shape, dtype=torch.float64, device=DEVICE)
        y = torch.round(y / step) * step
        for i, (at, n) in enumerate(zip(starts, counts)):
            codes[i, :, at:at + n] = y[i, :, :n]
            size[i, :, at:at + n] = f[i, :, :n]
        out[name], out[scales] = codes, size
    return {n: out[n] for n in ("k", "v", "ks", "vs")}


def _exact_attention(s):
    c, q = s["case"], s["q"]
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEVICE)
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEVICE)

    def of_head(kv, i, h):
        """Keys and values [n][d] of element i and head h."""
        if isinstance(kv, dict):
            return tuple(_decode(kv[n][i, h]) * kv[f][i, h].double()[:, None] for n, f in (("k", "ks"), ("v", "vs")))
        return tuple(x[i, :, h].double() if x.dim() == 4 else x[:, h].double() for x in kv)

    lens = s["lens"].tolist() if s["lens"] is not None else None
    for h in range(c["kv_heads"]):
        for i in range(c["batch"]):
            if c["op"] == "cross":
                k, v = of_head(s["kv"], i, h)
                keep = torch.arange(k.shape[0], device=DEVICE) < (lens[i] if lens else k.shape[0])
                keep = keep & s["mask"][i] if s["mask"] is not None else keep
                k, v = k[keep], v[keep]
            else:
                if i == 0:
                    pk, pv = of_head(s["kv"], 0, h)
                    if s["mask"] is not None:
                        pk, pv = pk[s["mask"]], pv[s["mask"]]
                ok, ov = of_head(s["own"], i, h)
                n = lens[i] if lens else ok.shape[0]
                k, v = torch.cat([pk, ok[:n]]), torch.cat([pv, ov[:n]])
            if k.shape[0] == 0:
                continue
            for j in range(h * group, (h + 1) * group):
                x = q[i, :, j].double() @ k.T / math.sqrt(c["dim"])
                total = torch.logsumexp(x, 1)
                out[i, :, j] = torch.exp(x - total[:, None]) @ v
                lse[i, :, j] = total
    return (out, lse) if c["lse"] else out
