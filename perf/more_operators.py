"""The attention-cache operators as they are measured: cases, plain forms, and definitions in 64 bits.

Five operators that belong together in the attention of a decode step whose cache is held in MXFP4
(E2M1 elements, one UE8M0 power-of-two scale per 32 elements of a head):

  table    cosines and sines of every position, plain or scaled for long contexts
  rope     rotary positions applied to part of each head
  write    keys and values -> MXFP4 rows of a paged cache
  read     rows of the cache -> the values they stand for
  attend   attention of query rows over the paged cache: single tokens, drafts and prompts

`run` makes the framework's calls where `own` is true; otherwise it computes the same in elementary
torch operations in 32 bits (64 for the angles of far positions).
"""
import math

import torch

own = False

_HANDLE = []


def _handle():
    """One library handle for the process, as a user's program keeps it."""
    if not _HANDLE:
        import mxfp8_block_scaled_06_gb300 as mx

        _HANDLE.append((mx, mx.mx_create(0)))
    return _HANDLE[0]


# ------------------------------------------------------------------------------------------ cases
def _table(positions, d, scaling, base=10000.0, factor=1.0, original=0):
    return {"op": "table", "positions": positions, "d": d, "scaling": scaling, "base": base, "factor": factor,
            "original": original}


def _rope(t, heads, d, d_rope, interleaved, last, inverse=False, more=0, dtype="bf16"):
    """more: heads behind these in each token's row, as keys and values behind the queries of one projection."""
    return {"op": "rope", "t": t, "heads": heads, "d": d, "d_rope": d_rope, "interleaved": interleaved, "last": last,
            "inverse": inverse, "more": more, "dtype": dtype}


def _write(t, heads, d, shared, page, dtype="bf16"):
    return {"op": "write", "t": t, "heads": heads, "d": d, "shared": shared, "page": page, "dtype": dtype}


def _read(rows, heads, d, shared, page, dtype="bf16"):
    return {"op": "read", "rows": rows, "heads": heads, "d": d, "shared": shared, "page": page, "dtype": dtype}


def _attend(b, new, longest, q_heads, heads, d, shared, page=64, window=0, dtype="bf16"):
    """b sequences of up to `longest` cached tokens; `new`: query tokens of a sequence (0: prompts of ragged
    lengths, a quarter of the longest on average)."""
    return {"op": "attend", "b": b, "new": new, "longest": longest, "q_heads": q_heads, "heads": heads, "d": d,
            "shared": shared, "page": page, "window": window, "dtype": dtype}


def listed():
    return [
        # the table of a short context, made when a model is loaded
        {"name": "table 4096 positions", **_table(4096, 64, "none")},
        # the table of a context stretched by interpolating the slow dimensions only
        {"name": "table 163840 positions, stretched", **_table(163840, 64, "yarn", 10000.0, 40.0, 4096)},
        # the query heads of one decode token, the last 64 of 512 dimensions rotated
        {"name": "rope 1 token", **_rope(1, 16, 512, 64, True, True)},
        # the query heads of a prompt out of a fused projection, whole heads rotated in halves
        {"name": "rope 8191 tokens", **_rope(8191, 32, 128, 128, False, True, more=16)},
        # one decode token's latent, keys and values in one
        {"name": "write 1 token", **_write(1, 1, 512, True, 64)},
        # a prompt's keys and values
        {"name": "write 16381 tokens", **_write(16381, 8, 128, False, 64)},
        # a short prefix's latents, read back
        {"name": "read 37 rows", **_read(37, 1, 512, True, 64)},
        # the keys and values of a long prefix, read back for a copy elsewhere
        {"name": "read 32749 rows", **_read(32749, 8, 128, False, 64)},
        # one decode token over a short context, sixteen heads over one latent
        {"name": "attend 1 sequence", **_attend(1, 1, 777, 16, 1, 512, True)},
        # a decode batch of ragged long contexts, grouped heads
        {"name": "attend 61 sequences", **_attend(61, 1, 16384, 32, 8, 128, False)},
        # a decode batch of ragged long contexts, sixteen heads over one latent
        {"name": "attend 48 sequences, latents", **_attend(48, 1, 32768, 16, 1, 512, True)},
        # prompts behind cached prefixes, grouped heads
        {"name": "attend 3 prompts", **_attend(3, 0, 8192, 32, 8, 128, False)},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "write", "write", "read", "attend", "attend", "attend", "attend"])
    if op == "table":
        d = 2 * _log(rng, 8, 128)
        scaling = rng.choice(["none", "linear", "yarn"])
        factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0])
        return _table(_log(rng, 1, 163840 * 64 // d), d, scaling, rng.choice([10000.0, 500000.0]), factor,
                      rng.choice([2048, 4096, 8192]) if scaling == "yarn" else 0)
    heads, d = rng.choice([(1, 512), (1, 512), (8, 128), (4, 128), (2, 256), (5, 64), (16, 64), (1, 128)])
    shared = heads == 1 and rng.random() < 0.8
    page = rng.choice([16, 32, 48, 64, 64, 128, 256])
    if op == "rope":
        heads = rng.choice([1, 7, 16, 24, 32, 64])
        d = 8 * _log(rng, 4, 64)
        d_rope = d if rng.random() < 0.4 else 16 * rng.randint(1, d // 16)
        return _rope(_log(rng, 1, max(1, 8191 * 32 * 128 // (heads * d))), heads, d, d_rope, rng.random() < 0.5,
                     rng.random() < 0.6, rng.random() < 0.3, rng.choice([0, 0, 2, 16]), rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "write":
        return _write(_log(rng, 1, 16381 * 8 * 128 // (heads * d)), heads, d, shared, page,
                      rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "read":
        return _read(_log(rng, 1, 32749 * 8 * 128 // (heads * d)), heads, d, shared, page,
                     rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    group = rng.choice([1, 2, 4, 5, 8, 16]) if heads > 1 else rng.choice([8, 16, 16, 32])
    new = rng.choice([1, 1, 1, rng.randint(2, 8), 0])
    b = rng.randint(1, 4) if new == 0 else _log(rng, 1, 128)
    # no more cached bytes than the listed decode batches, no more operations than the listed prompts
    most = 48 * 32768 * 512 // (b * heads * d)
    if new == 0:
        most = min(most, int(math.sqrt(3 * 8192**2 * 32 * 128 / (b * heads * group * d))))
    longest = _log(rng, max(1, new), max(8, min(65536, most)))
    return _attend(b, new, longest, heads * group, heads, d, shared, page, rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                   rng.choice(["bf16", "bf16", "fp16"]))


# ----------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (2**63))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(case, seed):
    """Cached tokens (the query tokens among them) and query tokens of each sequence. Prompts are the same ones
    for every seed, in another order: so many tokens make a step."""
    import random

    longest, new, b = case["longest"], case["new"], case["b"]
    rng = random.Random(seed * 7919 + 1 if new else 1)
    lengths = [rng.randint(max(new, 1, longest // 16), longest) for _ in range(b)]
    lengths[rng.randrange(b)] = longest
    counts = [new] * b if new else [max(1, rng.randint(n // 8, n * 3 // 8)) for n in lengths]
    order = random.Random(seed).sample(range(b), b)
    return [lengths[i] for i in order], [counts[i] for i in order]


def _keys(g, rows, heads, d):
    """Key-like rows: some channels are larger than the others in every row."""
    wide = torch.exp(0.5 * _normal(g, heads, d))
    return _normal(g, rows, heads, d) * wide


def _values(g, rows, heads, d):
    """Value-like rows: their size varies from token to token."""
    return _normal(g, rows, heads, d) * torch.exp(0.7 * _normal(g, rows, 1, 1))


def _empty_cache(pages, case):
    """Codes and scales of keys and, unless they are shared, of values: [pages, heads, page, bytes]."""
    heads, page, d = case["heads"], case["page"], case["d"]
    one = lambda n: torch.zeros(pages, heads, page, n, dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = {"k": one(d // 2), "k_scales": one(d // 32)}
    if not case["shared"]:
        cache.update(v=one(d // 2), v_scales=one(d // 32))
    return cache


def _filled(g, case, slots, pages):
    """A cache whose rows `slots` hold keys and values, quantized a part at a time."""
    cache, heads, d = _empty_cache(pages, case), case["heads"], case["d"]
    step = max(1, 2**27 // (heads * d))
    for i in range(0, len(slots), step):
        part = slots[i:i + step]
        for name, make in (("k", _keys), ("v", _values)):
            if name in cache:
                codes, scales = _mx4(make(g, len(part), heads, d).bfloat16().float())
                _store(cache[name], part, codes)
                _store(cache[name + "_scales"], part, scales)
    return cache


def _store(pool, slots, rows):
    """rows [n, heads, bytes] into the slots (page * page size + place) of pool."""
    page = pool.shape[2]
    pool[slots // page, :, slots % page] = rows


def _load(pool, slots):
    page = pool.shape[2]
    return pool[slots // page, :, slots % page]


def _spread(g, rows, page, spare=3):
    """Slots of `rows` tokens, one after another in pages that lie anywhere, and the number of pages."""
    used = (rows + page - 1) // page
    order = torch.randperm(used + spare, generator=g, device="cuda")[:used]
    at = torch.arange(rows, device="cuda")
    return order[at // page] * page + at % page, used + spare


def prepare(case, seed):
    g, s = _generator(seed), dict(case)
    if own:
        s["mx"], s["h"] = _handle()
    op = case["op"]
    if op == "table":
        s["magnitude"] = 1.0 + 0.01 * (seed % 50)  # the factor that a stretched context puts on the logits
    elif op == "rope":
        most = 32768
        s["positions"] = torch.randint(0, most, (case["t"],), generator=g, device="cuda")
        f = 10000.0 ** (-torch.arange(0, case["d_rope"], 2, dtype=torch.float64, device="cuda") / case["d_rope"])
        angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * f
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        wide = _normal(g, case["t"], case["heads"] + case["more"], case["d"]).to(_TYPES[case["dtype"]])
        s["x"] = wide[:, :case["heads"]]
    elif op == "write":
        t = case["t"]
        # the tokens of several requests at once: anywhere in their pages
        slots, pages = _spread(g, t + t // 4 + 1, case["page"])
        s["slots"] = slots[torch.randperm(len(slots), generator=g, device="cuda")[:t]]
        s["slots"][torch.rand(t, generator=g, device="cuda") < 0.01] = -1  # padding tokens
        s["cache"] = _empty_cache(pages, case)
        s["k"] = _keys(g, t, case["heads"], case["d"]).to(_TYPES[case["dtype"]])
        s["v"] = None if case["shared"] else _values(g, t, case["heads"], case["d"]).to(_TYPES[case["dtype"]])
    elif op == "read":
        s["slots"], pages = _spread(g, case["rows"], case["page"])
        s["cache"] = _filled(g, case, s["slots"], pages)
    else:
        lengths, counts = _lengths(case, seed)
        page = case["page"]
        held = [(n + page - 1) // page for n in lengths]
        pages = sum(held) + 3
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.full((case["b"], max(held)), -1, dtype=torch.int32, device="cuda")
        slots, at = [], 0
        for i, n in enumerate(lengths):
            mine = order[at:at + held[i]]
            table[i, :held[i]] = mine
            t = torch.arange(n, device="cuda")
            slots.append(mine.long()[t // page] * page + t % page)
            at += held[i]
        s["cache"] = _filled(g, case, torch.cat(slots), pages)
        s["table"], s["lengths_list"], s["counts"] = table, lengths, counts
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        offsets = [0]
        for n in counts:
            offsets.append(offsets[-1] + n)
        s["offsets_list"] = offsets
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda") if case["new"] == 0 else None
        s["q"] = (1.5 * _normal(g, offsets[-1], case["q_heads"], case["d"])).to(_TYPES[case["dtype"]])
        s["scale"] = 1 / math.sqrt(case["d"])
    if own and "cache" in s:
        c = s["cache"]
        s["own_cache"] = s["mx"].MxCache(c["k"], c["k_scales"], c.get("v"), c.get("v_scales"))
    return s


# ------------------------------------------------------------------------------------- plain forms
def _codes4(a):
    """Magnitude codes 0..7 of a >= 0, to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    return ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5).byte())


def _mx4(x):
    """float32 [.., d] -> (E2M1 codes, two to a byte, the first in the low bits, [.., d / 2]; scale bytes [.., d / 32]):
    the scale's exponent is floor(log2 amax) - 2, at least -127; a block that is not finite has scale byte 255."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    field = (amax.view(torch.int32) >> 23) & 255
    s = torch.where(torch.isfinite(amax), (field - 2).clamp(min=0), 255).to(torch.uint8)
    bad = (s == 255).unsqueeze(-1)
    y = torch.where(bad, 0.0, b) * ((254 - s.int()) << 23).view(torch.float32).unsqueeze(-1)
    c = _codes4(y.abs()) + torch.signbit(y).byte() * 8
    c = torch.where(bad, 0, c).reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), s


def _values4(q, s):
    """float32 values of packed E2M1 codes [.., d / 2] under scale bytes [.., d / 32]."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    two = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)
    v = two[q.int()].reshape(*s.shape, 32)
    bits = torch.where(s == 0, 0x00400000, s.int() << 23)  # 2^(s - 127); 2^-127 is subnormal
    power = torch.where(s == 255, math.nan, bits.int().view(torch.float32))
    return (v * power.unsqueeze(-1)).reshape(*q.shape[:-1], -1)


def _frequencies(s):
    """Radians per position of each pair, in 64 bits."""
    d, i = s["d"], torch.arange(s["d"] // 2, dtype=torch.float64, device="cuda")
    f = s["base"] ** (-2 * i / d)
    if s["scaling"] == "linear":
        f = f / s["factor"]
    elif s["scaling"] == "yarn":
        # dimensions of more than 32 turns in the original context keep their frequency, those of less than
        # one are interpolated, with a ramp between
        at = lambda turns: d * math.log(s["original"] / (2 * math.pi * turns)) / (2 * math.log(s["base"]))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d - 1)
        r = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - r) + f / s["factor"] * r
    return f


def _run_table(s):
    if own:
        return s["mx"].mx_rope_table(s["h"], s["positions"], s["d"], base=s["base"], scaling=s["scaling"],
                                     factor=s["factor"], original=s["original"], magnitude=s["magnitude"])
    angle = torch.arange(s["positions"], dtype=torch.float64, device="cuda")[:, None] * _frequencies(s)
    return (torch.cat([angle.cos(), angle.sin()], 1) * s["magnitude"]).float()


def _rotated(x, cs, s):
    """The rotated copy of x [t, heads, d] by cs [t, d_rope], cosines and then sines."""
    n, first = s["d_rope"], s["d"] - s["d_rope"] if s["last"] else 0
    c, w = cs[:, None, :n // 2], cs[:, None, n // 2:]
    if s["inverse"]:
        w = -w
    out = x.clone()
    part = x[..., first:first + n]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        out[..., first:first + n:2] = a * c - b * w
        out[..., first + 1:first + n:2] = b * c + a * w
    else:
        a, b = part[..., :n // 2], part[..., n // 2:]
        out[..., first:first + n // 2] = a * c - b * w
        out[..., first + n // 2:first + n] = b * c + a * w
    return out


def _run_rope(s):
    if own:
        return s["mx"].mx_rope(s["h"], s["x"], s["positions"], s["cos_sin"], first=s["d"] - s["d_rope"] if s["last"] else 0,
                               interleaved=s["interleaved"], inverse=s["inverse"])
    return _rotated(s["x"].float(), s["cos_sin"][s["positions"]], s).to(s["x"].dtype)


def _run_write(s):
    cache = s["cache"]
    if own:
        k, v = s["mx"].mx_cache_write(s["h"], s["own_cache"], s["slots"], s["k"], s["v"], values=True)
    else:
        out, valid = {}, s["slots"] >= 0
        slots = s["slots"][valid]
        for name in ("k", "v"):
            x = s[name]
            if x is not None:
                codes, scales = _mx4(x.float())
                _store(cache[name], slots, codes[valid])
                _store(cache[name + "_scales"], slots, scales[valid])
                out[name] = _values4(codes, scales).bfloat16()
        k, v = out["k"], out.get("v")
    return {"k_values": k, **({} if v is None else {"v_values": v}), **cache}


def _run_read(s):
    cache, kind = s["cache"], _TYPES[s["dtype"]]
    if own:
        k, v = s["mx"].mx_cache_read(s["h"], s["own_cache"], s["slots"], dtype=kind)
        return {"k": k} if v is None else {"k": k, "v": v}
    return {n: _values4(_load(cache[n], s["slots"]), _load(cache[n + "_scales"], s["slots"])).to(kind)
            for n in ("k", "v") if n in cache}


def _sequence(s, i):
    """Slots of sequence i's cached tokens."""
    t = torch.arange(s["lengths_list"][i], device="cuda")
    return s["table"][i].long()[t // s["page"]] * s["page"] + t % s["page"]


def _run_attend(s):
    if own:
        return s["mx"].mx_attend(s["h"], s["q"], s["own_cache"], s["table"], s["lengths"], q_offsets=s["offsets"],
                                 scale=s["scale"], window=s["window"])
    cache, out = s["cache"], torch.empty_like(s["q"])
    heads, group = s["heads"], s["q_heads"] // s["heads"]
    for i in range(s["b"]):
        slots = _sequence(s, i)
        k = _values4(_load(cache["k"], slots), _load(cache["k_scales"], slots))
        v = k if s["shared"] else _values4(_load(cache["v"], slots), _load(cache["v_scales"], slots))
        n, rows = len(slots), slice(s["offsets_list"][i], s["offsets_list"][i + 1])
        q = s["q"][rows].float()
        seen = torch.arange(n, device="cuda")[None, :]
        at = torch.arange(n - len(q), n, device="cuda")[:, None]  # positions of the query tokens
        hidden = seen > at
        if s["window"]:
            hidden = hidden | (seen <= at - s["window"])
        for h in range(heads):
            mine = q[:, h * group:(h + 1) * group]
            score = torch.matmul(mine.transpose(0, 1), k[:, h].T) * s["scale"]  # [group, queries, cached]
            score = score.masked_fill(hidden, -math.inf)
            p = torch.exp(score - score.amax(-1, keepdim=True))
            y = torch.matmul(p, v[:, h]) / p.sum(-1, keepdim=True)
            out[rows, h * group:(h + 1) * group] = y.transpose(0, 1).to(out.dtype)
    return out


def run(state):
    return {"table": _run_table, "rope": _run_rope, "write": _run_write, "read": _run_read,
            "attend": _run_attend}[state["op"]](state)


# -------------------------------------------------------------------------------------------- work
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    """Bytes: inputs read once, outputs written once. Of a table, the rows that the tokens' positions
    name. Operations: two for each multiply-add of a product."""
    op = case["op"]
    if op == "table":
        return {"bytes": case["positions"] * case["d"] * 4, "flops": 0}
    if op == "rope":
        return {"bytes": case["t"] * (case["heads"] * case["d"] * _SIZE[case["dtype"]] * 2 + 8 + case["d_rope"] * 4), "flops": 0}
    if op in ("write", "read"):
        rows = case["t"] if op == "write" else case["rows"]
        sides = 1 if case["shared"] else 2
        n = rows * case["heads"] * case["d"] * sides
        held = n // 2 + n // 32
        if op == "write":
            return {"bytes": n * _SIZE[case["dtype"]] + held + n * 2 + rows * 8, "flops": 0}
        return {"bytes": held + n * _SIZE[case["dtype"]] + rows * 8, "flops": 0}
    # the mean of the lengths that _lengths draws, one of them the longest
    b, longest, new, w = case["b"], case["longest"], case["new"], case["window"]
    mean = (longest + (b - 1) * (longest + max(new, 1, longest // 16)) / 2) / b
    queries = new if new else max(1.0, mean / 4)
    # pairs of a query and the tokens it sees; tokens that any query sees
    pairs = queries * min(mean - (queries - 1) / 2, w if w else math.inf)
    seen = min(mean, w + queries - 1 if w else math.inf)
    held = case["heads"] * (case["d"] // 2 + case["d"] // 32) * (1 if case["shared"] else 2)
    return {"bytes": int(b * (seen * held + 4 * queries * case["q_heads"] * case["d"])),
            "flops": int(4 * b * pairs * case["q_heads"] * case["d"])}


# ------------------------------------------------------------------------------- definition, 64 bits
def _decoded(codes, scales):
    """Values by the formats' definition: sign, exponent and mantissa fields, and the scale's power of two."""
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).int()
    m, e = (q & 1).double() / 2, (q >> 1) & 3
    power = torch.tensor([2.0**i for i in range(-127, 129)], dtype=torch.float64, device=codes.device)
    v = torch.where(e == 0, m, (1 + m) * power[(e - 1 + 127).clamp(min=0).long()])
    return torch.where(q >= 8, -v, v) * power[scales.long()].repeat_interleave(32, -1)


def _nearest(x):
    """The values that 32-blocks of x are held as."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    power = torch.tensor([2.0**i for i in range(-200, 201)], dtype=torch.float64, device=x.device)
    e = torch.bucketize(amax, power, right=True) - 1 - 200  # the largest power of two that amax reaches
    unit = power[torch.where(amax > 0, (e - 2).clamp(min=-127), -127) + 200]
    a = b.abs() / unit
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step).mul(step).clamp(max=6).mul(unit), b).reshape(x.shape)


def _exact_table(s):
    d, out = s["d"], torch.empty(s["positions"], s["d"], dtype=torch.float64, device="cuda")
    p = torch.arange(s["positions"], dtype=torch.float64, device="cuda")
    for i in range(d // 2):
        f = math.exp(-2 * i / d * math.log(s["base"]))
        if s["scaling"] == "linear":
            f /= s["factor"]
        elif s["scaling"] == "yarn":
            lo, hi = (d / 2 * math.log(s["original"] / (2 * math.pi * turns), s["base"]) for turns in (32, 1))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), d - 1)
            keep = 1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f *= keep + (1 - keep) / s["factor"]
        out[:, i] = torch.cos(p * f) * s["magnitude"]
        out[:, i + d // 2] = torch.sin(p * f) * s["magnitude"]
    return out


def _exact_rope(s):
    """Each pair as a complex number, times the unit number of its angle."""
    n, first = s["d_rope"], s["d"] - s["d_rope"] if s["last"] else 0
    x = s["x"].double()
    part = x[..., first:first + n].reshape(*x.shape[:-1], *((n // 2, 2) if s["interleaved"] else (2, n // 2)))
    at = -1 if s["interleaved"] else -2
    z = torch.complex(*part.unbind(at))
    cs = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(cs[:, :n // 2], cs[:, n // 2:])[:, None]
    z = z * (turn.conj() if s["inverse"] else turn)
    out = x.clone()
    out[..., first:first + n] = torch.stack([z.real, z.imag], at).reshape(*x.shape[:-1], n)
    return out


def _exact_attend(s):
    cache, heads, group = s["cache"], s["heads"], s["q_heads"] // s["heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for i in range(s["b"]):
        n, o = s["lengths_list"][i], s["offsets_list"]
        pages = s["table"][i, :(n + s["page"] - 1) // s["page"]].long()
        held = {name: pool[pages].transpose(0, 1).reshape(heads, -1, pool.shape[3])[:, :n] for name, pool in cache.items()}
        k = _decoded(held["k"], held["k_scales"])
        v = _decoded(held["v"], held["v_scales"]) if "v" in held else k
        q = s["q"][o[i]:o[i + 1]].double().unflatten(1, (heads, group))
        step = max(1, 2**27 // (heads * group * n))
        for j in range(0, len(q), step):
            x = torch.einsum("qhgd,hnd->hgqn", q[j:j + step], k) * s["scale"]
            at = torch.arange(n - len(q) + j, n - len(q) + j + x.shape[2], device="cuda")[:, None]
            gap = at - torch.arange(n, device="cuda")
            x = torch.where((gap >= 0) & (gap < (s["window"] or n + 1)), x, -math.inf)
            out[o[i] + j:o[i] + j + x.shape[2]] = torch.einsum("hgqn,hnd->qhgd", torch.softmax(x, -1), v).flatten(1, 2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        return _exact_table(s)
    if op == "rope":
        return _exact_rope(s)
    if op == "write":
        out = {"k_values": _nearest(s["k"])}
        if s["v"] is not None:
            out["v_values"] = _nearest(s["v"])
        return {**out, **{name: None for name in s["cache"]}}
    if op == "read":
        c = s["cache"]
        return {n: _decoded(_load(c[n], s["slots"]), _load(c[n + "_scales"], s["slots"])) for n in ("k", "v") if n in c}
    return _exact_attend(s)
