"""The MXFP4 and expert operators as they are measured: cases, plain forms, and definitions in 64 bits.

Five operators that belong together in a layer of experts whose weights are held in MXFP4
(E2M1 elements, one UE8M0 power-of-two scale per 32 elements along K):

  quantize   bf16 / fp16 / fp32 rows -> packed MXFP4 codes, scales and the values they stand for
  product    MXFP8 or MXFP4 activations x MXFP4 weights -> bf16
  route      router logits -> experts, weights, and the order of the rows by expert
  experts    rows gathered by expert x that expert's MXFP4 weights (optionally silu(gate) * up)
  combine    weighted sum of each token's expert rows -> bf16

`run` makes the framework's calls where `own` is true; otherwise it computes the same in elementary
torch operations in 32 bits (64 where the router's selection depends on values next to a border).
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
def _quantize(m, k, dtype="bf16", pad=0):
    return {"op": "quantize", "m": m, "k": k, "dtype": dtype, "pad": pad}


def _product(m, n, k, act):
    return {"op": "product", "m": m, "n": n, "k": k, "act": act}


def _route(t, e, k, scoring, groups=1, top_groups=1, bias=False, dtype="fp32"):
    return {"op": "route", "t": t, "e": e, "k": k, "scoring": scoring, "groups": groups,
            "top_groups": top_groups, "bias": bias, "dtype": dtype}


def _experts(t, e, k, n, kk, act, gated, gather=True):
    return {"op": "experts", "t": t, "e": e, "k": k, "n": n, "kk": kk, "act": act, "gated": gated, "gather": gather}


def _combine(t, k, n, residual):
    return {"op": "combine", "t": t, "k": k, "n": n, "residual": residual}


def listed():
    return [
        # one decode token's activation before a 4-bit product
        {"name": "quantize one row", **_quantize(1, 5120)},
        # a long prompt's activations, or a weight matrix laid out once
        {"name": "quantize 16381 rows", **_quantize(16381, 8192)},
        # the first projection of a decode step, weights in 4 bits, activations as the chain keeps them
        {"name": "product 1 row, 8-bit rows", **_product(1, 2048, 5120, "mx8")},
        # the second projection for a batch of eight, both operands in 4 bits
        {"name": "product 8 rows, 4-bit rows", **_product(8, 8192, 1536, "mx4")},
        # the third projection for a ragged batch of requests
        {"name": "product 201 rows, 8-bit rows", **_product(201, 5120, 8192, "mx8")},
        # a prompt through a wide projection
        {"name": "product 8192 rows, 4-bit rows", **_product(8192, 8192, 5120, "mx4")},
        # one decode token's experts
        {"name": "route 1 token", **_route(1, 256, 8, "sigmoid", 8, 4, True)},
        # a batch of prompts' experts
        {"name": "route 16384 tokens", **_route(16384, 256, 8, "sigmoid", 8, 4, True)},
        # eight decode tokens through the experts' first product: most experts read for one row
        {"name": "experts 8 tokens", **_experts(8, 64, 6, 4096, 2048, "mx8", True)},
        # a prompt through the experts' first product
        {"name": "experts 4093 tokens", **_experts(4093, 64, 8, 4096, 4096, "mx8", True)},
        # the sum over one decode token's experts
        {"name": "combine 1 token", **_combine(1, 8, 5120, False)},
        # the sum over a prompt's experts, with the residual stream
        {"name": "combine 8191 tokens", **_combine(8191, 8, 5120, True)},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _of128(rng, lo, hi):
    return 128 * _log(rng, lo // 128, hi // 128)


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "route", "experts", "experts", "combine"])
    if op == "quantize":
        k = 32 * _log(rng, 1, 512)
        m = _log(rng, 1, min(65536, 16381 * 8192 // k))
        return _quantize(m, k, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice([0, 0, 8, 520]))
    if op == "product":
        n, k = _of128(rng, 128, 16384), _of128(rng, 128, 16384)
        m = _log(rng, 1, max(1, min(16384, 8192 * 8192 * 5120 // (n * k))))
        return _product(m, n, k, rng.choice(["mx8", "mx4"]))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        size = _log(rng, 4, 512 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * size))
        return _route(_log(rng, 1, 16384), groups * size, k, rng.choice(["sigmoid", "softmax"]), groups, top_groups,
                      rng.random() < 0.6, rng.choice(["fp32", "bf16"]))
    if op == "experts":
        e = _log(rng, 2, 128)
        k = rng.randint(1, min(8, e))
        kk = _of128(rng, 256, 8192)
        n = 128 * _log(rng, 1, max(1, min(64, 2**30 // (e * kk * 128))))
        t = _log(rng, 1, max(1, min(8192, 4093 * 8 * 4096 * 4096 // (k * n * kk))))
        return _experts(t, e, k, n, kk, rng.choice(["mx8", "mx4"]), rng.random() < 0.5, rng.random() < 0.7)
    n = 8 * _log(rng, 16, 1024)
    k = rng.randint(1, 12)
    return _combine(_log(rng, 1, max(1, min(16384, 8191 * 8 * 5120 // (k * n)))), k, n, rng.random() < 0.5)


# ----------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (2**63))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, m, k, spread=2):
    """Activation-like rows: normal values whose size varies from block to block, a few blocks all zero."""
    x = _normal(g, m, k // 32, 32)
    u = torch.randint(-spread, spread + 1, (m, k // 32, 1), generator=g, device="cuda")
    alive = torch.rand(m, k // 32, 1, generator=g, device="cuda") > 0.002
    return (torch.ldexp(x, u) * alive).reshape(m, k)


def _routing(g, t, e, k):
    """Experts of t tokens (some experts favoured, some left without rows), sorted by expert:
    offsets [e + 1], the token of each sorted row, the sorted row of each (token, choice)."""
    liked = _normal(g, t, e) + 0.7 * _normal(g, e)
    chosen = liked.topk(k, dim=1).indices
    return _order(chosen, e)


def _order(chosen, e):
    flat = chosen.reshape(-1)
    by = torch.sort(flat, stable=True).indices
    counts = torch.zeros(e, dtype=torch.int64, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    slots = torch.empty_like(by).scatter_(0, by, torch.arange(by.numel(), device=by.device))
    return offsets, (by // chosen.shape[1]).int(), slots.reshape(chosen.shape).int()


def _swizzle(s):
    """Scale bytes [.., rows, K / 32] in the 128x4 layout of block scales (rows % 128 padded with zeros)."""
    rows, c = s.shape
    s = torch.nn.functional.pad(s, (0, -c % 4, 0, -rows % 128))
    r, c = s.shape
    return s.reshape(r // 128, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _activations(g, m, k, act):
    x = _rows(g, m, k).bfloat16().float()
    return _mx8(x) if act == "mx8" else _mx4(x)


def prepare(case, seed):
    g, s = _generator(seed), dict(case)
    if own:
        s["mx"], s["h"] = _handle()
    op = case["op"]
    if op == "quantize":
        wide = _rows(g, case["m"], case["k"], 6).to(_TYPES[case["dtype"]])
        if case["pad"]:  # the left columns of wider rows, as a split projection's output
            wide = torch.nn.functional.pad(wide, (0, case["pad"]), value=1.0)
        s["x"] = wide[:, :case["k"]]
    elif op == "product":
        s["a"], plain = _activations(g, case["m"], case["k"], case["act"])
        s["a_plain"], s["a_scales"] = plain, _swizzle(plain)
        s["w"], plain = _mx4(_normal(g, case["n"], case["k"]) * 0.03)
        s["w_plain"], s["w_scales"] = plain, _swizzle(plain)
    elif op == "route":
        # float32 from a linear layer, or what a bf16 router keeps; some experts are masked for some
        # tokens, and a few tokens (padding) have every expert masked
        logits = 1.5 * _normal(g, case["t"], case["e"])
        logits[torch.rand(logits.shape, generator=g, device="cuda") < 0.01] = -math.inf
        logits[torch.rand(case["t"], generator=g, device="cuda") < 0.003] = -math.inf
        s["logits"] = logits.to(_TYPES[case["dtype"]])
        s["bias"] = 0.1 * _normal(g, case["e"]) if case["bias"] else None
    elif op == "experts":
        s["offsets"], tokens, _ = _routing(g, case["t"], case["e"], case["k"])
        s["tokens"] = tokens if case["gather"] else None
        s["a"], s["a_scales"] = _activations(g, case["t"] * (1 if case["gather"] else case["k"]), case["kk"], case["act"])
        w, plain = _mx4(_normal(g, case["e"] * case["n"], case["kk"]) * 0.03)
        s["w"] = w.reshape(case["e"], case["n"], -1)
        s["w_plain"] = plain.reshape(case["e"], case["n"], -1)
        s["w_scales"] = _swizzle(plain).reshape(case["e"], -1)
    else:
        t, k, n = case["t"], case["k"], case["n"]
        s["slots"] = _routing(g, t, max(16, k), k)[2]
        s["y"] = _normal(g, t * k, n).bfloat16()
        s["weights"] = torch.rand(t, k, generator=g, device="cuda") + 0.05
        s["residual"] = _normal(g, t, n).bfloat16() if case["residual"] else None
    return s


# ------------------------------------------------------------------------------------- plain forms
def _scale_bytes(x, largest):
    """UE8M0 byte of each 32-block of float32 x [.., blocks, 32]: floor(log2 amax) - largest + 127 from
    amax's exponent field, at least 0; 255 for a block that is not finite."""
    amax = x.abs().amax(-1)
    field = (amax.view(torch.int32) >> 23) & 255
    return torch.where(torch.isfinite(amax), (field - largest).clamp(min=0), 255).to(torch.uint8)


def _scaled(x, s):
    """Blocks times 2^(127 - s), and zero where the block is not finite."""
    bad = (s == 255).unsqueeze(-1)
    return torch.where(bad, 0.0, x) * ((254 - s.int()) << 23).view(torch.float32).unsqueeze(-1), bad


def _mx8(x):
    """float32 [m, k] -> (E4M3 codes uint8 [m, k], scale bytes [m, k / 32])."""
    b = x.reshape(x.shape[0], -1, 32)
    s = _scale_bytes(b, 8)
    y, bad = _scaled(b, s)
    codes = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(bad, 0x7F, codes).to(torch.uint8).reshape(x.shape), s


def _codes4(a):
    """Magnitude codes 0..7 of a >= 0, to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    return ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5).byte())


def _mx4(x):
    """float32 [m, k] -> (E2M1 codes, two to a byte, the first in the low bits, [m, k / 2]; scale bytes [m, k / 32])."""
    b = x.reshape(x.shape[0], -1, 32)
    s = _scale_bytes(b, 2)
    y, bad = _scaled(b, s)
    c = _codes4(y.abs()) + torch.signbit(y).byte() * 8
    c = torch.where(bad, 0, c).reshape(x.shape[0], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), s


def _values4(q, s):
    """float32 values of packed E2M1 codes [.., k / 2] under scale bytes [.., k / 32]."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    two = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)
    v = two[q.int()].reshape(*s.shape, 32)
    return (v * _power(s).unsqueeze(-1)).reshape(*q.shape[:-1], -1)


def _values8(q, s):
    v = q.view(torch.float8_e4m3fn).float().reshape(*s.shape, 32)
    return (v * _power(s).unsqueeze(-1)).reshape(q.shape)


def _power(s):
    """2^(s - 127) exactly, from its bits (2^-127 is subnormal); NaN for 255."""
    bits = torch.where(s == 0, 0x00400000, s.int() << 23)
    return torch.where(s == 255, math.nan, bits.int().view(torch.float32))


def _values(q, s, act):
    return _values8(q, s) if act == "mx8" else _values4(q, s)


def _run_quantize(s):
    if own:
        q, scales, y = s["mx"].mx_quantize_rows_fp4(s["h"], s["x"], swizzled=False, y=True)
        return {"codes": q, "scales": scales, "values": y}
    q, scales = _mx4(s["x"].float())
    return {"codes": q, "scales": scales, "values": _values4(q, scales).bfloat16()}


def _run_product(s):
    if own:
        return s["mx"].mx_gemm_fp4(s["h"], s["a"], s["a_scales"], s["w"], s["w_scales"])
    return (_values(s["a"], s["a_plain"], s["act"]) @ _values4(s["w"], s["w_plain"]).T).bfloat16()


def _run_route(s):
    e, k, groups, top_groups = s["e"], s["k"], s["groups"], s["top_groups"]
    if own:
        r = s["mx"].mx_route(s["h"], s["logits"], k, bias=s["bias"], scoring=s["scoring"], n_groups=groups,
                             topk_groups=top_groups, renormalize=True, scale=2.5)
        return {n: r[n] for n in ("experts", "weights", "offsets", "tokens", "slots")}
    # selection in 64 bits: neighbouring scores differ by less than 32 bits hold
    x = s["logits"].double()
    if s["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        ex = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        score = ex / ex.sum(1, keepdim=True).clamp(min=1e-300)
    # without a bias the scores' order is the logits' order
    key = x if s["bias"] is None else torch.where(x == -math.inf, -math.inf, score + s["bias"].double())
    if groups > 1:
        ranked = torch.sort(key.reshape(-1, groups, e // groups), dim=2, descending=True).values
        best = ranked[..., 0] if s["bias"] is None else ranked[..., :2].sum(2)
        first = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :top_groups]
        open_ = torch.zeros_like(best, dtype=torch.bool).scatter_(1, first, True).repeat_interleave(e // groups, 1)
    else:
        open_ = torch.ones_like(key, dtype=torch.bool)
    # experts of closed groups come after every open one, masked experts included
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(open_.gather(1, order).byte(), dim=1, descending=True, stable=True).indices)
    chosen = order[:, :k]
    w = score.gather(1, chosen)
    w = 2.5 * w / w.sum(1, keepdim=True).clamp(min=1e-300)
    offsets, tokens, slots = _order(chosen, e)
    return {"experts": chosen.int(), "weights": w.float(), "offsets": offsets, "tokens": tokens, "slots": slots}


def _run_experts(s):
    if own:
        return s["mx"].mx_gemm_fp4_grouped(s["h"], s["a"], s["a_scales"], s["w"], s["w_scales"], s["offsets"],
                                           tokens=s["tokens"], gated=s["gated"])
    a, w = _values(s["a"], s["a_scales"], s["act"]), _values4(s["w"], s["w_plain"])
    x = a if s["tokens"] is None else a[s["tokens"].long()]
    # each expert's rows, padded to the largest count, in one batched product
    off = s["offsets"].long()
    most = int((off[1:] - off[:-1]).max())
    at = off[:-1, None] + torch.arange(most, device=off.device)
    inside = at < off[1:, None]
    y = torch.matmul(x[at.clamp(max=x.shape[0] - 1)], w.transpose(1, 2))[inside]
    if s["gated"]:  # rows 2i and 2i + 1 of the weights are gate i and up i
        y = y[:, 0::2] / (1 + torch.exp(-y[:, 0::2])) * y[:, 1::2]
    return y.bfloat16()


def _run_combine(s):
    if own:
        return s["mx"].mx_combine(s["h"], s["y"], s["slots"], s["weights"], residual=s["residual"])
    out = (s["y"][s["slots"].long()].float() * s["weights"].unsqueeze(-1)).sum(1)
    return (out if s["residual"] is None else out + s["residual"].float()).bfloat16()


def run(state):
    return {"quantize": _run_quantize, "product": _run_product, "route": _run_route, "experts": _run_experts,
            "combine": _run_combine}[state["op"]](state)


# -------------------------------------------------------------------------------------------- work
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def work(case):
    """Bytes: inputs read once, outputs written once. An expert's weights count when a row reaches it (at most
    t * k experts). Operations: two for each multiply-add of a product."""
    op = case["op"]
    bits = lambda rows, k, b: rows * k * b // 8 + rows * k // 32  # noqa: E731
    if op == "quantize":
        mk = case["m"] * case["k"]
        return {"bytes": mk * _SIZE[case["dtype"]] + bits(case["m"], case["k"], 4) + mk * 2, "flops": 0}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": bits(m, k, 8 if case["act"] == "mx8" else 4) + bits(n, k, 4) + m * n * 2, "flops": 2 * m * n * k}
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        return {"bytes": t * e * _SIZE[case["dtype"]] + (e * 4 if case["bias"] else 0) + t * k * 16 + (e + 1) * 4,
                "flops": 0}
    if op == "experts":
        t, e, k, n, kk = case["t"], case["e"], case["k"], case["n"], case["kk"]
        a = bits(t if case["gather"] else t * k, kk, 8 if case["act"] == "mx8" else 4)
        out = t * k * (n // 2 if case["gated"] else n) * 2
        return {"bytes": a + bits(min(e, t * k) * n, kk, 4) + out + t * k * 4 * case["gather"] + (e + 1) * 4,
                "flops": 2 * t * k * n * kk}
    t, k, n = case["t"], case["k"], case["n"]
    return {"bytes": t * k * (n * 2 + 8) + t * n * 2 * (2 if case["residual"] else 1), "flops": 2 * t * k * n}


# ------------------------------------------------------------------------------- definition, 64 bits
def _powers64(device):
    """2^-200 .. 2^200."""
    return torch.tensor([2.0**i for i in range(-200, 201)], dtype=torch.float64, device=device)


def _decode64(q, s, act):
    """Values of codes by the formats' definition: sign, exponent and mantissa fields."""
    if act == "mx4":
        q = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    top, mant, bias = (3, 3, 7) if act == "mx8" else (2, 1, 1)  # exponent bits - 1, mantissa bits, bias
    q = q.int()
    m, e = q & ((1 << mant) - 1), (q >> mant) & ((1 << (top + (act == "mx8"))) - 1)
    f = m.double() / (1 << mant)
    power = _powers64(q.device)
    v = torch.where(e == 0, f * 2.0 ** (1 - bias), (1 + f) * power[e - bias + 200])
    v = torch.where((q >> (7 if act == "mx8" else 3)) > 0, -v, v)
    return v * power[s.int() - 127 + 200].repeat_interleave(32, -1)


def _exact_quantize(s):
    x = s["x"].double().reshape(s["m"], -1, 32)
    amax = x.abs().amax(-1, keepdim=True)
    power = _powers64(x.device)
    e = torch.bucketize(amax, power, right=True) - 1 - 200  # the largest power of two that amax reaches
    unit = power[torch.where(amax > 0, (e - 2).clamp(min=-127), -127) + 200]
    a = x.abs() / unit
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.round(a / step).mul(step).clamp(max=6).mul(unit)
    return {"codes": None, "scales": None, "values": torch.copysign(v, x).reshape(s["m"], s["k"])}


def _exact_route(s):
    x = s["logits"].double()
    score = torch.sigmoid(x) if s["scoring"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
    key = x
    if s["bias"] is not None:
        key = (score + s["bias"].double()).masked_fill(x == -math.inf, -math.inf)
    # ranks by counting: an expert comes after every expert of a larger key, and of the same key and a lower index
    t, e, groups = s["t"], s["e"], s["groups"]
    parts = key.reshape(t, groups, -1)
    if groups > 1:
        best = parts.amax(2) if s["bias"] is None else parts.topk(min(2, e // groups), dim=2).values.sum(2)
        shut = (_rank(best) >= s["top_groups"]).repeat_interleave(e // groups, 1)
    else:
        shut = torch.zeros_like(key, dtype=torch.bool)
    rank = torch.cat([_rank(k, z) for k, z in zip(key.split(512), shut.split(512))])
    experts = torch.empty(t, e, dtype=torch.int64, device=x.device)
    experts.scatter_(1, rank, torch.arange(e, device=x.device).expand(t, e).contiguous())
    w = torch.gather(score, 1, experts[:, :s["k"]])
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, 2.5 * w / torch.where(total > 0, total, 1.0), 0.0)
    return {"experts": None, "weights": w, "offsets": None, "tokens": None, "slots": None}


def _rank(key, shut=None):
    a, b = key.unsqueeze(2), key.unsqueeze(1)  # [t, i, 1], [t, 1, j]
    i = torch.arange(key.shape[1], device=key.device)
    before = (b > a) | ((b == a) & (i[None, :] < i[:, None]))
    if shut is not None:
        za, zb = shut.unsqueeze(2), shut.unsqueeze(1)
        before = (za & ~zb) | (before & (za == zb))
    return before.sum(2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s)
    if op == "product":
        return _decode64(s["a"], s["a_plain"], s["act"]) @ _decode64(s["w"], s["w_plain"], "mx4").T
    if op == "route":
        return _exact_route(s)
    if op == "experts":
        off, a, out = s["offsets"].tolist(), _decode64(s["a"], s["a_scales"], s["act"]), []
        for i in range(s["e"]):
            rows = slice(off[i], off[i + 1])
            x = a[rows] if s["tokens"] is None else a[s["tokens"][rows].long()]
            y = x @ _decode64(s["w"][i], s["w_plain"][i], "mx4").T if len(x) else x.new_zeros(0, s["n"])
            if s["gated"]:
                y = y.reshape(len(y), s["n"] // 2, 2)
                y = y[..., 0] * torch.sigmoid(y[..., 0]) * y[..., 1]
            out.append(y)
        return torch.cat(out)
    out = torch.einsum("tk,tkn->tn", s["weights"].double(), s["y"].double()[s["slots"].long()])
    return out if s["residual"] is None else out + s["residual"].double()
