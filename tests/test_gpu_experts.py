"""Routing, the experts' grouped product and the weighted sum against the float64 oracle.

Selections and row orders are whole numbers and equal the oracle's. Weights: a float32
exp of an argument of size d is off by at most (2 + d) units, the sum of the scores and
the divisions by a few more: (40 + d) 2^-23 of the value bounds them. Products as in
test_gpu_fp4; the gate adds the float32 exp (2 + 1.2 |g| units) and a division."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import dev, handle
from oracle import experts as ox
from test_gpu_fp4 import guarded, intact, on_gpu, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    handle()
    import mxfp8_block_scaled_06_gb300 as mod

    return mod


def check_route(mx, logits, top_k, **kw):
    """logits: a device tensor; compares every output of the call with the oracle."""
    t, e = logits.shape
    bias = kw.get("bias")
    got = mx.mx_route(handle(), logits, top_k, **{**kw, "bias": None if bias is None else on_gpu(bias)})
    w, experts = ox.route(logits.double().cpu().numpy(), top_k, **kw)
    assert np.array_equal(got["experts"].cpu().numpy(), experts)
    offsets, tokens, slots = ox.row_order(experts, e)
    assert np.array_equal(got["offsets"].cpu().numpy(), offsets)
    assert np.array_equal(got["tokens"].cpu().numpy(), tokens)
    assert np.array_equal(got["slots"].cpu().numpy(), slots)
    x = logits.double().cpu().numpy()
    x = x[np.isfinite(x)]
    d = np.ptp(x) if x.size else 0.0
    err = np.abs(got["weights"].cpu().numpy().astype(np.float64) - w)
    assert (err <= (40 + d) * 2.0**-23 * np.abs(w) + 1e-30).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("t,e,k,groups,top", [(1, 256, 8, 8, 4), (1, 1, 1, 1, 1), (2, 512, 32, 1, 1), (33, 37, 5, 1, 1),
                                              (31, 60, 3, 5, 2), (64, 64, 6, 4, 1), (257, 96, 8, 3, 3), (40, 512, 10, 32, 7),
                                              (1000, 128, 4, 16, 2), (100, 8, 8, 8, 8)])
def test_route(mx, t, e, k, groups, top, bias, scoring):
    rng = np.random.default_rng(t + e)
    logits = on_gpu((2 * rng.standard_normal((t, e))).astype(np.float32))
    b = (0.2 * rng.standard_normal(e)).astype(np.float32) if bias else None
    check_route(mx, logits, k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top, scale=1.5)


@pytest.mark.parametrize("bias", [False, True])
def test_route_ties(mx, bias):
    """bf16 logits on a coarse grid: most selections meet equal logits, and with a bias keys that
    only float64 tells apart."""
    rng = np.random.default_rng(11)
    logits = on_gpu((rng.integers(-4, 5, (300, 128)) / 2).astype(np.float32)).bfloat16()
    b = (rng.integers(0, 3, 128) * 2.0**-26).astype(np.float32) if bias else None
    for groups, top in ((1, 1), (8, 3)):
        check_route(mx, logits, 7, bias=b, scoring="sigmoid", n_groups=groups, topk_groups=top)
        check_route(mx, logits, 7, bias=b, scoring="softmax", n_groups=groups, topk_groups=top)


def test_route_neighbours_of_one_unit(mx):
    """Keys a float32 unit and less apart: s(x) + b of different (x, b) with the same float32 sum."""
    rng = np.random.default_rng(12)
    x = rng.standard_normal((200, 64))
    b = 0.5 - 1 / (1 + np.exp(-x[0]))  # row 0's keys are all 0.5 but for the roundings of b
    logits = np.repeat(x[:1], 200, 0) + rng.integers(-2, 3, (200, 64)) * 2.0**-24
    check_route(mx, on_gpu(logits.astype(np.float32)), 8, bias=b.astype(np.float32), scoring="sigmoid")
    check_route(mx, on_gpu(logits.astype(np.float32)), 4, bias=b.astype(np.float32), scoring="sigmoid", n_groups=8,
                topk_groups=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masks_and_extremes(mx, bias, scoring):
    rng = np.random.default_rng(13)
    x = rng.standard_normal((64, 48)).astype(np.float32)
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2] = np.finfo(np.float32).min
    x[3, 7] = np.inf
    x[4, 5] = np.nan
    x[5] = 80.0
    x[6] = -120.0
    x[7, ::2], x[7, 1::2] = -0.0, 0.0
    b = (0.1 * rng.standard_normal(48)).astype(np.float32) if bias else None
    for groups, top, k in ((1, 1, 6), (6, 2, 6), (6, 6, 20)):
        check_route(mx, on_gpu(x), k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top)
    check_route(mx, on_gpu(x), 6, bias=b, scoring=scoring, renormalize=False, scale=0.25)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, "numbers", "some -inf"])
@pytest.mark.parametrize("e,k,groups,top", [(512, 16, 1, 1), (512, 16, 8, 2), (96, 32, 1, 1), (160, 5, 5, 1), (70, 9, 7, 3)])
def test_route_fewer_experts_than_choices(mx, e, k, groups, top, bias, scoring):
    """Rows with 0 to k + 2 experts that are not masked, anywhere, or in the first or last places."""
    rng = np.random.default_rng(e + k)
    x = np.full((4 * (k + 3), e), -np.inf)
    for r in range(len(x)):
        n = r // 4
        at = (rng.permutation(e)[:n], np.arange(n), np.arange(e - n, e), 32 * np.arange(n) % e)[r % 4]
        x[r, at] = 2 * rng.standard_normal(n)
    b = None if bias is None else (0.2 * rng.standard_normal(e)).astype(np.float32)
    if bias == "some -inf":
        b[rng.random(e) < 0.7] = -np.inf
    check_route(mx, on_gpu(x.astype(np.float32)), k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top)


@pytest.mark.parametrize("t", [16384, 20011])
def test_route_many_tokens(mx, t):
    rng = np.random.default_rng(t)
    logits = on_gpu(rng.standard_normal((t, 16)).astype(np.float32))
    check_route(mx, logits, 2, bias=(0.1 * rng.standard_normal(16)).astype(np.float32), scoring="softmax")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("t,e,k,groups,top", [(1100, 256, 8, 8, 4), (1024, 64, 6, 1, 1), (1031, 96, 16, 3, 2),
                                              (1500, 128, 1, 8, 1), (1200, 240, 5, 5, 5), (1025, 256, 17, 2, 1),
                                              (1333, 16, 4, 1, 1), (1027, 256, 4, 16, 3), (1026, 200, 4, 1, 1)])
def test_route_over_a_thousand_tokens(mx, t, e, k, groups, top, bias, scoring):
    rng = np.random.default_rng(t * e)
    x = 2 * rng.standard_normal((t, e))
    x[rng.random((t, e)) < 0.02] = -np.inf
    x[::97] = -np.inf
    x[5::131, 1:] = -np.inf
    x[3, 0], x[4, 1] = np.nan, np.inf
    b = (0.2 * rng.standard_normal(e)).astype(np.float32) if bias else None
    logits = on_gpu(x.astype(np.float32))
    check_route(mx, logits, k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top, scale=2.5)
    check_route(mx, logits.bfloat16(), k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top, renormalize=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_close_keys_over_a_thousand_tokens(mx, scoring):
    """As the tests of ties and of neighbours, in many blocks."""
    rng = np.random.default_rng(15)
    grid = on_gpu((rng.integers(-4, 5, (1100, 128)) / 2).astype(np.float32))
    tiny = (rng.integers(0, 3, 128) * 2.0**-26).astype(np.float32)
    for b in (None, tiny):
        for groups, top in ((1, 1), (8, 3)):
            check_route(mx, grid.bfloat16(), 7, bias=b, scoring=scoring, n_groups=groups, topk_groups=top)
    x = rng.standard_normal(64)
    b = (0.5 - 1 / (1 + np.exp(-x))).astype(np.float32)
    near = on_gpu((x + rng.integers(-2, 3, (1060, 64)) * 2.0**-24).astype(np.float32))
    check_route(mx, near, 8, bias=b, scoring=scoring)
    check_route(mx, near, 4, bias=b, scoring=scoring, n_groups=4, topk_groups=2)
    # equal logits: more candidates than there are lanes; odd strides
    check_route(mx, torch.zeros((1100, 256), device=dev()), 8, bias=np.zeros(256, np.float32), scoring=scoring)
    check_route(mx, torch.zeros((1100, 64), device=dev()), 3, scoring=scoring)
    wide = on_gpu(rng.standard_normal((1100, 131)).astype(np.float32))
    check_route(mx, wide[:, 3:131], 6, bias=np.zeros(128, np.float32), scoring=scoring)


def test_route_strides_types_and_guards(mx):
    rng = np.random.default_rng(14)
    wide = on_gpu(rng.standard_normal((70, 101)).astype(np.float32))
    check_route(mx, wide[:, 3:44], 4, scoring="sigmoid")
    check_route(mx, wide.bfloat16()[:, 1:42], 4)
    t, e, k = 70, 41, 3
    sizes = dict(weights=t * k, experts=t * k, offsets=e + 1, tokens=t * k, slots=t * k)
    bufs = {n: guarded(4 * c) for n, c in sizes.items()}
    outs = {n: b[1].view(torch.float32 if n == "weights" else torch.int32) for n, b in bufs.items()}
    mx.mx_route(handle(), wide[:, :e], k, **outs)
    torch.cuda.synchronize()
    assert all(intact(bufs[n][0], 4 * c) for n, c in sizes.items())


def experts_case(rng, counts, rows_a, k, n, fp4, gather):
    e = len(counts)
    r = int(sum(counts))
    rows = rows_a if gather else r
    aq, as_, av = operand(rng, rows, k, fp4, 2)
    ws = [operand(rng, n, k, True, 2) for _ in range(e)]
    tokens = rng.integers(0, rows, r) if gather else np.arange(r)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    args = dict(a=on_gpu(aq), a_scales=on_gpu(as_), w=on_gpu(np.stack([w[0] for w in ws])),
                w_scales=on_gpu(np.stack([oracle.swizzle_scales(w[1]).reshape(-1) for w in ws])),
                offsets=on_gpu(offsets.astype(np.int32)),
                tokens=on_gpu(tokens.astype(np.int32)) if gather else None)
    x = av[tokens]
    which = np.repeat(np.arange(e), counts)
    ref = np.stack([ws[which[i]][2] @ x[i] for i in range(r)])
    size = np.stack([np.abs(ws[which[i]][2]) @ np.abs(x[i]) for i in range(r)])
    return args, ref, k * 2.0**-22 * size


def check_grouped(mx, counts, rows_a, k, n, gather, fp4, gated):
    rng = np.random.default_rng(sum(counts) + k)
    args, y, err = experts_case(rng, counts, rows_a, k, n, fp4, gather)
    r, cols = len(y), n // 2 if gated else n
    ob, o = guarded(r * cols * 2)
    out = mx.mx_gemm_fp4_grouped(handle(), gated=gated, out=o.view(torch.bfloat16).view(r, cols), **args)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    ref, tol = y, err
    if gated:
        g, u, eg, eu = y[:, 0::2], y[:, 1::2], err[:, 0::2], err[:, 1::2]
        ref = ox.silu_gate(y)
        with np.errstate(over="ignore"):
            sg = np.abs(g / (1 + np.exp(-g)))
        tol = 1.1 * eg * np.abs(u) + (sg + 1.1 * eg) * eu + (6 + 1.2 * np.abs(g)) * 2.0**-22 * np.abs(ref)
    tol = tol + 2.0**-8 * (np.abs(ref) + tol) + 1e-37
    d = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (d <= tol).all(), (d / tol).max()
    assert intact(ob, r * cols * 2)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,k,n", [([200, 90, 0, 431], 640, 256), ([100, 160], 128, 512), ([70, 224, 225], 256, 256),
                                        ([97], 1408, 768), ([0, 0, 500, 0], 896, 256), ([97, 31], 384, 384)])
def test_grouped_product_of_wide_tiles(mx, counts, k, n, gather, fp4, gated):
    """Pairs of SMs (256 weight rows at a time) and single ones (384), K of one stage and more."""
    check_grouped(mx, counts, 150, k, n, gather, fp4, gated)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,k,n", [([430, 0, 215, 900, 417], 1024, 640), ([3000], 2048, 128), ([1700, 5, 224], 640, 1920)])
def test_grouped_product_of_the_widest_tiles(mx, counts, k, n, gather, fp4):
    """Tiles of 200 rows and more with one CTA to an SM: the shortest rings, over many stages."""
    check_grouped(mx, counts, 800, k, n, gather, fp4, False)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("counts,rows_a,k,n,gather", [
    ([1], 1, 128, 128, True), ([0, 3, 0, 0, 1, 0], 4, 384, 256, True), ([1] * 40, 8, 512, 128, True),
    ([5, 16, 17, 0, 33, 2], 30, 640, 256, True), ([130, 0, 1, 300], 200, 256, 128, True),
    ([224, 225, 448, 7], 500, 128, 128, True), ([3, 0, 50], 0, 896, 384, False), ([700, 13], 0, 256, 128, False)])
def test_grouped_product(mx, counts, rows_a, k, n, gather, fp4, gated):
    check_grouped(mx, counts, rows_a, k, n, gather, fp4, gated)


def test_grouped_rows_outside(mx):
    """Tokens that are not rows of a read as zero rows and are reported; offsets beyond the output are cut
    there; rows of no expert are not written."""
    rng = np.random.default_rng(3)
    args, y, err = experts_case(rng, [4, 0, 6], 5, 256, 128, False, True)
    args["tokens"][1], args["tokens"][7] = -3, 5
    args["offsets"] = on_gpu(np.array([2, 4, 4, 1000], np.int32))
    out = torch.full((10, 128), 7.0, dtype=torch.bfloat16, device=dev())
    mx.mx_gemm_fp4_grouped(handle(), out=out, **args)
    assert mx.mx_device_status(handle()) == mx.MX_ERR_INVALID_ARG
    assert mx.mx_device_status(handle()) == mx.MX_OK
    got = out.float().cpu().numpy()
    assert (got[:2] == 7).all() and (got[7] == 0).all()
    keep = [2, 3, 4, 5, 6, 8, 9]
    tol = 2.0**-8 * np.abs(y) + err * 1.01
    assert (np.abs(got - y) <= tol)[keep].all()


@pytest.mark.parametrize("t,k,n,residual,pad", [(1, 8, 5120, False, 0), (1, 1, 8, True, 0), (7, 3, 1032, True, 0),
                                               (65, 32, 128, False, 8), (300, 6, 2056, True, 64)])
def test_combine(mx, t, k, n, residual, pad):
    rng = np.random.default_rng(t * k)
    y = on_gpu(rng.standard_normal((t * k + 3, n + pad)).astype(np.float32)).bfloat16()[:, :n]
    slots = rng.integers(0, t * k + 3, (t, k))
    w = rng.random((t, k)).astype(np.float32)
    res = on_gpu(rng.standard_normal((t, n)).astype(np.float32)).bfloat16() if residual else None
    ob, o = guarded(t * n * 2)
    out = mx.mx_combine(handle(), y, on_gpu(slots.astype(np.int32)), on_gpu(w), residual=res,
                        out=o.view(torch.bfloat16).view(t, n))
    yv, rv = y.double().cpu().numpy(), None if res is None else res.double().cpu().numpy()
    ref = ox.combine(yv, slots, w, rv)
    size = ox.combine(np.abs(yv), slots, w, None if rv is None else np.abs(rv))
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= 2.0**-8 * np.abs(ref) + (k + 2) * 2.0**-23 * size).all()
    assert mx.mx_device_status(handle()) == mx.MX_OK and intact(ob, t * n * 2)
    if residual:  # in place
        mx.mx_combine(handle(), y, on_gpu(slots.astype(np.int32)), on_gpu(w), residual=res, out=res)
        assert torch.equal(res, out)


def test_grouped_product_past_32_bit_offsets(mx):
    """Five gigabytes of weights: rows of the first and of the last experts."""
    rng = np.random.default_rng(21)
    e, n, k, r = 40, 8192, 32768, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(0, 256, (e, n, k // 2), generator=g, device=dev(), dtype=torch.uint8)
    s = torch.randint(120, 124, (e, n * k // 32), generator=g, device=dev(), dtype=torch.uint8)
    aq, as_, av = operand(rng, r, k, True, 0)
    counts = np.zeros(e, np.int64)
    counts[[0, e - 2, e - 1]] = 1, 2, 2
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = mx.mx_gemm_fp4_grouped(handle(), on_gpu(aq), on_gpu(as_), w, s, on_gpu(offsets)).double().cpu().numpy()
    assert mx.mx_device_status(handle()) == mx.MX_OK
    which = np.repeat(np.arange(e), counts)
    for i, c in enumerate(which):
        rows = rng.integers(0, n, 64)
        q = w[c][on_gpu(rows)].cpu().numpy()
        plain = s[c].view(n // 128, k // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(n, k // 32)
        wv = ox.decode_fp4(q, plain[on_gpu(rows)].cpu().numpy())
        ref, size = wv @ av[i], np.abs(wv) @ np.abs(av[i])
        assert (np.abs(out[i, rows] - ref) <= 2.0**-8 * np.abs(ref) + k * 2.0**-22 * size).all()


def test_combine_past_32_bit_offsets(mx):
    r, n = 300_000, 8192
    y = torch.zeros((r, n), dtype=torch.bfloat16, device=dev())
    slots = torch.tensor([[r - 1, 0], [r - 2, 262_144]], dtype=torch.int32, device=dev())
    y[slots.long().reshape(-1)] = torch.arange(1, 5, device=dev()).bfloat16()[:, None].expand(4, n)
    out = mx.mx_combine(handle(), y, slots, torch.ones((2, 2), device=dev()))
    assert out[0].eq(3).all() and out[1].eq(7).all()


def test_combine_slots_outside(mx):
    y = torch.ones((4, 64), dtype=torch.bfloat16, device=dev())
    slots = on_gpu(np.array([[0, 4], [-1, 3]], np.int32))
    w = on_gpu(np.array([[1, 10], [100, 2]], np.float32))
    out = mx.mx_combine(handle(), y, slots, w)
    assert mx.mx_device_status(handle()) == mx.MX_ERR_INVALID_ARG
    assert out[0].eq(1).all() and out[1].eq(2).all()


def test_c_entry_refusals(mx):
    h, lib = handle(), mx.load_library()
    z = torch.zeros(1 << 16, dtype=torch.uint8, device=dev())
    out = torch.full((1 << 16,), 0xA5, dtype=torch.uint8, device=dev())
    p, o = z.data_ptr(), out.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    bad, no = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED

    def route(t=2, e=8, k=2, ldl=8, ty=mx.MX_TYPE_F32, score=0, g=1, tg=1, x=p, w=o, off=o):
        return lib.mx_route(h.ptr, t, e, k, x, ldl, ty, None, score, g, tg, 1, 1.0, w, o, off, o, o, st)

    for kw in (dict(t=0), dict(e=0), dict(k=0), dict(k=9), dict(ldl=7), dict(ty=1), dict(score=2), dict(g=3), dict(g=0),
               dict(g=2, tg=3), dict(g=4, k=3), dict(x=None), dict(w=None), dict(x=p + 2), dict(off=o + 1)):
        assert route(**kw) == bad, kw
    for kw in (dict(e=513, ldl=513), dict(e=64, ldl=64, k=33), dict(e=66, ldl=66, g=33, tg=33), dict(t=1 << 24)):
        assert route(**kw) == no, kw

    def grouped(e=2, r=4, n=128, k=128, a=p, rows=4, w=p, off=p, tok=p, out=o):
        return lib.mx_gemm_fp4_grouped(h.ptr, e, r, n, k, a, rows, p, 0, w, p, off, tok, 0, out, st)

    for kw in (dict(e=0), dict(r=0), dict(rows=0), dict(k=100), dict(a=None), dict(off=None), dict(tok=None, rows=3),
               dict(a=p + 8), dict(w=p + 16), dict(out=o + 8), dict(off=p + 2), dict(tok=p + 1)):
        assert grouped(**kw) == bad, kw
    for kw in (dict(n=64), dict(k=160), dict(e=513), dict(r=(1 << 24) + 1), dict(e=512, n=1 << 22),
               dict(e=1, r=1 << 24, n=1 << 18, rows=1 << 24)):
        assert grouped(**kw) == no, kw

    def combine(t=2, k=2, n=64, y=p, r=4, ldy=64, s=p, w=p, res=None, out=o):
        return lib.mx_combine(h.ptr, t, k, n, y, r, ldy, s, w, res, out, st)

    for kw in (dict(t=0), dict(k=0), dict(n=0), dict(n=60), dict(r=0), dict(ldy=32), dict(ldy=68), dict(y=None),
               dict(s=None), dict(w=None), dict(y=p + 8), dict(res=p + 8), dict(out=o + 8)):
        assert combine(**kw) == bad, kw
    for kw in (dict(k=33), dict(t=(1 << 24) + 1), dict(n=(1 << 20) + 8, ldy=(1 << 20) + 8)):
        assert combine(**kw) == no, kw
    torch.cuda.synchronize()
    assert (out == 0xA5).all()
