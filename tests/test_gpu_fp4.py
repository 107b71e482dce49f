"""MXFP4 quantization and products against the float64 oracle.

Products: the float32 sum of K products is off by at most about K 2^-22 sum |a w|
(each addition rounds or truncates once, to 2^-23 of a partial sum of that size),
and the bf16 result rounds by 2^-8 of its value."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import bf16_to_device, dev, handle
from oracle import experts as ox

pytestmark = pytest.mark.gpu

PATTERN = 0xA5


@pytest.fixture(scope="module")
def mx():
    handle()
    import mxfp8_block_scaled_06_gb300 as mod

    return mod


def guarded(nbytes):
    """A buffer with 4 KB of a known pattern on either side."""
    buf = torch.full((nbytes + 8192,), PATTERN, dtype=torch.uint8, device=dev())
    return buf, buf[4096:4096 + nbytes]


def intact(buf, nbytes):
    host = buf.cpu().numpy()
    return (host[:4096] == PATTERN).all() and (host[4096 + nbytes:] == PATTERN).all()


def same_floats(a, b):
    """Equal, NaN where NaN, and elsewhere of the same sign of zero."""
    ok = ~np.isnan(b)
    return np.array_equal(a, b, equal_nan=True) and np.array_equal(np.signbit(a)[ok], np.signbit(b)[ok])


def values(rng, m, k, spread=6):
    x = rng.standard_normal((m, k // 32, 32)) * np.exp2(rng.integers(-spread, spread + 1, (m, k // 32, 1)).astype(float))
    return x.reshape(m, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,k,pad", [(1, 32, 0), (1, 5120, 0), (3, 96, 8), (130, 160, 0), (257, 2080, 520), (64, 128, 0)])
def test_quantize(mx, m, k, pad, dtype):
    rng = np.random.default_rng(m * k)
    x = torch.from_numpy(values(rng, m, k)).to(dtype)
    x = torch.nn.functional.pad(x, (0, pad), value=100.0).to(dev())[:, :k]
    q0, s0, v0 = ox.quantize_fp4(x.cpu().double().numpy())
    qb, q = guarded(m * k // 2)
    n = mx.mx_scale_bytes(m, k)
    sb, s = guarded(n)
    mx.mx_quantize_rows_fp4(handle(), x, q=q.view(m, k // 2), scales=s)
    assert np.array_equal(q.cpu().numpy().reshape(m, -1), q0)
    assert np.array_equal(s.cpu().numpy(), oracle.swizzle_scales(s0))
    assert intact(qb, m * k // 2) and intact(sb, n)
    q, s, y = mx.mx_quantize_rows_fp4(handle(), x, swizzled=False, y=True)
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)
    assert same_floats(y.float().cpu().numpy().astype(np.float64), v0)


def test_quantize_every_bf16(mx):
    """Every bf16 pattern, Inf and NaN among them, as the first value of a block of zeros."""
    bits = np.zeros((2048, 1024), np.uint16)
    bits[:, ::32] = np.arange(65536, dtype=np.uint16).reshape(2048, 32)
    x = bf16_to_device(bits)
    q0, s0, v0 = ox.quantize_fp4(x.cpu().double().numpy())
    q, s, y = mx.mx_quantize_rows_fp4(handle(), x, swizzled=False, y=True)
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)
    assert same_floats(y.float().cpu().numpy().astype(np.float64), v0)


def test_quantize_every_code_at_every_scale(mx):
    """All E2M1 values and the ties between them under block maxima of every exponent."""
    grid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    block = np.concatenate([grid, -grid])
    x = torch.from_numpy(block[None] * np.exp2(np.arange(-133.0, 126))[:, None]).float().to(dev())
    q0, s0, v0 = ox.quantize_fp4(x.cpu().double().numpy())
    q, s, y = mx.mx_quantize_rows_fp4(handle(), x, swizzled=False, y=True)
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)
    assert same_floats(y.float().cpu().numpy().astype(np.float64), v0)


def operand(rng, rows, k, fp4, spread=4):
    """(codes, plain scale bytes, values) of an operand."""
    x = values(rng, rows, k, spread).astype(np.float32).astype(np.float64)
    if fp4:
        return ox.quantize_fp4(x)
    q, s = oracle.mx_quantize(x)
    return q, s, ox.decode_fp8(q, s)


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev())


def bound(a, w, ref):
    size = np.abs(a) @ np.abs(w).T
    return 2.0**-8 * np.abs(ref) + a.shape[1] * 2.0**-22 * size + 1e-37


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 128, 128), (1, 2048, 5120), (3, 256, 384), (8, 8192, 1536), (16, 128, 4096),
                                   (17, 384, 640), (33, 128, 128), (129, 256, 896), (201, 640, 1024), (256, 128, 256),
                                   (257, 256, 512), (300, 128, 1152), (449, 384, 2176), (1000, 1280, 384),
                                   (230, 512, 128), (700, 256, 256), (90, 16384, 128), (40, 16384, 384)])
def test_product(mx, m, n, k, fp4):
    rng = np.random.default_rng(m + n + k)
    aq, as_, av = operand(rng, m, k, fp4)
    wq, ws, wv = operand(rng, n, k, True)
    ob, o = guarded(m * n * 2)
    out = o.view(torch.bfloat16).view(m, n)
    mx.mx_gemm_fp4(handle(), on_gpu(aq), on_gpu(oracle.swizzle_scales(as_)), on_gpu(wq),
                   on_gpu(oracle.swizzle_scales(ws)), out=out)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    ref = av @ wv.T
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(av, wv, ref)).all(), (err / bound(av, wv, ref)).max()
    assert intact(ob, m * n * 2)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("m,n,k", [(2230, 384, 1152), (4300, 128, 2048), (3360, 640, 1536), (8400, 384, 640)])
def test_product_of_the_widest_tiles(mx, m, n, k, fp4):
    """Tiles of 200 rows and more with one CTA to an SM: the shortest rings, over many stages."""
    test_product(mx, m, n, k, fp4)


@pytest.mark.parametrize("m,n,k,fp4", [(26500, 512, 640, False), (30011, 384, 1152, True), (33000, 384, 512, False)])
def test_product_of_more_rows_than_a_band(mx, m, n, k, fp4):
    """Activations of over 16 MB go over the weights in bands of rows."""
    test_product(mx, m, n, k, fp4)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1024, 2688), (1, 8192, 3840), (7, 256, 6016), (16, 128, 4096), (17, 6144, 2560),
                                   (64, 640, 3968), (128, 384, 5760), (129, 128, 5248), (201, 3840, 4096),
                                   (255, 512, 3200), (344, 256, 4224), (513, 128, 8064), (1300, 128, 4736)])
def test_product_split_along_k(mx, m, n, k, pdl, fp4):
    """Clusters along K: of 2 to 8, several row slices, two to an SM, behind an earlier kernel or not."""
    rng = np.random.default_rng(m + n + k)
    aq, as_, av = operand(rng, m, k, fp4)
    wq, ws, wv = operand(rng, n, k, True)
    ob, o = guarded(m * n * 2)
    out = o.view(torch.bfloat16).view(m, n)
    args = [on_gpu(aq), on_gpu(oracle.swizzle_scales(as_)), on_gpu(wq), on_gpu(oracle.swizzle_scales(ws))]
    torch.cuda.synchronize()
    for _ in range(2):
        mx.mx_gemm_fp4(handle(), *args, out=out, pdl=pdl)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    ref = av @ wv.T
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(av, wv, ref)).all(), (err / bound(av, wv, ref)).max()
    assert intact(ob, m * n * 2)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("m", [2, 40, 500])
def test_product_of_exact_values(mx, m, fp4):
    """E2M1 values under scales of one: every sum is exact in float32."""
    rng = np.random.default_rng(m)
    n, k = 256, 768
    aq = rng.integers(0, 16, (m, k)).astype(np.uint8)
    wq = rng.integers(0, 16, (n, k)).astype(np.uint8)
    av, wv = ox.e2m1_decode(aq), ox.e2m1_decode(wq)
    a = ox.pack(aq) if fp4 else oracle.e4m3_encode(av)
    ones = lambda r: np.full((r, k // 32), 127, np.uint8)  # noqa: E731
    out = mx.mx_gemm_fp4(handle(), on_gpu(a), on_gpu(oracle.swizzle_scales(ones(m))), on_gpu(ox.pack(wq)),
                         on_gpu(oracle.swizzle_scales(ones(n))))
    want = torch.from_numpy(av @ wv.T).float().bfloat16()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("m", [5, 700])
def test_product_twice_and_in_a_graph(mx, m):
    """The same bits from a repeated call, another stream and a replayed graph."""
    rng = np.random.default_rng(2)
    aq, as_, _ = operand(rng, m, 640, True)
    wq, ws, _ = operand(rng, 512, 640, True)
    args = [on_gpu(aq), on_gpu(oracle.swizzle_scales(as_)), on_gpu(wq), on_gpu(oracle.swizzle_scales(ws))]
    first = mx.mx_gemm_fp4(handle(), *args)
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = mx.mx_gemm_fp4(handle(), *args)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.mx_gemm_fp4(handle(), *args, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, out)


@pytest.mark.parametrize("m", [6, 300])
def test_nan_scale_reaches_its_row_only(mx, m):
    rng = np.random.default_rng(4)
    n, k = 128, 512
    aq, as_, _ = operand(rng, m, k, True)
    wq, ws, _ = operand(rng, n, k, True)
    as_[2, 3] = 255
    ws[77, 9] = 255
    out = mx.mx_gemm_fp4(handle(), on_gpu(aq), on_gpu(oracle.swizzle_scales(as_)), on_gpu(wq),
                         on_gpu(oracle.swizzle_scales(ws))).float().cpu().numpy()
    bad = np.zeros((m, n), bool)
    bad[2] = True
    bad[:, 77] = True
    assert np.array_equal(np.isnan(out), bad)


def test_c_entry_refusals(mx):
    """The library's own checks: an error before anything is launched."""
    h, lib = handle(), mx.load_library()
    z = torch.zeros(1 << 16, dtype=torch.uint8, device=dev())
    out = torch.full((1 << 16,), PATTERN, dtype=torch.uint8, device=dev())
    p, o = z.data_ptr(), out.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    bad, no = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED
    q = lambda *a: lib.mx_quantize_rows_fp4(h.ptr, *a, st)  # noqa: E731
    assert q(0, 32, p, 32, 0, o, o, 1, None) == bad
    assert q(1, 48, p, 48, 0, o, o, 1, None) == bad
    assert q(1, 64, p, 32, 0, o, o, 1, None) == bad
    assert q(1, 64, p, 68, 0, o, o, 1, None) == bad
    assert q(1, 64, p, 64, 3, o, o, 1, None) == bad
    assert q(1, 64, p + 2, 64, 0, o, o, 1, None) == bad
    assert q(1, 64, p, 64, 0, o, o + 1, 1, None) == bad
    assert q(1, 64, p, 64, 0, o, o, 1, o + 2) == bad
    assert q(1 << 24, 1024, p, 1024, 0, o, o, 1, None) == no
    g = lambda m, n, k, a=p, w=p, r=o, f=0: lib.mx_gemm_fp4(h.ptr, m, n, k, a, p, 1, w, p, r, f, st)  # noqa: E731
    assert g(0, 128, 128) == bad and g(1, 128, 100) == bad and g(1, 128, 128, f=2) == bad
    assert g(1, 128, 128, a=p + 8) == bad and g(1, 128, 128, w=p + 16) == bad and g(1, 128, 128, r=None) == bad
    assert g(1, 100, 128) == no and g(1, 128, 96) == no and g((1 << 24) + 1, 128, 128) == no
    torch.cuda.synchronize()
    assert (out == PATTERN).all()
