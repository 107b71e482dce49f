"""The tensor checks of the MXFP4 and expert entry points, on the CPU: each case is right in
every respect but one; tensors that are right but in host memory fail the last check."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def mx():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp8_block_scaled_06_gb300 as mod

    mod.load_library()
    return mod


@pytest.fixture
def h(mx):
    return mx.Handle(0, 0)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def quantize(mx):
    return mx.mx_quantize_rows_fp4, dict(x=bf16(4, 512), q=u8(4, 256), scales=u8(mx.mx_scale_bytes(4, 512)))


def product(mx):
    return mx.mx_gemm_fp4, dict(a=u8(4, 512), a_scales=u8(mx.mx_scale_bytes(4, 512)), w=u8(256, 256),
                                w_scales=u8(mx.mx_scale_bytes(256, 512)), out=bf16(4, 256))


def grouped(mx):
    return mx.mx_gemm_fp4_grouped, dict(a=u8(4, 512), a_scales=u8(4, 16), w=u8(3, 256, 256),
                                        w_scales=u8(3, mx.mx_scale_bytes(256, 512)), offsets=i32(4), tokens=i32(9),
                                        out=bf16(9, 256))


def route(mx):
    return mx.mx_route, dict(logits=f32(5, 64), top_k=4, bias=f32(64), weights=f32(5, 4), experts=i32(5, 4),
                             offsets=i32(65), tokens=i32(20), slots=i32(5, 4))


def combine(mx):
    return mx.mx_combine, dict(y=bf16(9, 64), slots=i32(3, 2), weights=f32(3, 2), residual=bf16(3, 64),
                               out=bf16(3, 64))


CASES = [
    (quantize, dict(x=bf16(512)), ValueError), (quantize, dict(x=u8(4, 512)), TypeError),
    (quantize, dict(x=bf16(4, 500)), ValueError), (quantize, dict(x=bf16(512, 4).t()), ValueError),
    (quantize, dict(q=u8(4, 512)), ValueError), (quantize, dict(q=bf16(4, 256)), TypeError),
    (quantize, dict(scales=u8(100)), ValueError),
    (product, dict(a=u8(4, 128)), ValueError), (product, dict(a=bf16(4, 512)), TypeError),
    (product, dict(a_scales=u8(64)), ValueError), (product, dict(w=u8(256 * 256)), ValueError),
    (product, dict(w=u8(256, 512)[:, :256]), ValueError), (product, dict(w_scales=u8(9)), ValueError),
    (product, dict(out=bf16(3, 256)), ValueError), (product, dict(m=5), ValueError),
    (grouped, dict(w=u8(256, 256)), ValueError), (grouped, dict(w=u8(3, 200, 256)), ValueError),
    (grouped, dict(w_scales=u8(2, 4096)), ValueError), (grouped, dict(a=u8(4, 100)), ValueError),
    (grouped, dict(a_scales=u8(4, 15)), ValueError), (grouped, dict(offsets=i32(3)), ValueError),
    (grouped, dict(offsets=f32(4)), TypeError), (grouped, dict(tokens=i32(9).long()), TypeError),
    (grouped, dict(tokens=i32(18)[::2]), ValueError), (grouped, dict(out=bf16(9, 128)), ValueError),
    (grouped, dict(gated=True), ValueError),
    (route, dict(logits=f32(64)), ValueError), (route, dict(logits=f32(5, 64).half()), TypeError),
    (route, dict(logits=f32(64, 5).t()), ValueError), (route, dict(top_k=0), ValueError),
    (route, dict(scoring="linear"), ValueError), (route, dict(bias=f32(63)), ValueError),
    (route, dict(bias=bf16(64)), TypeError), (route, dict(slots=i32(5, 3)), ValueError),
    (route, dict(offsets=i32(64)), ValueError), (route, dict(weights=bf16(5, 4)), TypeError),
    (combine, dict(y=f32(9, 64)), TypeError), (combine, dict(y=bf16(64, 9).t()), ValueError),
    (combine, dict(slots=i32(6)), ValueError), (combine, dict(weights=f32(3, 3)), ValueError),
    (combine, dict(residual=bf16(3, 32)), ValueError), (combine, dict(out=bf16(2, 64)), ValueError),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_one_wrong_argument(mx, h, i):
    make, wrong, exc = CASES[i]
    call, args = make(mx)
    with pytest.raises(exc) as e:
        call(h, **{**args, **wrong})
    assert "cuda:0" not in str(e.value)  # refused for what is wrong, before residency


@pytest.mark.parametrize("make", [quantize, product, grouped, route, combine])
def test_host_tensors_fail_the_residency_check(mx, h, make):
    call, args = make(mx)
    with pytest.raises(ValueError, match="cuda:0"):
        call(h, **args)


def test_null_handle(mx):
    lib, n = mx.load_library(), None
    bad = mx.MX_ERR_INVALID_ARG
    assert lib.mx_quantize_rows_fp4(n, 1, 32, n, 32, 0, n, n, 1, n, n) == bad
    assert lib.mx_gemm_fp4(n, 1, 128, 128, n, n, 0, n, n, n, 0, n) == bad
    assert lib.mx_gemm_fp4_grouped(n, 1, 1, 128, 128, n, 1, n, 0, n, n, n, n, 0, n, n) == bad
    assert lib.mx_route(n, 1, 1, 1, n, 1, 2, n, 0, 1, 1, 1, ctypes.c_float(1), n, n, n, n, n, n) == bad
    assert lib.mx_combine(n, 1, 1, 8, n, 1, 8, n, n, n, n, n) == bad
