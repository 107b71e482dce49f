"""Outputs that a call on a given stream allocates: their memory must not be what work on the
current stream still writes, although the tensor that held it is gone."""
import pytest
import torch

from gpu_helpers import dev, handle
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu

T, N, K, E = 64, 1024, 512, 8


def calls(mx):  # noqa: F811
    """name -> (sizes of the outputs, call)"""
    h = handle()
    g = torch.Generator(device=dev()).manual_seed(5)
    normal = lambda *s: torch.randn(*s, generator=g, device=dev())  # noqa: E731
    x, w = normal(T, K).bfloat16(), normal(N, K)
    a8, s8 = mx.mx_quantize_rows(h, x)
    w8, ws8 = mx.mx_quantize_rows(h, w.bfloat16())
    w4, ws4, _ = mx.mx_quantize_rows_fp4(h, w)
    a4, s4, _ = mx.mx_quantize_rows_fp4(h, x, swizzled=False)
    we, wse, _ = mx.mx_quantize_rows_fp4(h, normal(E * N, K))
    logits = normal(T, E)
    r = mx.mx_route(h, logits, 1)
    y = normal(T, N).bfloat16()
    return {
        "quantize": lambda **kw: mx.mx_quantize_rows(h, x, **kw),
        "quantize fp4": lambda **kw: mx.mx_quantize_rows_fp4(h, x, y=True, **kw),
        "gemm": lambda **kw: [mx.mx_gemm(h, a8, s8, w8, ws8, **kw)],
        "gemm bf16": lambda **kw: [mx.mx_gemm_bf16(h, x[:4], w8, ws8, **kw)],
        "gemm fp4": lambda **kw: [mx.mx_gemm_fp4(h, a8, s8, w4, ws4, **kw)],
        "grouped": lambda **kw: [mx.mx_gemm_fp4_grouped(h, a4, s4, we.view(E, N, K // 2), wse.view(E, -1), r["offsets"],
                                                        tokens=r["tokens"], **kw)],
        "route": lambda **kw: [t for _, t in sorted(mx.mx_route(h, logits, 1, **kw).items())],
        "combine": lambda **kw: [mx.mx_combine(h, y, r["slots"], r["weights"], **kw)],
    }


@pytest.mark.parametrize("name", ["quantize", "quantize fp4", "gemm", "gemm bf16", "gemm fp4", "grouped", "route", "combine"])
def test_outputs_are_not_in_use_on_the_current_stream(mx, name):  # noqa: F811
    call = calls(mx)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call()]
    sizes = [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    # buffers of the outputs' sizes, written late on the current stream and free for it at once
    held = [torch.empty(n, dtype=torch.uint8, device=dev()) for n in sizes for _ in range(4)]
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for t in held:
        t.fill_(0xFF)
    del held, t
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
