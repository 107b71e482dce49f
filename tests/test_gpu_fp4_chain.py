"""Many expert-layer calls in a row on the same buffers, each kernel starting while the ones before
it end, against the same calls with a synchronization after each: the same bits."""
import pytest
import torch

from gpu_helpers import handle
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda:0")


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t", [1, 40, 700])
def test_chain_on_reused_buffers(mx, t, fp4):  # noqa: F811
    """Router outputs, codes and scales are written again in every step and read by the next kernels:
    products of narrow and wide tiles, gathered or not, K split under PDL, with whole K under PDL."""
    h, e, hidden, inner, k, steps = handle(), 8, 512, 256, 2, 12
    g = torch.Generator(device="cuda:0").manual_seed(t)
    weights = []
    for n, kk in ((2 * inner, hidden), (hidden, inner)):
        q, s, _ = mx.mx_quantize_rows_fp4(h, normal(g, e * n, kk))
        weights.append((q.view(e, n, kk // 2), s.view(e, -1)))
    dense = [mx.mx_quantize_rows_fp4(h, normal(g, n, hidden))[:2] for n in (hidden, 16384)]
    x = normal(g, steps, t, hidden).bfloat16()
    logits = normal(g, steps, t, e)
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda:0")  # noqa: E731
    quantize = mx.mx_quantize_rows_fp4 if fp4 else mx.mx_quantize_rows
    width = lambda n: n // 2 if fp4 else n  # noqa: E731
    r = dict(weights=z(t, k, dtype=torch.float32), experts=z(t, k, dtype=torch.int32), offsets=z(e + 1, dtype=torch.int32),
             tokens=z(t * k, dtype=torch.int32), slots=z(t, k, dtype=torch.int32))
    b = [(z(t, width(hidden)), z(t, hidden // 32)), (z(t * k, width(inner)), z(t * k, inner // 32)),
         (z(t, width(hidden)), z(mx.mx_scale_bytes(t, hidden)))]
    up, down = z(t * k, inner, dtype=torch.bfloat16), z(t * k, hidden, dtype=torch.bfloat16)
    mixed = z(t, hidden, dtype=torch.bfloat16)
    outs = [[z(steps, t, n, dtype=torch.bfloat16) for n in (hidden, 16384)] for _ in range(2)]

    def quantized(src, dst, swizzled):
        quantize(h, src, q=dst[0], scales=dst[1] if swizzled else dst[1].reshape(-1), swizzled=swizzled)

    def run(out, after):
        for i in range(steps):
            calls = [lambda: mx.mx_route(h, logits[i], k, **r),
                     lambda: quantized(x[i], b[0], False),
                     lambda: mx.mx_gemm_fp4_grouped(h, *b[0], *weights[0], r["offsets"], tokens=r["tokens"], gated=True, out=up),
                     lambda: quantized(up, b[1], False),
                     lambda: mx.mx_gemm_fp4_grouped(h, *b[1], *weights[1], r["offsets"], out=down),
                     lambda: mx.mx_combine(h, down, r["slots"], r["weights"], residual=x[i], out=mixed),
                     lambda: quantized(mixed, b[2], True),
                     lambda: mx.mx_gemm_fp4(h, *b[2], *dense[0], out=out[0][i], pdl=True),
                     lambda: mx.mx_gemm_fp4(h, *b[2], *dense[1], out=out[1][i], pdl=True)]
            for call in calls:
                call()
                after()

    run(outs[0], torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[1], lambda: None)
    for _ in range(3):
        for o in outs[1]:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(*outs))
    assert mx.mx_device_status(h) == mx.MX_OK


@pytest.mark.parametrize("m,n,k", [(8, 16384, 4096), (100, 16384, 2048)])
def test_weights_made_on_the_stream(mx, m, n, k):  # noqa: F811
    """New weights for every product under PDL: safe behind an ordinary kernel, which starts when
    all before it has ended."""
    h = handle()
    g = torch.Generator(device="cuda:0").manual_seed(n)
    x, w = normal(g, m, k), [normal(g, n, k).bfloat16() for _ in range(3)]
    q, s, _ = mx.mx_quantize_rows_fp4(h, w[0])
    want = []
    for v in w:
        mx.mx_quantize_rows_fp4(h, v, q=q, scales=s)
        a, a_s, _ = mx.mx_quantize_rows_fp4(h, x)
        torch.cuda.synchronize()
        want.append(mx.mx_gemm_fp4(h, a, a_s, q, s))
    got = [torch.zeros_like(o) for o in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for v, out in zip(w, got):
            mx.mx_quantize_rows_fp4(h, v, q=q, scales=s)
            out.fill_(7.0)  # the ordinary kernel
            mx.mx_quantize_rows_fp4(h, x, q=a, scales=a_s)
            mx.mx_gemm_fp4(h, a, a_s, q, s, out=out, pdl=True)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, e) for o, e in zip(got, want))
    assert mx.mx_device_status(h) == mx.MX_OK
