"""An expert layer with MXFP4 weights, from router logits to the residual stream.

    route     mx_route: experts and weights of each token, rows in expert order
    quantize  mx_quantize_rows (MXFP8) or mx_quantize_rows_fp4 (MXFP4) of the tokens
    up        mx_gemm_fp4_grouped, gated: silu(gate) * up of the rows of every expert
    quantize  the same for the products
    down      mx_gemm_fp4_grouped
    sum       mx_combine: each token's rows by their weights, plus the residual

The weights are laid out once: gate row i and up row i are rows 2i and 2i + 1. After a
first step every step reuses its buffers, so it also runs as a CUDA graph.

    python examples/expert_layer.py --tokens 64
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import mxfp8_block_scaled_06_gb300 as mx

MOST_ROWS = 65536  # of one mx_quantize_rows call


class ExpertLayer:
    """gate, up: [E, I, H]; down: [E, H, I] (bf16, fp16 or fp32 on the GPU); H % 128 == 0, I % 128 == 0."""

    def __init__(self, handle, router, gate, up, down, top_k, bias=None, scoring="sigmoid", n_groups=1,
                 topk_groups=1, scale=1.0, fp4_activations=False):
        self.h, self.router, self.bias = handle, router, bias
        self.top_k, self.kw = top_k, dict(scoring=scoring, n_groups=n_groups, topk_groups=topk_groups, scale=scale)
        self.quantize_rows = mx.mx_quantize_rows_fp4 if fp4_activations else mx.mx_quantize_rows
        e, i, hidden = gate.shape
        self.w13, self.s13 = self._weights(torch.stack([gate, up], 2).reshape(e, 2 * i, hidden))
        self.w2, self.s2 = self._weights(down)

    def _weights(self, w):
        e, n, k = w.shape
        q, s, _ = mx.mx_quantize_rows_fp4(self.h, w.reshape(e * n, k))
        return q.view(e, n, k // 2), s.view(e, -1)

    def _quantize(self, x):
        rows, k = x.shape
        if rows <= MOST_ROWS or self.quantize_rows is mx.mx_quantize_rows_fp4:
            return self.quantize_rows(self.h, x, swizzled=False)[:2]
        q, s = (torch.empty((rows, c), dtype=torch.uint8, device=x.device) for c in (k, k // 32))
        for i in range(0, rows, MOST_ROWS):
            part = slice(i, i + MOST_ROWS)
            self.quantize_rows(self.h, x[part], q=q[part], scales=s[part], swizzled=False)
        return q, s

    def __call__(self, x, residual=None):
        """x [T, H] bf16 -> residual + the experts' weighted sum, bf16."""
        logits = x.float() @ self.router.T
        r = mx.mx_route(self.h, logits, self.top_k, bias=self.bias, **self.kw)
        a, s = self._quantize(x)
        y = mx.mx_gemm_fp4_grouped(self.h, a, s, self.w13, self.s13, r["offsets"], tokens=r["tokens"], gated=True)
        a, s = self._quantize(y)
        y = mx.mx_gemm_fp4_grouped(self.h, a, s, self.w2, self.s2, r["offsets"])
        return mx.mx_combine(self.h, y, r["slots"], r["weights"], residual=residual)


def random_layer(handle, experts=32, hidden=1024, inner=512, top_k=4, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return ExpertLayer(handle, 0.05 * normal(experts, hidden), *(0.05 * normal(experts, inner, hidden) for _ in range(2)),
                       0.05 * normal(experts, hidden, inner), top_k, bias=0.05 * normal(experts), n_groups=4,
                       topk_groups=2, **kw)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--fp4-activations", action="store_true")
    a = ap.parse_args()
    torch.cuda.set_device(0)
    h = mx.mx_create(0)
    layer = random_layer(h, a.experts, a.hidden, a.inner, a.top_k, fp4_activations=a.fp4_activations)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    eager = layer(x, residual=x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, residual=x)
    graph.replay()
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if mx.mx_device_status(h) != mx.MX_OK or not torch.equal(out, eager):
        raise SystemExit("the graph's result differs from the eager one")
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, top {a.top_k}: "
          f"{begin.elapsed_time(end) * 10:.1f} us a step")


if __name__ == "__main__":
    main()
