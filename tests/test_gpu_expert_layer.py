"""examples/expert_layer.py against the float64 oracle, operator by operator: each call's
inputs are the layer's own, so a rounding of one does not count against the next."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import dev, handle
from oracle import experts as ox

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    handle()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t", [1, 9, 70])
def test_layer(example, t, fp4):
    e, hidden, inner, k = 16, 256, 128, 3
    layer = example.random_layer(handle(), e, hidden, inner, k, seed=t, fp4_activations=fp4)
    x = torch.randn(t, hidden, generator=torch.Generator(device="cuda").manual_seed(t), device=dev()).bfloat16()
    out = f64(layer(x, residual=x))

    # the layer in float64 from its quantized weights, with its own two roundings to
    # MX activations and bf16 products
    def quantized(v):
        q, s = (ox.quantize_fp4(v)[:2] if fp4 else oracle.mx_quantize(v))
        return ox.decode_fp4(q, s) if fp4 else ox.decode_fp8(q, s)

    def weights(q, s, n, kk):
        """[E, n, kk] values; the swizzled scales are undone by their index table."""
        where = oracle.swizzle_scales(np.arange(n * (kk // 32)).reshape(n, -1) % 251)
        q, s = q.cpu().numpy(), s.cpu().numpy()
        flat = [s[i].reshape(n // 128, kk // 128, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(n, kk // 32) for i in range(e)]
        again = where.reshape(n // 128, kk // 128, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(n, kk // 32)
        assert (again == np.arange(n * (kk // 32)).reshape(n, -1) % 251).all()
        return np.stack([ox.decode_fp4(q[i], flat[i]) for i in range(e)])

    w13, w2 = weights(layer.w13, layer.s13, 2 * inner, hidden), weights(layer.w2, layer.s2, hidden, inner)
    bf16 = lambda v: f64(torch.from_numpy(v).float().bfloat16())  # noqa: E731
    logits = f64(x.float() @ layer.router.T)
    gates, chosen = ox.route(logits, k, bias=f64(layer.bias), **layer.kw)
    xq = quantized(f64(x))
    ref, size = f64(x), np.abs(f64(x))
    for i in range(t):
        for j in range(k):
            c = chosen[i, j]
            y = bf16(ox.silu_gate((w13[c] @ xq[i])[None]))
            z = w2[c] @ quantized(y)[0]
            ref[i] += gates[i, j] * z
            size[i] += gates[i, j] * (np.abs(w2[c]) @ np.abs(quantized(y)[0]))
    # a product at a rounding border may take the other code: a step of the code (at most
    # 2^-1 of a 4-bit value, 2^-3 of an 8-bit one) in a few of the inner products' terms;
    # everything else is below the final bf16 rounding of the products and of the sum
    tol = 2.0**-7 * np.abs(ref) + size * (2.0**-6 if fp4 else 2.0**-7)
    assert (np.abs(out - ref) <= tol).all(), (np.abs(out - ref) / tol).max()


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["expert_layer.py", "--tokens", "20", "--experts", "8"])
    example.main()
    assert "us a step" in capsys.readouterr().out
