"""examples/expert_layer.py call by call: every call's outputs against the float64 oracle on the very
inputs that it got, with each operator's own bounds (those of test_gpu_fp4 and test_gpu_experts)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import dev, handle
from oracle import experts as ox
from test_gpu_expert_layer import example, f64  # noqa: F401

pytestmark = pytest.mark.gpu


class Recorder:
    """The binding as the example sees it, keeping (name, arguments, options, outputs) of each call."""

    def __init__(self, mod):
        self.mod, self.calls = mod, []

    def __getattr__(self, name):
        f = getattr(self.mod, name)

        def call(h, *args, **kw):
            out = f(h, *args, **kw)
            self.calls.append((name, args, kw, out))
            return out
        return call


def plain(s, n, k):
    """[n, k / 32] scales of swizzled ones (n % 128 == 0, k % 128 == 0)."""
    return s.cpu().numpy().reshape(n // 128, k // 128, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(n, k // 32)


def grouped(a, s, w, w_scales, offsets, tokens=None, gated=False):
    """(reference, bound) of a grouped product."""
    e, n, k = w.shape[0], w.shape[1], 2 * w.shape[2]
    q, s, off = a.view(torch.uint8).cpu().numpy(), s.cpu().numpy().reshape(a.shape[0], -1), offsets.cpu().numpy()
    x = ox.decode_fp4(q, s) if a.shape[1] == k // 2 else ox.decode_fp8(q, s)
    x = x if tokens is None else x[tokens.cpu().numpy()]
    y, err = np.zeros((len(x), n)), np.zeros((len(x), n))
    for i in range(e):
        wv, rows = ox.decode_fp4(w[i].cpu().numpy(), plain(w_scales[i], n, k)), slice(off[i], off[i + 1])
        y[rows], err[rows] = x[rows] @ wv.T, k * 2.0**-22 * (np.abs(x[rows]) @ np.abs(wv).T)
    if not gated:
        return y, err
    g, u, eg, eu = y[:, 0::2], y[:, 1::2], err[:, 0::2], err[:, 1::2]
    ref = ox.silu_gate(y)
    sg = np.abs(g / (1 + np.exp(-g)))
    return ref, 1.1 * eg * np.abs(u) + (sg + 1.1 * eg) * eu + (6 + 1.2 * np.abs(g)) * 2.0**-22 * np.abs(ref)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t", [1, 9, 70, 400])
def test_every_call_of_the_layer(example, monkeypatch, t, fp4):  # noqa: F811
    e, hidden, inner, k = 16, 256, 128, 3
    rec = Recorder(example.mx)
    monkeypatch.setattr(example, "mx", rec)
    layer = example.random_layer(handle(), e, hidden, inner, k, seed=t, fp4_activations=fp4)
    rec.calls.clear()
    x = torch.randn(t, hidden, generator=torch.Generator(device="cuda").manual_seed(t), device=dev()).bfloat16()
    layer(x, residual=x)
    torch.cuda.synchronize()
    quantizer = "mx_quantize_rows_fp4" if fp4 else "mx_quantize_rows"
    names = [c[0] for c in rec.calls]
    assert names == ["mx_route", quantizer, "mx_gemm_fp4_grouped", quantizer, "mx_gemm_fp4_grouped", "mx_combine"]
    for name, args, kw, out in rec.calls:
        if name == "mx_route":
            lg = f64(args[0])
            w, chosen = ox.route(lg, args[1], bias=f64(kw["bias"]), **{a: b for a, b in kw.items() if a != "bias"})
            assert np.array_equal(out["experts"].cpu().numpy(), chosen)
            offsets, tokens, slots = ox.row_order(chosen, e)
            assert np.array_equal(out["offsets"].cpu().numpy(), offsets)
            assert np.array_equal(out["tokens"].cpu().numpy(), tokens)
            assert np.array_equal(out["slots"].cpu().numpy(), slots)
            assert (np.abs(f64(out["weights"]) - w) <= 40 * 2.0**-23 * np.abs(w)).all()  # sigmoid scores
        elif name == quantizer:
            q, s = ox.quantize_fp4(f64(args[0]))[:2] if fp4 else oracle.mx_quantize(f64(args[0]))
            assert np.array_equal(out[0].view(torch.uint8).cpu().numpy(), q)
            assert np.array_equal(out[1].cpu().numpy().reshape(s.shape), s)
        elif name == "mx_gemm_fp4_grouped":
            ref, tol = grouped(*args, **kw)
            tol = tol + 2.0**-8 * (np.abs(ref) + tol) + 1e-37
            d = np.abs(f64(out) - ref)
            assert (d <= tol).all(), (d / tol).max()
        else:
            y, slots, w = f64(args[0]), args[1].cpu().numpy(), f64(args[2])
            ref = ox.combine(y, slots, w, f64(kw["residual"]))
            size = ox.combine(np.abs(y), slots, w, np.abs(f64(kw["residual"])))
            assert (np.abs(f64(out) - ref) <= 2.0**-8 * np.abs(ref) + (k + 2) * 2.0**-23 * size).all()


@pytest.mark.parametrize("fp4", [False, True])
def test_more_rows_than_one_quantizer_call_takes(example, fp4):  # noqa: F811
    """22100 tokens to three experts each: 66300 rows of products, as the same tokens in two calls."""
    layer = example.random_layer(handle(), 8, 128, 128, 3, fp4_activations=fp4)
    x = torch.randn(22100, 128, generator=torch.Generator(device="cuda").manual_seed(1), device=dev()).bfloat16()
    whole, parts = layer(x, residual=x), [layer(p, residual=p) for p in (x[:9000], x[9000:])]
    assert example.mx.mx_device_status(handle()) == example.mx.MX_OK
    assert torch.equal(whole, torch.cat(parts))
