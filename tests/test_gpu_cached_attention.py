"""The rotary, cache and attention calls as a decode layer runs them (examples/cached_attention.py): prompts, then
single tokens, each step against the oracle on the step's own inputs; and the example itself."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gpu_helpers import dev, handle
from oracle import attention as oa
from oracle import experts as oe
from test_gpu_experts import mx  # noqa: F401

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_prompts_and_steps(mx):  # noqa: F811
    from cached_attention import D, D_ROPE, HEADS, CachedAttention, place

    h, page, hidden = handle(), 16, 256
    layer = CachedAttention(h, hidden, pages=24, page_size=page, max_pos=512)
    table = torch.randperm(24, device=dev()).int().view(3, 8)
    cos_sin = layer.cos_sin.cpu().numpy()
    held = [np.zeros((0, D)) for _ in range(3)]
    for counts in ([70, 1, 40], [1, 1, 1], [1, 5, 2], [1, 1, 1]):
        seq = np.repeat(np.arange(3), counts)
        pos = np.concatenate([len(held[b]) + np.arange(n) for b, n in enumerate(counts)])
        at = lambda v, t=torch.int64: torch.tensor(np.asarray(v), dtype=t, device=dev())  # noqa: E731
        lengths = [len(x) + n for x, n in zip(held, counts)]
        offsets = np.concatenate([[0], np.cumsum(counts)])
        parts = {}
        x = torch.randn(len(pos), hidden, device=dev()).bfloat16()
        y = layer(x, at(pos), place(table, page, at(seq), at(pos)), table, at(lengths, torch.int32),
                  at(offsets, torch.int32) if max(counts) > 1 else None, parts)
        assert y.shape == (len(pos), hidden) and torch.isfinite(y).all()
        latent = parts["latent"].double().cpu().numpy()[:, 0]
        values = oe.quantize_fp4(latent)[2]
        q = parts["q"].double().cpu().numpy()
        out = parts["out"].double().cpu().numpy()
        for b in range(3):
            rows = slice(offsets[b], offsets[b + 1])
            held[b] = np.concatenate([held[b], values[rows]])
            for j in range(HEADS):
                want, _, size, reach = oa.attend(q[rows, j], held[b], held[b], D ** -0.5, pos[rows])
                # as for mx_attend alone: the output's half step, weights of 11 bits, float32 scores
                e = (D + 8) * 2.0**-23 * reach[:, None]
                tol = 2.0**-8 * np.abs(want) + size * (2.0**-11 + 2 * e + 2.0**-20) * 1.01 + len(held[b]) * 2.0**-33 * size.max()
                assert (np.abs(out[rows, j] - want) <= tol).all()
        # the rotations of the queries: their 64-bit inverse turns the lengths of no pair
        part = q[..., D - D_ROPE:]
        back = oa.rope(q, cos_sin[pos].astype(np.float64), D - D_ROPE, True, True)[..., D - D_ROPE:]
        assert np.allclose((part ** 2).sum(-1), (back ** 2).sum(-1), rtol=1e-5)
    assert mx.mx_device_status(h) == mx.MX_OK


def test_example_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "cached_attention.py"), "--prompt", "150", "--steps", "5"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "us a step" in r.stdout, r.stdout + r.stderr
