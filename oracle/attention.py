"""CPU oracle of the rotary, cache and attention operators, in numpy float64.

TEST INFRASTRUCTURE ONLY, as the package's main module. Written from the operators'
definitions; it shares no code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(d_rope, base=10000.0, scaling="none", factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each of the d_rope / 2 pairs."""
    out = []
    for i in range(d_rope // 2):
        f = base ** (-2.0 * i / d_rope)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            c = lambda turns: d_rope * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(c(beta_fast)), 0), min(math.ceil(c(beta_slow)), d_rope - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return np.array(out)


def rope_table(max_pos, d_rope, magnitude=1.0, **kw):
    angle = np.arange(max_pos)[:, None] * rope_frequencies(d_rope, **kw)[None, :]
    return np.concatenate([np.cos(angle), np.sin(angle)], 1) * magnitude


def rope(x, cos_sin, first, interleaved, inverse):
    """x [T, heads, d] turned by cos_sin [T, d_rope]; float32 arrays step by step in float32, float64 ones in 64."""
    n = cos_sin.shape[1]
    h = n // 2
    c, s = cos_sin[:, None, :h], cos_sin[:, None, h:]
    s = -s if inverse else s
    out = x.copy()
    at = [first + 2 * i for i in range(h)] if interleaved else [first + i for i in range(h)]
    to = [p + 1 for p in at] if interleaved else [p + h for p in at]
    a, b = x[..., at], x[..., to]
    out[..., at] = a * c - b * s
    out[..., to] = b * c + a * s
    return out


def attend(q, k, v, scale, pos, causal=True, window=0):
    """One sequence and kv head: q [rows, d] at positions pos [rows], k and v [n, d]. Returns out, the log of
    the sums, and what bounds the rounding: the sums of |weights v| and the largest sum of |q k| scale of a row."""
    out, lse = np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf)
    size, reach = np.zeros_like(out), np.zeros(len(q))
    for i, (row, p) in enumerate(zip(q, pos)):
        hi = min(p + 1, len(k)) if causal else len(k)
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        x = k[lo:hi] @ row * scale
        with np.errstate(invalid="ignore"):
            w = np.exp(x - x.max())
            out[i] = w @ v[lo:hi] / w.sum()
            size[i] = w @ np.abs(v[lo:hi]) / w.sum()
            lse[i] = x.max() + np.log(w.sum())
            reach[i] = (np.abs(k[lo:hi]) @ np.abs(row)).max() * abs(scale)
    return out, lse, size, reach
