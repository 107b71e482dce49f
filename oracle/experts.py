"""CPU oracle of the MXFP4 and expert-layer operators, in numpy float64.

TEST INFRASTRUCTURE ONLY, as the package's main module. Written from the formats'
and operators' definitions; it shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import SCALE_NAN, SF_VEC, e4m3_decode, ue8m0_decode

# E2M1: sign, two exponent bits (bias 1), one mantissa bit; no infinity, no NaN
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(v) -> np.ndarray:
    """Codes 0..15 of float64 values: the nearest of the eight magnitudes, ties to the
    even code, larger ones saturate; the sign of zero is kept."""
    v = np.asarray(v, dtype=np.float64)
    d = np.abs(np.abs(v)[..., None] - E2M1)
    # an odd code loses a tie: the distances are exact for the values met here
    best = d.min(-1, keepdims=True)
    tied = d == best
    even = tied & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tied.argmax(-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def e2m1_decode(c) -> np.ndarray:
    c = np.asarray(c).astype(np.int64)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def pack(codes) -> np.ndarray:
    """Two codes to a byte, the first in the low bits."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q) -> np.ndarray:
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)


def quantize_fp4(x) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """Rows [R, K] -> (packed codes [R, K/2], scale bytes [R, K/32], values [R, K])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, SF_VEC)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, np.abs(b).max(-1))
    _, ex = np.frexp(amax)
    e = np.where(amax > 0, np.maximum(ex - 1 - 2, -127), -127)
    unit = np.exp2(e.astype(np.float64))[..., None]
    codes = e2m1_encode(np.where(bad[..., None], 0.0, b) / unit)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    values = np.where(bad[..., None], np.nan, e2m1_decode(codes) * unit)
    scales = np.where(bad, SCALE_NAN, e + 127).astype(np.uint8)
    return pack(codes.reshape(x.shape)), scales, values.reshape(x.shape)


def decode_fp4(q, s) -> np.ndarray:
    return e2m1_decode(unpack(q)) * np.repeat(ue8m0_decode(s), SF_VEC, -1)


def decode_fp8(q, s) -> np.ndarray:
    return e4m3_decode(q) * np.repeat(ue8m0_decode(s), SF_VEC, -1)


def route(logits, top_k, bias=None, scoring="softmax", n_groups=1, topk_groups=1, renormalize=True, scale=1.0):
    """Selection by sorting float64 keys token by token."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    t, e = x.shape
    size = e // n_groups
    weights = np.zeros((t, top_k))
    experts = np.zeros((t, top_k), dtype=np.int64)
    for i in range(t):
        row = x[i]
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-row))
        elif np.isneginf(row).all():
            s = np.zeros(e)
        else:
            s = np.exp(row - row.max())
            s /= s.sum()
        key = row.copy()
        if bias is not None:
            b = np.minimum(np.asarray(bias, dtype=np.float64), np.finfo(np.float32).max)  # NaN stays
            key = np.where(np.isneginf(row) | np.isnan(b), -np.inf, s + b)
        allowed = range(e)
        if n_groups > 1:
            g = np.sort(key.reshape(n_groups, size), 1)[:, ::-1]
            best = g[:, 0] if bias is None or size == 1 else g[:, 0] + g[:, 1]
            chosen = sorted(range(n_groups), key=lambda j: (-best[j], j))[:topk_groups]
            allowed = [j for j in range(e) if j // size in chosen]
        picked = sorted(allowed, key=lambda j: (-key[j], j))[:top_k]
        w = s[picked]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        experts[i], weights[i] = picked, w * scale
    return weights, experts


def row_order(experts, e):
    """offsets [e + 1], tokens [t * k], slots [t, k] of the pairs ordered by expert."""
    t, k = experts.shape
    flat = experts.reshape(-1)
    pairs = sorted(range(t * k), key=lambda r: (flat[r], r))
    slots = np.zeros(t * k, dtype=np.int64)
    slots[pairs] = np.arange(t * k)
    counts = np.bincount(flat, minlength=e)
    return np.concatenate([[0], np.cumsum(counts)]), np.array(pairs) // k, slots.reshape(t, k)


def silu_gate(y):
    """silu(column 2i) * column 2i + 1."""
    g, u = y[:, 0::2], y[:, 1::2]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def combine(y, slots, weights, residual=None):
    out = np.einsum("tk,tkn->tn", np.asarray(weights, np.float64), np.asarray(y, np.float64)[slots])
    return out if residual is None else out + residual
