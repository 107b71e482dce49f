"""The gate far below zero: silu(g) of -87 to -103 is 1e-36 and less, times an up of 2^60 and more
an ordinary number. Products of one term, exact in float32; the gate as bounded in test_gpu_experts."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import handle
from oracle import experts as ox
from test_gpu_experts import mx  # noqa: F401
from test_gpu_fp4 import on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 30, 300])
@pytest.mark.parametrize("n", [128, 256])
def test_gate_far_below_zero(mx, rows, n):  # noqa: F811
    """Gate i of row r: E4M3 code a[r] times 1, and up i 2^60 to 2^100: g from -120 to 120."""
    k = 128
    grid = np.array([-120, -104, -96, -88, -80, -72, -60, -44, -20, -9, -1, 0, 1, 9, 20, 80, 88, 96, 120.0])
    a = np.zeros((rows, k))
    a[:, 0] = grid[np.arange(rows) % grid.size]
    a[:, 32] = 1.0
    aq = oracle.e4m3_encode(a)
    as_ = np.full((rows, k // 32), 127, np.uint8)
    codes = np.zeros((n, k), np.uint8)
    codes[0::2, 0] = 2   # 1.0
    codes[1::2, 32] = 2
    ws = np.full((n, k // 32), 127, np.uint8)
    up = 60 + np.arange(n // 2) % 41
    ws[1::2, 1] = 127 + up
    # eighths between the grid's values: a second term of the gate rows, 0 to 7/8 of -1
    codes[0::2, 1] = np.arange(n // 2) % 3
    a2 = a.copy()
    a2[:, 1] = -1.0
    aq = oracle.e4m3_encode(a2)
    av, wv = ox.decode_fp8(aq, as_), ox.decode_fp4(ox.pack(codes), ws)
    y = av @ wv.T
    offsets = np.array([0, rows], np.int32)
    out = mx.mx_gemm_fp4_grouped(handle(), on_gpu(aq), on_gpu(as_), on_gpu(ox.pack(codes)[None]),
                                 on_gpu(oracle.swizzle_scales(ws).reshape(1, -1)), on_gpu(offsets), gated=True)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    ref, g = ox.silu_gate(y), y[:, 0::2]
    # below -87 exp(g) is a float32 subnormal, off by half of 2^-149
    tiny = np.abs(g) * 2.0**-149 * np.abs(y[:, 1::2])
    tol = (6 + 1.2 * np.abs(g)) * 2.0**-22 * np.abs(ref) + tiny
    tol = tol + 2.0**-8 * (np.abs(ref) + tol) + 1e-37
    d = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (d <= tol).all(), (d / tol).max()
