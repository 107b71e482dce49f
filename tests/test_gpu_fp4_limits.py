"""Sizes at the ends of the MXFP4 quantizer's range: refused before anything is launched, or right."""
import pytest
import torch

from gpu_helpers import dev, handle
from test_gpu_experts import mx  # noqa: F401

pytestmark = pytest.mark.gpu


def test_swizzled_scales_past_32_bits_are_refused(mx):  # noqa: F811
    """A few rows of 2^30 elements and more: their scales, padded to 128 rows, pass 2^32 bytes."""
    h, lib = handle(), mx.load_library()
    out = torch.full((4096,), 0xA5, dtype=torch.uint8, device=dev())
    p, st = out.data_ptr(), torch.cuda.current_stream().cuda_stream
    for m, k in ((1, 1 << 30), (15, 1 << 30), (7, 2147483616)):
        assert m * k < 1 << 34 and mx.mx_scale_bytes(m, k) >= 1 << 32
        assert lib.mx_quantize_rows_fp4(h.ptr, m, k, p, k, 0, p, p, 1, None, st) == mx.MX_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (out == 0xA5).all()


def test_longest_swizzled_row(mx):  # noqa: F811
    """One row of 2^30 - 128 elements: its last scales lie 4 GB into the buffer."""
    k = (1 << 30) - 128
    x = torch.zeros((1, k), dtype=torch.bfloat16, device=dev())
    x[0, -32:] = 6.0
    x[0, :32] = 12.0
    q, s, _ = mx.mx_quantize_rows_fp4(handle(), x)
    assert s.numel() == mx.mx_scale_bytes(1, k) < 1 << 32
    assert q[0, :16].eq(0x77).all() and q[0, -16:].eq(0x77).all() and q[0, 16:-16].max() == 0
    last = s.numel() - 512  # the last 128x4 tile; its row 0 is the first four bytes
    assert s[0] == 128 and s[last + 3] == 127
    assert int(s.count_nonzero()) == 2
