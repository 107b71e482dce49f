"""Offsets of the grouped product that fall: reported, and nothing is written."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, handle
from test_gpu_experts import experts_case, mx  # noqa: F401
from test_gpu_fp4 import on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("n", [128, 256])
@pytest.mark.parametrize("r", [10, 400])
def test_falling_offsets(mx, r, n, fp4, gather):  # noqa: F811
    rng = np.random.default_rng(r)
    counts = [r // 2, 0, r - r // 2] + [0] * 37
    args, _, _ = experts_case(rng, counts, 20, 256, n, fp4, gather)
    right = args["offsets"].clone()
    want = mx.mx_gemm_fp4_grouped(handle(), **args)
    out = torch.full((r, n), 7.0, dtype=torch.bfloat16, device=dev())
    for at, value in ((2, 1), (40, r - 1), (1, r), (33, -4)):
        args["offsets"] = right.clone()
        args["offsets"][at] = value
        mx.mx_gemm_fp4_grouped(handle(), out=out, **args)
        assert mx.mx_device_status(handle()) == mx.MX_ERR_INVALID_ARG, (at, value)
        assert out.eq(7).all()
    # falling beyond the ends is the same end
    args["offsets"] = right.clone()
    args["offsets"][0], args["offsets"][1:][right[1:] == r] = -3, r + 9
    args["offsets"][40] = r + 2
    mx.mx_gemm_fp4_grouped(handle(), out=out, **args)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    assert torch.equal(out, want)
