"""Products with MXFP4 weights whose rows are cut into slices for clusters along K, the last
slice shorter than the others, against the float64 oracle (bounds as in test_gpu_fp4)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import handle
from test_gpu_fp4 import bound, guarded, intact, mx, on_gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("m,n,k,fp4", [(300, 4096, 8192, False), (300, 2048, 10368, True), (257, 2048, 10368, False),
                                       (257, 4096, 8192, True), (340, 2560, 8192, False), (600, 2048, 8192, False)])
def test_product_in_slices_with_a_short_last_one(mx, m, n, k, fp4, pdl):  # noqa: F811
    """The activation scales end with the last row's tile; what follows them is scales of NaN."""
    rng = np.random.default_rng(m + n + k)
    aq, as_, av = operand(rng, m, k, fp4)
    wq, ws, wv = operand(rng, n, k, True)
    scales = oracle.swizzle_scales(as_).reshape(-1)
    assert scales.size == mx.mx_scale_bytes(m, k)
    buf = torch.full((scales.size + (1 << 18),), 0xFF, dtype=torch.uint8, device="cuda:0")
    buf[:scales.size] = on_gpu(scales)
    ob, o = guarded(m * n * 2)
    out = o.view(torch.bfloat16).view(m, n)
    args = [on_gpu(aq), buf[:scales.size], on_gpu(wq), on_gpu(oracle.swizzle_scales(ws))]
    torch.cuda.synchronize()
    for _ in range(2):
        mx.mx_gemm_fp4(handle(), *args, out=out, pdl=pdl)
    assert mx.mx_device_status(handle()) == mx.MX_OK
    ref = av @ wv.T
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound(av, wv, ref)).all(), (err / bound(av, wv, ref)).max()
    assert intact(ob, m * n * 2)
