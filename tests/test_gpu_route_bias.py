"""Routing with biases that are infinite or large against the float64 oracle: every output as in
test_gpu_experts."""
import numpy as np
import pytest

from test_gpu_experts import check_route, mx  # noqa: F401
from test_gpu_fp4 import on_gpu

pytestmark = pytest.mark.gpu


def biases(rng, e):
    """(name, bias): +inf at one, several and all experts, with and without others masked."""
    base = (0.2 * rng.standard_normal(e)).astype(np.float32)
    for name, at in (("one", [e // 3]), ("two", [1, e - 1]), ("four neighbours", [4, 5, 6, 7]),
                     ("every third", np.arange(0, e, 3)), ("all", np.arange(e))):
        b = base.copy()
        b[at] = np.inf
        yield name, b
    b = np.full(e, -np.inf, np.float32)
    b[2], b[5], b[9] = np.inf, 0.1, np.finfo(np.float32).max
    yield "one among -inf", b
    b = base.copy()
    b[::2], b[3], b[8] = np.nan, np.inf, -np.finfo(np.float32).max
    yield "one among NaN", b


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,groups,top", [(12, 1, 1, 1), (64, 1, 1, 1), (64, 6, 1, 1), (64, 6, 8, 2), (128, 3, 4, 1),
                                            (512, 32, 1, 1), (60, 4, 5, 2)])
def test_bias_of_plus_infinity(mx, e, k, groups, top, scoring):  # noqa: F811
    rng = np.random.default_rng(e + k)
    x = (2 * rng.standard_normal((21, e))).astype(np.float32)
    x[3, ::2] = -np.inf
    x[4] = -np.inf
    x[5, 1:] = -np.inf
    for _, b in biases(rng, e):
        check_route(mx, on_gpu(x), k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top)
