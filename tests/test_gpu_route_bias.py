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


def large_biases(rng, e):
    """Finite masks of some experts, keys that cancel in a group's sum, biases of many sizes, and
    sums beyond float32."""
    base = (0.2 * rng.standard_normal(e)).astype(np.float32)
    for v in (-1e9, 1e9, -1e4, 3e38, -3e38):
        for at in ([e // 2], np.arange(0, e, 5), np.arange(e // 4, e)):
            b = base.copy()
            b[at] = v
            yield b
    b = base.copy()
    b[::4], b[1::4] = 1e9, -1e9
    yield b
    b = base.copy()
    b[0::8], b[1::8] = 1e7 * (1 + rng.random(len(b[0::8]))), -1e7 * (1 + rng.random(len(b[1::8])))
    yield b
    yield (rng.standard_normal(e) * 10.0 ** rng.integers(-6, 9, e)).astype(np.float32)
    yield (rng.integers(-3, 4, e) * 2.0 ** rng.integers(-26, 26, e)).astype(np.float32)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,groups,top", [(64, 6, 1, 1), (64, 6, 8, 2), (64, 4, 32, 5), (48, 5, 48 // 2, 7), (32, 3, 32, 4),
                                            (256, 8, 8, 4), (512, 32, 1, 1)])
def test_large_biases(mx, e, k, groups, top, scoring):  # noqa: F811
    rng = np.random.default_rng(e * k)
    x = (2 * rng.standard_normal((33, e))).astype(np.float32)
    x[3, ::2] = -np.inf
    x[4] = -np.inf
    x[5, 1:] = -np.inf
    x[6:9] = np.round(2 * x[6:9]) / 2
    x[6:9][np.isinf(x[6:9])] = 0
    for b in large_biases(rng, e):
        check_route(mx, on_gpu(x), k, bias=b, scoring=scoring, n_groups=groups, topk_groups=top)
