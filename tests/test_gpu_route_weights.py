"""Router weights at the end of the scores' range against the float64 oracle, row by row.

Bound: float32 scores are off by (2 + d) units where the logit is d below the top one (0 for
sigmoid), the sum and the divisions by a few more: (40 + d) 2^-23 of the weight. A score below
float32's normal range is off by up to 2^-149 and is used where the sum is 2^-20 at least:
2^-129 of a weight's unit."""
import numpy as np
import pytest

from gpu_helpers import handle
from oracle import experts as ox
from test_gpu_experts import mx  # noqa: F401
from test_gpu_fp4 import on_gpu

pytestmark = pytest.mark.gpu


def check_weights(mx, x, top_k, **kw):  # noqa: F811
    bias = kw.get("bias")
    got = mx.mx_route(handle(), on_gpu(x), top_k, **{**kw, "bias": None if bias is None else on_gpu(bias)})
    w, experts = ox.route(x, top_k, **kw)
    assert np.array_equal(got["experts"].cpu().numpy(), experts)
    picked = np.take_along_axis(x.astype(np.float64), experts, 1)
    top = x.max(1, keepdims=True) if kw["scoring"] == "softmax" else picked
    d = np.where(np.isfinite(picked), np.where(np.isfinite(top), top, 0.0) - np.where(np.isfinite(picked), picked, 0.0), 0.0)
    scale = kw.get("scale", 1.0)
    err = np.abs(got["weights"].cpu().numpy().astype(np.float64) - w)
    tol = (40 + d) * 2.0**-23 * np.abs(w) + scale * 2.0**-129
    assert (err <= tol).all(), (err / tol).max()
    return w


@pytest.mark.parametrize("groups,top,k", [(1, 1, 6), (6, 2, 6), (6, 6, 20)])
@pytest.mark.parametrize("bias", [False, True])
def test_sigmoid_scores_far_below_zero(mx, groups, top, k, bias):  # noqa: F811
    """Logits around -14 (sums near 2^-20) to -700: their scores' float32 is small, subnormal or 0."""
    rng = np.random.default_rng(k)
    at = np.repeat([-5, -10, -13, -14, -16, -20, -40, -79, -81, -86, -88, -90, -95, -100, -103, -105, -120, -300, -690.0], 3)
    x = (at[:, None] + 2 * rng.standard_normal((at.size, 48))).astype(np.float32)
    x[1::3, ::5] = -np.inf
    x[2::3, 7] = 0.0
    b = (0.1 * rng.standard_normal(48)).astype(np.float32) if bias else None
    w = check_weights(mx, x, k, bias=b, scoring="sigmoid", n_groups=groups, topk_groups=top, scale=2.5)
    # all weights are of a full sum, unless every chosen expert is masked
    assert np.allclose(w.sum(1), 2.5)
    check_weights(mx, x, k, bias=b, scoring="sigmoid", n_groups=groups, topk_groups=top, renormalize=False)


@pytest.mark.parametrize("far", [5, 14, 50, 86, 95, 104, 120, 400, 600])
def test_softmax_scores_far_below_the_top(mx, far):  # noqa: F811
    """A bias that chooses experts `far` below the top logit."""
    rng = np.random.default_rng(far)
    x = rng.standard_normal((40, 64)).astype(np.float32)
    x[:, :32] += far
    x[3, 40:50] = -np.inf
    b = np.where(np.arange(64) < 32, -4.0, 0.0).astype(np.float32) + (0.1 * rng.random(64)).astype(np.float32)
    for groups, top in ((1, 1), (8, 3)):
        w = check_weights(mx, x, 5, bias=b, scoring="softmax", n_groups=groups, topk_groups=top)
        assert np.allclose(w.sum(1), 1.0)
        check_weights(mx, x, 5, bias=b, scoring="softmax", n_groups=groups, topk_groups=top, renormalize=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_no_score_at_all(mx, scoring):  # noqa: F811
    x = np.full((9, 20), -np.inf, np.float32)
    x[1], x[2] = -2000.0, np.finfo(np.float32).min
    b = np.zeros(20, np.float32)
    w = check_weights(mx, x, 4, bias=b, scoring=scoring)
    assert (w[0] == 0).all() and (w[3:] == 0).all()
