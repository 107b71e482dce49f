"""Pins of the attention oracle: closed forms, invariants and brute force, on the CPU."""
import math

import numpy as np
import pytest

from oracle import attention as oa


def test_plain_frequencies_are_a_geometric_sequence():
    f = oa.rope_frequencies(64, base=10000.0)
    assert f[0] == 1 and np.allclose(f[1:] / f[:-1], 10000.0 ** (-1 / 32), rtol=1e-13)


def test_linear_scaling_divides_the_angles():
    a, b = oa.rope_table(40, 16, scaling="linear", factor=4.0), oa.rope_table(10, 16)
    assert np.allclose(a[::4], b, atol=1e-12)


def test_yarn_keeps_fast_pairs_and_interpolates_slow_ones():
    base, d, orig, factor = 10000.0, 64, 4096, 40.0
    f = oa.rope_frequencies(d, base=base)
    g = oa.rope_frequencies(d, base=base, scaling="yarn", factor=factor, original=orig)
    turns = orig * f / (2 * math.pi)
    # a whole pair's width away from the two bounds, whatever their rounding
    step = f[0] / f[1]
    assert np.array_equal(g[turns > 32 * step], f[turns > 32 * step])
    assert np.allclose(g[turns < 1 / step], f[turns < 1 / step] / factor, rtol=1e-15)
    between = (turns < 32 / step) & (turns > step)
    assert between.sum() > 3 and (g[between] < f[between]).all() and (g[between] > f[between] / factor).all()
    assert (np.diff(g) < 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_pairs(interleaved):
    rng = np.random.default_rng(0)
    x, cs = rng.normal(size=(3, 2, 10)), oa.rope_table(7, 6)[[0, 3, 6]]
    y = oa.rope(x, cs, 2, interleaved, False)
    assert np.array_equal(y[..., [0, 1, 8, 9]], x[..., [0, 1, 8, 9]])  # outside the part
    assert np.array_equal(y[0], x[0])                                  # position 0
    assert np.allclose(oa.rope(y, cs, 2, interleaved, True), x, atol=1e-14)
    pair = (2, 3) if interleaved else (2, 5)                           # the first pair turns one radian a position
    z = (x[..., pair[0]] + 1j * x[..., pair[1]]) * np.exp(1j * np.array([0, 3, 6]))[:, None]
    assert np.allclose(y[..., pair[0]], z.real) and np.allclose(y[..., pair[1]], z.imag)


def test_attention_of_equal_keys_is_the_mean_of_what_is_seen():
    v = np.arange(12.0).reshape(6, 2)
    out, lse, _, _ = oa.attend(np.ones((3, 4)), np.zeros((6, 4)), v, 0.5, [3, 4, 5], window=3)
    assert np.allclose(out, [v[1:4].mean(0), v[2:5].mean(0), v[3:6].mean(0)])
    assert np.allclose(lse, math.log(3))
    out, _, _, _ = oa.attend(np.ones((2, 4)), np.zeros((6, 4)), v, 0.5, [0, 1], causal=False)
    assert np.allclose(out, v.mean(0))


def test_attention_by_brute_force():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(2, 8)), rng.normal(size=(5, 8)), rng.normal(size=(5, 3))
    out, lse, size, reach = oa.attend(q, k, v, 0.3, [2, 4])
    for i, p in enumerate((2, 4)):
        e = [math.exp(0.3 * sum(a * b for a, b in zip(q[i], k[t]))) for t in range(p + 1)]
        for d in range(3):
            assert math.isclose(out[i, d], sum(w * v[t, d] for t, w in enumerate(e)) / sum(e), rel_tol=1e-12)
        assert math.isclose(lse[i], math.log(sum(e)), rel_tol=1e-12)
    assert (size >= np.abs(out)).all() and (reach > 0).all()


def test_a_row_that_sees_nothing_is_zero():
    out, lse, _, _ = oa.attend(np.ones((2, 4)), np.ones((1, 4)), np.ones((1, 2)), 1.0, [-1, 0])
    assert (out[0] == 0).all() and lse[0] == -np.inf and (out[1] == 1).all()
