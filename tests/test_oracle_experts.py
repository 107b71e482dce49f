"""Pins of the oracle's MXFP4 and routing functions against closed forms, exact
fractions and other ways to the same answer."""
import itertools
from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle import experts as ox


def test_e2m1_values_and_ties():
    assert ox.e2m1_decode(np.arange(16)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, code in ties.items():
        assert ox.e2m1_encode(v) == code
        assert ox.e2m1_encode(-v) == code + 8
        assert ox.e2m1_encode(np.nextafter(v, 9)) == code + (ox.E2M1[code] < v)
        assert ox.e2m1_encode(np.nextafter(v, 0)) == code - (ox.E2M1[code] > v)
    assert ox.e2m1_encode(100.0) == 7 and ox.e2m1_encode(-0.0) == 8


def test_pack_order():
    c = np.arange(8, dtype=np.uint8)[None]
    assert ox.pack(c).tolist() == [[0x10, 0x32, 0x54, 0x76]]
    assert (ox.unpack(ox.pack(c)) == c).all()


def test_quantize_special_blocks():
    x = np.zeros((1, 32 * 5))
    x[0, 32:64] = 6.0
    x[0, 64:96] = -7.99  # saturates under the block's exponent
    x[0, 96] = np.inf
    x[0, 128:] = 2.0**-130
    q, s, v = ox.quantize_fp4(x)
    assert s.tolist() == [[0, 127, 127, 255, 0]]
    assert (v[0, :32] == 0).all() and (v[0, 32:64] == 6).all() and (v[0, 64:96] == -6).all()
    assert np.isnan(v[0, 96:128]).all() and (v[0, 128:] == 0).all()
    ok = ~np.isnan(v)
    assert (ox.decode_fp4(q, s)[ok] == v[ok]).all()


def test_quantize_is_nearest_in_fractions():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((4, 64)) * np.exp2(rng.integers(-20, 20, (4, 2)).astype(float)).repeat(32, 1)).astype(np.float32)
    _, s, v = ox.quantize_fp4(x)
    for r, c in itertools.product(range(4), range(64)):
        unit = Fraction(2) ** (int(s[r, c // 32]) - 127)
        exact = Fraction(float(x[r, c]))
        best = min(abs(abs(exact) - Fraction(float(m)) * unit) for m in ox.E2M1)
        assert abs(exact - Fraction(float(v[r, c]))) == best


def test_route_against_counting():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 24))
    bias = 0.3 * rng.standard_normal(24)
    w, e = ox.route(x, 4, bias=bias, scoring="sigmoid", n_groups=4, topk_groups=2, scale=2.0)
    key = 1 / (1 + np.exp(-x)) + bias
    for i in range(40):
        top2 = np.sort(key[i].reshape(4, 6), 1)[:, -2:].sum(1)
        groups = [g for g in range(4) if (top2 > top2[g]).sum() < 2]
        allowed = [6 * g + j for g in groups for j in range(6)]
        want = [j for j in allowed if sum(key[i, k] > key[i, j] for k in allowed) < 4]
        assert sorted(e[i]) == sorted(want)
        assert (np.diff(key[i, e[i]]) <= 0).all()
    assert np.allclose(w.sum(1), 2.0)


def test_route_masks_and_ties():
    x = np.full((3, 8), -np.inf)
    x[1, 5] = 0.0
    x[2] = 1.0
    w, e = ox.route(x, 3)
    assert e.tolist() == [[0, 1, 2], [5, 0, 1], [0, 1, 2]]
    assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0] and np.allclose(w[2], 1 / 3)


def test_row_order_is_stable_and_inverse():
    rng = np.random.default_rng(7)
    experts = np.argsort(rng.random((50, 9)), 1)[:, :3]
    offsets, tokens, slots = ox.row_order(experts, 9)
    flat = np.argsort(experts.reshape(-1), kind="stable")
    assert (tokens == flat // 3).all() and offsets[-1] == 150
    assert (slots.reshape(-1)[flat] == np.arange(150)).all()


@pytest.mark.parametrize("g,u", [(0.0, 3.0), (50.0, 2.0), (-20.0, 2.0), (1.0, -1.0)])
def test_silu_gate(g, u):
    got = ox.silu_gate(np.array([[g, u]]))[0, 0]
    assert np.isclose(got, u * g * 0.5 * (1 + np.tanh(g / 2)), rtol=1e-6)


def test_fp8_decode_shares_the_scale_rule():
    q, s = oracle.mx_quantize(np.linspace(-3, 3, 64)[None])
    assert np.abs(ox.decode_fp8(q, s) - np.linspace(-3, 3, 64)).max() < 3 * 2.0**-4


def test_route_bias_of_plus_infinity():
    """+inf counts as the largest float32: such experts come first, the lowest index first."""
    x = np.zeros((1, 6))
    bias = np.array([0.1, np.inf, 0.3, np.inf, np.nan, np.finfo(np.float32).max])
    _, e = ox.route(x, 6, bias=bias, scoring="sigmoid")
    assert e.tolist() == [[1, 3, 5, 2, 0, 4]]
