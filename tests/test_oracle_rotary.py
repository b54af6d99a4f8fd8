"""Pins of the rotary oracle: independent formulas, hand values, what rotations keep."""
import math

import numpy as np
import pytest

from oracle import rotary


def freqs(rd, **kw):
    return [rotary.frequency(i, rd, 10000.0, **kw) for i in range(rd // 2)]


def test_plain_frequencies_by_hand():
    assert freqs(16) == pytest.approx([1, 0.31622776601683794, 0.1, 0.031622776601683794, 0.01, 0.0031622776601683794, 0.001, 0.00031622776601683794], rel=1e-14)


@pytest.mark.parametrize("scaling,kw", [("linear", {}), ("ntk", {}), ("yarn", dict(original=4096, low=1, high=32)), ("banded", dict(original=8192, low=1, high=4))])
def test_scalings_stay_between_their_limits(scaling, kw):
    f, g = freqs(64), freqs(64, scaling=scaling, factor=8.0, **kw)
    assert all(a / 8 * (1 - 1e-12) <= b <= a * (1 + 1e-12) for a, b in zip(f, g))
    assert all(x > y for x, y in zip(g, g[1:]))  # slower from pair to pair
    if scaling in ("yarn", "banded"):
        assert g[0] == f[0] and g[-1] == pytest.approx(f[-1] / 8, rel=1e-14)
    if scaling == "ntk":
        assert g[0] == 1 and g[-1] == pytest.approx(f[-1] / 8, rel=1e-12)  # the slowest pair is stretched by the factor
    assert freqs(64, scaling=scaling, factor=1.0, **kw) == pytest.approx(f, rel=1e-14)


def test_banded_half_way_by_hand():
    f = 2.5 * 2 * math.pi / 8192  # turns 2.5 times: half way between 1 and 4
    i = -math.log(f, 10000.0) * 64
    assert rotary.frequency(i, 128, 10000.0, "banded", 8.0, 8192, 1, 4) == pytest.approx((f + f / 8) / 2, rel=1e-12)


def test_norm_by_hand():
    x = np.zeros((1, 256))
    x[0, :4] = 8, -8, 8, -8  # mean of squares 1
    w = np.arange(256.0)
    assert rotary.norm(x, w, 0.0)[0, :5].tolist() == [0, -8, 16, -24, 0]
    assert rotary.norm(np.full((1, 256), 3.0), np.ones(256), 7.0)[0, 0] == 0.75


def test_quarter_turns_by_hand():
    x = np.arange(512.0).reshape(2, 256)
    f = [math.pi / 2] * 8
    y = rotary.turn(x, np.array([1, 2]), f, True)
    assert np.allclose(y[0, :4], [-1, 0, -3, 2]) and np.allclose(y[1, :2], [-256, -257]) and (y[:, 16:] == x[:, 16:]).all()
    y = rotary.turn(x, np.array([1, 3]), f, False, 2.0)
    assert np.allclose(y[0, [0, 8, 1, 9]], [-16, 0, -18, 2]) and np.allclose(y[1, [0, 8]], [2 * 264, -2 * 256])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rd", [16, 96, 256])
def test_products_see_distances_only(interleaved, rd):
    g = np.random.default_rng(1)
    q, k = g.standard_normal((2, 1, 256))
    f = freqs(rd)

    def score(t, s):
        return float((rotary.turn(q, np.array([t]), f, interleaved) @ rotary.turn(k, np.array([s]), f, interleaved).T)[0, 0])
    assert score(70, 3) == pytest.approx(score(1000070, 1000003), abs=1e-7)
    assert abs(score(70, 3) - score(71, 3)) > 1e-3
    y = rotary.turn(q, np.array([12345]), f, interleaved)
    assert np.linalg.norm(y) == pytest.approx(np.linalg.norm(q), rel=1e-12) and (y[:, rd:] == q[:, rd:]).all()
    assert np.allclose(rotary.turn(y, np.array([-12345]), f, interleaved), q, atol=1e-12)


def test_layouts_are_one_permutation_apart():
    x = np.random.default_rng(2).standard_normal((3, 256))
    f, at = freqs(64), np.array([5, 6, 700])
    order = np.arange(256)
    order[0:64:2], order[1:64:2] = np.arange(32), np.arange(32, 64)
    assert np.allclose(rotary.turn(x[:, order], at, f, True), rotary.turn(x, at, f, False)[:, order], atol=1e-14)
