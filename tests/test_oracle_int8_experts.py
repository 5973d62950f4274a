"""Pins of the integer and routing oracles (no GPU): closed forms, invariants and
planted mistakes."""

import numpy as np
import pytest

from oracle import experts as X
from oracle import int8 as I


def test_quantizer_closed_forms():
    y = np.zeros((3, 32), np.float32)
    y[0, :6] = [127.0, -127.0, 0.5, 1.5, -2.5, 3.49]
    y[2, 3] = 1e-40
    codes, s, _ = I.quantize_rows(y)
    assert s.tolist() == [1.0, 2.0**-126, 2.0**-126]
    assert codes[0, :6].tolist() == [127, -127, 0, 2, -2, 3]
    assert (codes[1] == 0).all() and (codes[2] == 0).all()


def test_quantizer_error_is_half_a_step():
    rng = np.random.default_rng(2)
    y = (rng.standard_normal((40, 96)) * np.exp2(rng.integers(-60, 60, (40, 1)))).astype(np.float32)
    codes, s, _ = I.quantize_rows(y)
    assert np.abs(codes).max() == 127
    assert (np.abs(I.dequant(codes, s) - y) <= s[:, None].astype(np.float64) * (0.5 + 2.0**-16)).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_quantizer_nonfinite_rows(bad):
    y = np.ones((3, 16), np.float32)
    y[1, 5] = bad
    codes, s, _ = I.quantize_rows(y)
    assert np.isnan(s[1]) and (codes[1] == 0).all() and np.isfinite(s[[0, 2]]).all()


def test_linear_against_integers():
    rng = np.random.default_rng(3)
    x, w = rng.integers(-127, 128, (5, 4000)), rng.integers(-127, 128, (7, 4000))
    y, size = I.linear(x.astype(np.int8), np.ones(5, np.float32), w.astype(np.int8), np.full(7, 2.0, np.float32))
    assert np.array_equal(y, 2.0 * (x @ w.T)) and np.array_equal(size, np.abs(y))


def test_route_closed_forms():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    ids, w = X.route_token(l, 2, renormalize=False)
    assert ids.tolist() == [1, 2] and np.allclose(w, [0.5, 0.25])
    ids, w = X.route_token(l, 3)
    assert ids.tolist() == [1, 2, 0] and np.allclose(w, np.array([4, 2, 1]) / 7)  # a tie goes to the lowest index
    ids, w = X.route_token(np.zeros(4), 2, kind="sigmoid", bias=[0, 0, 0.5, 0.25], renormalize=False, scale=3.0)
    assert ids.tolist() == [2, 3] and np.allclose(w, 1.5)  # the bias chooses and does not weigh


def test_route_groups():
    l = np.array([9.0, 0.0, 5.0, 5.0, 4.0, 4.5])
    assert X.route_token(l, 2, groups=3, keep=1)[0].tolist() == [0, 1]
    s = X.scores(l, "sigmoid")
    assert s[2] + s[3] > s[0] + s[1]
    assert X.route_token(l, 2, kind="sigmoid", groups=3, keep=1, pairs=True)[0].tolist() == [2, 3]
    # a group with one expert left counts by that one
    l = np.array([3.0, -np.inf, 1.0, 1.0])
    assert X.route_token(l, 2, kind="sigmoid", groups=2, keep=1, pairs=True)[0].tolist() == [2, 3]
    assert X.route_token(l, 3, kind="sigmoid", groups=2, keep=1)[0].tolist() == [0, -1, -1]


def test_route_masks_and_nan():
    inf, nan = np.inf, np.nan
    ids, w = X.route_token(np.full(4, -inf), 2)
    assert ids.tolist() == [-1, -1] and (w == 0).all()
    ids, w = X.route_token(np.array([-inf, 0.0, -inf, -inf]), 2)
    assert ids.tolist() == [1, -1] and w.tolist() == [1.0, 0.0]
    ids, w = X.route_token(np.array([1.0, nan, 2.0, nan]), 3)
    assert ids.tolist() == [1, 3, 2] and np.isnan(w).all()
    ids, w = X.route_token(np.array([1.0, nan, 2.0]), 2, kind="sigmoid", renormalize=False)
    assert ids.tolist() == [1, 2] and np.isnan(w[0]) and w[1] == 1 / (1 + np.exp(-2.0))
    assert np.isnan(X.route_token(np.array([1.0, inf, 2.0]), 2)[1]).all()


def test_order():
    ids = np.array([[2, 0], [0, -1], [2, 1]], np.int32)
    off, rows, places = X.order(ids, 4)
    assert off.tolist() == [0, 2, 3, 5, 5] and rows.tolist() == [0, 1, 2, 0, 2]
    assert places.tolist() == [[3, 0], [1, -1], [4, 2]]


def test_combine():
    y = np.array([[1.0, 2.0], [10.0, 20.0]])
    out, size = X.combine(y, np.array([[1, 0], [-1, 1], [7, -1]]), np.array([[0.5, -1.0], [9.0, 2.0], [1.0, 1.0]]), np.ones((3, 2)))
    assert out.tolist() == [[5.0, 9.0], [21.0, 41.0], [1.0, 1.0]] and size[0].tolist() == [7.0, 13.0]
