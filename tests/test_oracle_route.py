"""The router oracle pinned by hand and its gradient against differences."""

import numpy as np
import pytest

from oracle import route as R


def test_choice_by_hand():
    inf = np.inf
    l = np.array([[1.0, 3.0, 3.0, 2.0],             # a tie: the lower expert first
                  [-inf, -inf, -inf, -inf],         # nothing to choose
                  [-inf, 0.0, -inf, -inf],          # one of two
                  [0.0, np.nan, 1.0, -0.0],         # a NaN is not chosen
                  [9.0, 9.0, 9.0, 9.0]])            # masked
    r = R.route(l, 2, mask=np.array([1, 1, 1, 1, 0]), alpha=1.0)
    assert r["index"].tolist() == [[1, 2], [-1, -1], [1, -1], [2, 0], [-1, -1]]
    assert r["counts"].tolist() == [1, 2, 2, 0] and r["offsets"].tolist() == [0, 1, 3, 5, 5]
    assert r["order"].tolist() == [7, 0, 4, 1, 6, 2, 3, 5, 8, 9] and r["live"] == 3
    assert r["weight"][0].tolist() == [0.5, 0.5] and r["weight"][2].tolist() == [1.0, 0.0]
    assert np.isnan(r["weight"][3]).all() and np.isnan(r["loss"])


def test_loss_is_one_when_balanced():
    # every expert once, uniform probabilities: E * sum (1/E) (1/E) = 1
    l = np.zeros((4, 4))
    l[np.arange(4), np.arange(4)] = 1e-9
    r = R.route(l, 1, alpha=1.0)
    assert r["counts"].tolist() == [1, 1, 1, 1] and abs(r["loss"] - 1.0) < 1e-6


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    rng = np.random.default_rng(1)
    T, E, k = 5, 7, 3
    l = rng.standard_normal((T, E))
    l[1, 2:6] = -np.inf
    l[2] = -np.inf
    mask = np.array([1, 1, 1, 0, 1])
    r = R.route(l, k, mask, renorm, 0.7)
    dw, dl = rng.standard_normal((T, k)), 1.3
    args = (r["index"], r["counts"], r["live"], dw, dl, 0.7, mask, renorm)
    g = R.gradient(l, *args)
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert g[t, e] == 0.0
                continue
            h = 1e-6
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            d = (R.objective(a, *args) - R.objective(b, *args)) / (2 * h)
            assert abs(d - g[t, e]) < 1e-8
