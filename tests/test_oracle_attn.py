"""Pins of oracle.attn: hand-worked masks and weights, closed forms, gradients against differences."""

import numpy as np
import pytest

from oracle import attn as oa


def test_masks_by_hand():
    p, j = [1, 2], range(4)
    assert oa.seen(p, j).astype(int).tolist() == [[1, 1, 0, 0], [1, 1, 1, 0]]
    assert oa.seen(p, j, causal=False).all()
    assert oa.seen(p, j, window=2).astype(int).tolist() == [[1, 1, 0, 0], [0, 1, 1, 0]]
    assert oa.seen(p, j, window=1, prefix=1).astype(int).tolist() == [[1, 1, 0, 0], [1, 0, 1, 0]]
    assert oa.seen([0], j, prefix=3).astype(int).tolist() == [[1, 1, 1, 0]]
    assert oa.seen([-1], j).sum() == 0
    assert oa.seen([1], j, causal=False, window=1).astype(int).tolist() == [[0, 1, 1, 1]]


def test_weights_by_hand():
    a = np.log(np.array([[1.0, 3.0, 5.0], [2.0, 2.0, 7.0]]))
    ok = np.array([[True, True, False], [False, False, False]])
    w, lse = oa.weights(a, ok)
    np.testing.assert_allclose(w, [[0.25, 0.75, 0.0], [0, 0, 0]], rtol=1e-15)
    np.testing.assert_allclose(lse, [np.log(4.0), -np.inf], rtol=1e-15)


def test_equal_scores_average_and_slopes_decay():
    v = np.arange(12.0).reshape(4, 3)
    q, k = np.zeros((1, 2)), np.ones((4, 2))
    out, lse, *_ = oa.attend(q, k, v, [3], range(4), sm_scale=1.0)
    np.testing.assert_allclose(out[0], v.mean(0), rtol=1e-14)
    assert abs(lse[0] - np.log(4)) < 1e-14
    out, *_ = oa.attend(q, k, v, [3], range(4), sm_scale=1.0, slope=np.log(2.0))
    np.testing.assert_allclose(out[0], (np.array([1, 2, 4, 8.0]) @ v) / 15, rtol=1e-14)


def test_cap_bounds_scores():
    q, k = np.full((1, 1), 100.0), np.array([[1.0], [-1.0], [0.001]])
    a, slant, _ = oa.scores(q, k, [2], range(3), sm_scale=1.0, cap=5.0)
    np.testing.assert_allclose(a[0], [5, -5, 5 * np.tanh(0.02)], rtol=1e-12)
    np.testing.assert_allclose(slant[0], [0, 0, 1 - np.tanh(0.02) ** 2], atol=1e-12)


@pytest.mark.parametrize("more", [{}, dict(causal=False), dict(window=3), dict(prefix=2, window=2),
                                  dict(cap=0.7), dict(cap=2.0, slope=0.3, prefix=4)])
def test_gradients_against_differences(more):
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((n, 4)) for n in (5, 7, 7))
    dout = rng.standard_normal((5, 4))
    p, j = np.arange(5) + 2, np.arange(7)
    args = dict(sm_scale=0.6, **more)
    got, _ = oa.gradients(q, k, v, dout, p, j, **args)
    for x, g in zip((q, k, v), got):
        for at in np.ndindex(*x.shape):
            old, d = x[at], 1e-5
            x[at] = old + d
            up = (oa.attend(q, k, v, p, j, **args)[0] * dout).sum()
            x[at] = old - d
            down = (oa.attend(q, k, v, p, j, **args)[0] * dout).sum()
            x[at] = old
            assert abs((up - down) / (2 * d) - g[at]) < 1e-8


def test_cached_rows():
    cache = np.arange(3 * 2 * 1 * 2).reshape(3, 2, 1, 2)
    assert oa.cached_row(cache, [2, 0], 1).tolist() == [[10, 11]]
    assert oa.cached_row(cache, [2, 0], 2).tolist() == [[0, 1]]
    assert oa.cached_row(cache, [2, 0], 4) is None
    assert oa.cached_row(cache, [3, -1], 0) is None
    assert oa.cached_row(cache, [3, -1], 3) is None
