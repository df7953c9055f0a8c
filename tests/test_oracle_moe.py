"""Pins of oracle/moe.py: hand-written routings, and each gradient against
central differences of the function it is the gradient of."""

import numpy as np
import pytest

from oracle import moe


def test_route_by_hand():
    inf = np.inf
    l = np.array([[1.0, 3.0, 3.0, 2.0],        # a tie: the lower expert first
                  [-inf, -inf, 5.0, -inf],     # one open expert
                  [-inf] * 4,                  # none
                  [0.0, np.nan, 1.0, 2.0]])    # NaN above everything
    ids, w = moe.route(l, 2, True)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [1, 3]]
    np.testing.assert_allclose(w[0], [0.5, 0.5])
    np.testing.assert_allclose(w[1:3], [[1.0, 0.0], [0.0, 0.0]])
    assert np.isnan(w[3]).all()
    ids, w = moe.route(l[:1], 3, False)
    z = np.exp([3.0, 3.0, 2.0]) / np.exp(l[0]).sum()
    assert ids.tolist() == [[1, 2, 3]]
    np.testing.assert_allclose(w[0], z)


def test_sort_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 7]])
    offsets, pos, src = moe.sort(ids, 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert src.tolist() == [1, 4, 0, 3, 2, 5]
    assert pos.tolist() == [[2, 0], [~4, 3], [1, ~5]]


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    rng = np.random.default_rng(0)
    l = rng.standard_normal((5, 7))
    l[1, 2] = -np.inf
    l[2, 1:] = -np.inf
    l[3] = -np.inf
    ids, _ = moe.route(l, 3, renorm)
    dw = rng.standard_normal((5, 3))

    def loss(x):
        t, k = ids.shape
        s = 0.0
        for i in range(t):
            ch = [e for e in ids[i] if e >= 0]
            if ch:
                p = moe.softmax(x[i], ch if renorm else None)
                s += sum(dw[i, j] * p[ids[i, j]] for j in range(k) if ids[i, j] >= 0)
        return s
    g = moe.route_grad(l, ids, dw, renorm)
    h = 1e-5
    for i in range(5):
        for e in range(7):
            if l[i, e] == -np.inf:
                assert g[i, e] == 0.0
                continue
            a, b = l.copy(), l.copy()
            a[i, e] += h
            b[i, e] -= h
            # central differences: h^2 |f'''| / 6 + rounding 1e-16 / h
            assert abs((loss(a) - loss(b)) / (2 * h) - g[i, e]) < 1e-9


def test_exchange_gradients_against_differences():
    # both are linear (combine in rows and in weights): a difference is the
    # derivative up to rounding
    rng = np.random.default_rng(1)
    ids = np.array([[1, 0], [-1, 2], [2, 1], [-1, -1]])
    _, pos, _ = moe.sort(ids, 3)
    x, rows = rng.standard_normal((4, 6)), rng.standard_normal((8, 6))
    w, dy, dr = rng.random((4, 2)), rng.standard_normal((4, 6)), rng.standard_normal((8, 6))
    drows, dw, _ = moe.combine_grad(dy, rows, pos, w)
    base = np.sum(moe.combine(rows, pos, w)[0] * dy)
    for r in range(8):
        for c in range(6):
            p = rows.copy()
            p[r, c] += 1.0
            assert abs(np.sum(moe.combine(p, pos, w)[0] * dy) - base - drows[r, c]) < 1e-12
    for i in range(4):
        for j in range(2):
            p = w.copy()
            p[i, j] += 1.0
            assert abs(np.sum(moe.combine(rows, pos, p)[0] * dy) - base - dw[i, j]) < 1e-12
    dx = moe.combine(dr, pos)[0]
    base = np.sum(moe.dispatch(x, pos) * dr)
    for i in range(4):
        for c in range(6):
            p = x.copy()
            p[i, c] += 1.0
            assert abs(np.sum(moe.dispatch(p, pos) * dr) - base - dx[i, c]) < 1e-12


def test_clip_by_hand():
    norm, out = moe.grad_clip([np.array([3.0]), np.array([[4.0]])], 1.0, 0.0)
    assert norm == 5.0
    np.testing.assert_allclose([out[0][0], out[1][0, 0]], [0.6, 0.8])
    norm, out = moe.grad_clip([np.array([0.3, 0.4])], 1.0, 0.0)
    np.testing.assert_array_equal(out[0], [0.3, 0.4])
