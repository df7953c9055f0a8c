"""Pins of oracle/block.py: hand-made cases, torch's own functions in float64,
and differences for every gradient."""

import numpy as np
import pytest
import torch

from oracle import block, moe


def test_rmsnorm_by_hand():
    rstd, y = block.rmsnorm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    assert rstd[0] == pytest.approx(np.sqrt(2.0) / 5.0)
    np.testing.assert_allclose(y[0], [3 * np.sqrt(2) / 5, 8 * np.sqrt(2) / 5])
    assert np.isnan(y[1]).all()
    rstd, y = block.rmsnorm(np.zeros((1, 3)), np.ones(3), 0.25)
    assert rstd[0] == 2.0 and (y == 0).all()


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(0)
    h, w, dy, v = rng.standard_normal((3, 5)), rng.standard_normal(5), rng.standard_normal((3, 5)), rng.standard_normal((3, 5))
    rstd, _ = block.rmsnorm(h, w, 1e-3)
    dh, dw = block.rmsnorm_grad(dy, h, w, rstd)
    f = lambda h, w: np.sum(dy * block.rmsnorm(h, w, 1e-3)[1])
    e = 1e-5
    assert np.sum(dh * v) == pytest.approx((f(h + e * v, w) - f(h - e * v, w)) / (2 * e), rel=1e-7)
    u = v[0]
    assert np.sum(dw * u) == pytest.approx((f(h, w + e * u) - f(h, w - e * u)) / (2 * e), rel=1e-7)


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_activations(name):
    z = np.linspace(-30.0, 30.0, 4001)[1::2]
    t = torch.from_numpy(z)
    ref = {"none": t, "relu": torch.relu(t), "silu": torch.nn.functional.silu(t),
           "gelu": torch.nn.functional.gelu(t, approximate="tanh")}[name]
    np.testing.assert_allclose(block.act(z, name), ref.numpy(), rtol=1e-12, atol=1e-15)
    e = 1e-6
    diff = (block.act(z + e, name) - block.act(z - e, name)) / (2 * e)
    np.testing.assert_allclose(block.act_slope(z, name), diff, atol=1e-8)


def test_one_group_of_softmax_is_the_plain_router():
    rng = np.random.default_rng(1)
    l = rng.standard_normal((20, 12)) * 3
    l[rng.random((20, 12)) < 0.4] = -np.inf
    l[3] = -np.inf
    for renorm in (True, False):
        ids, w = block.route_groups(l, 4, score="softmax", renorm=renorm)
        rid, rw = moe.route(l, 4, renorm)
        np.testing.assert_array_equal(ids, rid)
        np.testing.assert_allclose(w, rw, rtol=1e-12)
        dw = rng.standard_normal((20, 4))
        np.testing.assert_allclose(block.route_groups_grad(l, ids, dw, "softmax", renorm)[0],
                                   moe.route_grad(l, rid, dw, renorm), atol=1e-14)


def test_groups_by_hand():
    # four groups of two; sigmoid(0) = 1/2 everywhere, so the bias alone decides
    b = np.array([0.1, 0.1, 0.3, -0.2, 0.0, 0.25, 0.2, 0.0])
    z = np.zeros((1, 8))
    # sums 0.2, 0.1, 0.25, 0.2: groups 2 and (equal, the lower) 0
    ids, w = block.route_groups(z, 3, bias=b, groups=4, topk_groups=2)
    assert ids.tolist() == [[5, 0, 1]]
    np.testing.assert_allclose(w, 1 / 3)
    # largest alone 0.1, 0.3, 0.25, 0.2: groups 1 and 2
    ids, w = block.route_groups(z, 3, bias=b, groups=4, topk_groups=2, group_top=1, renorm=False, scale=3.0)
    assert ids.tolist() == [[2, 5, 4]]
    np.testing.assert_allclose(w, 1.5)
    # a group with one open expert counts with that one; closed groups never stay
    l = z.copy()
    l[0, [2, 4, 5, 6, 7]] = -np.inf
    ids, w = block.route_groups(l, 4, bias=b, groups=4, topk_groups=3)
    assert ids.tolist() == [[0, 1, 3, -1]] and w[0, 3] == 0
    ids, _ = block.route_groups(z, 2, bias=np.where(np.arange(8) < 6, -np.inf, 0.0), groups=4, topk_groups=1)
    assert ids.tolist() == [[6, 7]]
    l = z.copy()
    l[0, 6] = np.nan
    ids, w = block.route_groups(l, 2, bias=b, groups=4, topk_groups=1)
    assert ids.tolist() == [[6, 7]] and np.isnan(w).all()


def test_weights_whose_scores_are_all_tiny():
    ids, w = block.route_groups(np.array([[-2000.0, -2001.0, -2000.0]]), 2)
    assert ids.tolist() == [[0, 2]]
    np.testing.assert_allclose(w, 0.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    l = rng.standard_normal((6, 8)) + 3.0 * (np.arange(8) % 2)
    v, dw = rng.standard_normal((6, 8)), rng.standard_normal((6, 4))
    kw = dict(score=score, renorm=renorm, scale=1.7)
    ids, _ = block.route_groups(l, 4, groups=2, topk_groups=2, **kw)
    d, mag = block.route_groups_grad(l, ids, dw, **kw)
    e = 1e-5
    f = lambda x: np.sum(dw * block.route_groups(x, 4, groups=2, topk_groups=2, **kw)[1])
    assert (block.route_groups(l + e * v, 4, groups=2, **kw)[0] == ids).all()
    assert np.sum(d * v) == pytest.approx((f(l + e * v) - f(l - e * v)) / (2 * e), rel=1e-6)
    assert (np.abs(d) <= mag * (1 + 1e-12)).all()
