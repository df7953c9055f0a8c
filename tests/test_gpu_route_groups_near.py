"""Grouped routing where scores lie close together, a token a call.

In a batch one token whose scores only fp64 tells apart has its neighbours'
choices made in fp64 too; alone, each way of settling a near choice is seen.
The choice is determined by the float64 oracle: its scores and the kernel's
differ by 2^-50 at most, and no two here are so near but equal ones."""

import numpy as np
import pytest
import torch

from oracle import block
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def check_alone(l, k, bias=None, **kw):
    """Each token's experts in a call of its own, and all tokens' in one, against the oracle."""
    want, _ = block.route_groups(l.double().numpy(), k, bias, **kw)
    lg = l.cuda()
    bg = None if bias is None else torch.from_numpy(bias).cuda()
    got = torch.cat([av.averis_moe_route_groups(lg[i:i + 1], k, bias=bg, **kw)[0] for i in range(len(l))])
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    np.testing.assert_array_equal(av.averis_moe_route_groups(lg, k, bias=bg, **kw)[0].cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_larger_score_behind_equal_ones(dtype):
    """Three equal experts lead their group; the fourth is larger by less than fp32 tells."""
    l = torch.full((1, 16), -5.0)
    l[0, :4] = torch.tensor([18.0, 18.0, 18.0, 18.25])
    l[0, 8:11] = torch.tensor([18.125, 18.0, 18.0])
    check_alone(l.to(dtype), 3, groups=2, topk_groups=1)
    check_alone(l.to(dtype), 3, np.full(16, 0.25, np.float32), groups=2, topk_groups=1, group_top=1)
    if dtype == F32:
        u = 2.0 ** -23
        l[0, :4], l[0, 8:11] = torch.tensor([1.0, 1.0, 1.0, 1.0 + 2 * u]), torch.tensor([1.0 + u, 1.0, 1.0])
        for score in ("sigmoid", "softmax"):
            check_alone(l, 3, score=score, groups=2, topk_groups=1, group_top=1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_smaller_score_before_equal_ones(dtype):
    """The first of a group is smaller than those behind it by less than fp32 tells: it is none of the two that count."""
    l = torch.full((1, 10), 18.0)
    l[0, 0] = 17.875
    check_alone(l.to(dtype), 3, groups=2, topk_groups=1)
    check_alone(l.to(dtype), 3, np.full(10, 0.25, np.float32), groups=2, topk_groups=1)
    check_alone(l.to(dtype), 3, np.full(10, 0.25, np.float32), groups=2, topk_groups=1, group_top=1)
    wide = torch.full((1, 32), -float("inf"))               # a group on several lanes
    wide[0, [0, 9, 10, 15, 17, 31]] = 18.0
    wide[0, 0] = 17.875
    for many in (1, 3):
        check_alone(wide.to(dtype).repeat(1, many), 2, groups=2 * many, topk_groups=many)


NEAR = [(8, 3, 2, 1), (64, 8, 8, 4), (160, 6, 8, 3), (600, 8, 4, 2), (1000, 12, 8, 2)]


@pytest.mark.parametrize("e,k,groups,keep", NEAR)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_mostly_equal_scores(e, k, groups, keep, dtype):
    """Most experts of a token alike, a few larger by less than an fp32 step of the score."""
    rng = np.random.default_rng([e, k])
    few = lambda p: torch.from_numpy(rng.choice(3, size=(60, e), p=[1 - p, p / 2, p / 2]).astype(np.float32))
    equal = np.full(e, 0.25, np.float32)
    for p in (0.02, 0.2):
        n = few(p)
        high = (18.0 + 0.125 * n).to(dtype)                 # sigmoids of nearly 1
        low = (-30.0 + 0.125 * n).to(dtype)                 # of nearly 0, beside a bias
        for top in (1, 2):
            check_alone(high, k, groups=groups, topk_groups=keep, group_top=top)
            check_alone(high, k, equal, groups=groups, topk_groups=keep, group_top=top)
            check_alone(low, k, equal, groups=groups, topk_groups=keep, group_top=top)
            check_alone(low, k, equal, score="softmax", groups=groups, topk_groups=keep, group_top=top)
        if dtype == F32:                                    # by the logits themselves, a few steps apart
            check_alone(1.0 + 2.0 ** -23 * n, k, groups=groups, topk_groups=keep, group_top=1)
            check_alone(-1.0 + 2.0 ** -24 * n, k, score="softmax", groups=groups, topk_groups=keep, group_top=1)
            check_alone(1.0 + 2.0 ** -23 * n, k)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_group_scores_around_the_smallest_normal_number(dtype):
    """Sums of two scores of which fp32 has none, one or both: e^-87.34 is 2^-126."""
    l = torch.full((1, 8), -200.0)
    l[0, :2] = torch.tensor([-87.5, -87.5]) if dtype == BF16 else torch.tensor([-87.4, -87.4])
    l[0, 4] = -87.0 if dtype == BF16 else -87.3
    check_alone(l.to(dtype), 2, groups=2, topk_groups=1)
    three = torch.cat([torch.tensor([[0.0, -1.0, -300.0, -300.0]]), l], 1)   # the same below the largest logit
    check_alone(three.to(dtype), 4, score="softmax", groups=3, topk_groups=2, renorm=False)


@pytest.mark.parametrize("e,k,groups,keep", NEAR)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_around_the_smallest_normal_number(e, k, groups, keep, dtype):
    rng = np.random.default_rng([e, k, 1])
    step = 0.5 if dtype == BF16 else 2.0 ** -13
    n = rng.integers(-3 if dtype == BF16 else -6000, 2 if dtype == BF16 else 4000, (80, e))
    l = torch.from_numpy((-87.0 + step * n).astype(np.float32))
    l[::2][torch.from_numpy(rng.random((40, e)) < 0.8)] = -200.0
    check_alone(l.to(dtype), k, groups=groups, topk_groups=keep)
    top = l.clone()
    top[:, 0] = 0.0
    check_alone(top.to(dtype), k, score="softmax", groups=groups, topk_groups=keep)


def test_group_scores_of_large_parts():
    """Two large parts that cancel: their sum is known less well than those of the groups beside it."""
    l = torch.full((1, 12), -8.0)
    l[0, [0, 1, 4, 5, 8, 9]] = 0.0
    bias = np.full(12, -2000.0, np.float32)
    bias[[0, 1]], bias[[4, 5]], bias[[8, 9]] = (1000.30005, -1000.29999), (2.5e-5, 0.0), (-1.42e-4, 0.0)
    check_alone(l, 1, bias, groups=3, topk_groups=1)
    rng = np.random.default_rng(5)
    for _ in range(200):
        b = np.zeros(12, np.float32)
        b[0], b[1] = 1000.3 + 1e-3 * rng.random(), -1000.3
        b[4] = 2e-4 * rng.random()
        b[8] = b[4] - 1e-4 * (1 + rng.random())
        b[[2, 3, 6, 7, 10, 11]] = -2000.0
        order = rng.permutation(3)
        b, li = b.reshape(3, 4)[order].ravel(), l.reshape(3, 4)[torch.from_numpy(order)].reshape(1, 12)
        check_alone(li, 2, b, groups=3, topk_groups=1)


def test_group_scores_past_the_largest_number():
    """Sums of two that fp32 does not hold, on either side."""
    l = torch.zeros(1, 8)
    bias = np.array([3e38, 1e38, 0, 0, 3e38, 2e38, 0, 0], np.float32)
    check_alone(l, 1, bias, groups=2, topk_groups=1)
    bias = np.array([-1e38, -3e38, -3.3e38, -3.3e38, -1e38, -2.9e38, -3.3e38, -3.3e38], np.float32)
    check_alone(l, 1, bias, groups=2, topk_groups=1)
    bias = np.array([3e38, 1e38, 3e38, 2e38, 3e38, 1.5e38, 1.0, 2.0], np.float32)
    check_alone(l, 4, bias, groups=4, topk_groups=2)
