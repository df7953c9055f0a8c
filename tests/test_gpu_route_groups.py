"""Routing by scores with a bias and groups of experts, and its gradient, on the
GPU against the float64 oracle.

The choice is determined (the oracle's scores and the kernel's fp64 ones differ
by 2^-50 at most, and no test has scores so near but equal ones).  Weights in
fp32: an exponent of at most 64 rounded once, exp, a division and 32 + 6
additions: 2^-17 relative, as for the plain router; the scale adds a rounding.
The gradient's differences: 2^-15 of their magnitudes, and half a step."""

import numpy as np
import pytest
import torch

from oracle import block
from tests.parity import BF16_REL
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

REL_W = 2.0 ** -17
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def strided(a, pad, lead=0):
    buf = torch.full((a.shape[0] * (a.shape[1] + pad) + lead,), 7.0, dtype=a.dtype, device="cuda")
    v = buf[lead:].as_strided(a.shape, (a.shape[1] + pad, 1), lead)
    v.copy_(a)
    return v


def check(l, k, bias=None, grad=True, lead=1, **kw):
    """l: logits on the CPU; against the oracle, gradient included."""
    n = l.double().numpy()
    lg = strided(l, 3, lead)
    bg = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = av.averis_moe_route_groups(lg, k, bias=bg, **kw)
    rid, rw = block.route_groups(n, k, bias, **kw)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    np.testing.assert_array_equal(ids, rid)
    np.testing.assert_array_equal(w[rid < 0], 0.0)
    np.testing.assert_array_equal(np.isnan(w), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert np.all(np.abs(w[ok] - rw[ok]) <= REL_W * rw[ok] + 1e-38)
    if not grad:
        return
    g = {key: kw[key] for key in ("score", "renorm", "scale") if key in kw}
    dw = np.random.default_rng(1).standard_normal(rid.shape).astype(np.float32)
    d = av.averis_moe_route_groups_grad(lg, torch.from_numpy(rid).cuda(), torch.from_numpy(dw).cuda(), **g)
    ref, mag = block.route_groups_grad(n, rid, dw, **g)
    assert d.dtype == l.dtype
    lim = 2.0 ** -15 * mag + np.abs(ref) * (BF16_REL if l.dtype == BF16 else 2.0 ** -24) + 1e-38
    assert np.all(np.abs(d.double().cpu().numpy() - ref) <= lim)
    again = av.averis_moe_route_groups_grad(lg, torch.from_numpy(rid).cuda(), torch.from_numpy(dw).cuda(), out=lg, **g)
    assert torch.equal(again, d)                             # in place


def logits_of(rng, t, e, dtype, masked):
    l = rng.standard_normal((t, e)).astype(np.float32) * 2.0
    if masked:
        l[rng.random((t, e)) < 0.4] = -np.inf
        l[rng.random(t) < 0.2] = -np.inf
        if t > 2:
            l[2, : e - 1] = -np.inf                          # a single open expert
    l[0] = np.round(l[0])                                    # equal ones
    return torch.from_numpy(l).to(dtype)


# tokens, experts, top-k, groups, groups that stay: every number of lanes a token; groups of
# whole lanes, of several, and that end inside one
CASES = [(1, 1, 1, 1, 1), (3, 8, 3, 2, 1), (65, 16, 4, 2, 1), (33, 32, 6, 4, 2), (70, 64, 8, 8, 4), (129, 64, 8, 16, 5),
         (20, 128, 6, 4, 4), (19, 256, 8, 8, 4), (9, 160, 6, 8, 3), (7, 300, 10, 12, 5), (5, 512, 8, 2, 1),
         (4, 520, 7, 13, 6), (3, 1024, 32, 64, 30), (5, 1000, 32, 8, 2), (40, 12, 2, 12, 3), (31, 40, 32, 5, 4),
         (6, 64, 32, 64, 40), (17, 21, 3, 7, 2)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("t,e,k,groups,keep", CASES)
def test_route(t, e, k, groups, keep, masked, dtype):
    rng = np.random.default_rng([t, e, k, masked])
    l = logits_of(rng, t, e, dtype, masked)
    bias = (0.2 * rng.standard_normal(e)).astype(np.float32)
    steps = np.round(bias, 3).astype(np.float32)
    zero = np.zeros(e, np.float32)
    for i, (b, score, top, renorm) in enumerate([
            (None, "sigmoid", 2, True), (bias, "sigmoid", 2, True), (steps, "softmax", 1, False),
            (None, "softmax", 1, True), (None, "softmax", 1, False), (zero, "sigmoid", 1, False),
            (bias, "sigmoid", 1, False), (None, "softmax", 2, False)]):
        check(l, k, b, score=score, groups=groups, topk_groups=keep, group_top=top, renorm=renorm,
              scale=(1.0, 2.5)[i % 2], lead=i % 3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_groups(dtype):
    """All groups stay: the same as one group, and as the plain router without a bias."""
    rng = np.random.default_rng(3)
    l = logits_of(rng, 200, 64, dtype, True).cuda()
    b = torch.from_numpy(rng.standard_normal(64).astype(np.float32)).cuda()
    for kw in (dict(bias=b), dict(bias=None), dict(bias=b, score="softmax")):
        one = av.averis_moe_route_groups(l, 6, **kw)
        for extra in (dict(groups=8), dict(groups=8, topk_groups=8), dict(groups=16, group_top=1)):
            got = av.averis_moe_route_groups(l, 6, **extra, **kw)
            assert torch.equal(got[0], one[0]) and torch.equal(got[1], one[1])
    ids, _ = av.averis_moe_route(l, 6)
    assert torch.equal(av.averis_moe_route_groups(l, 6, score="softmax")[0], ids)
    assert torch.equal(av.averis_moe_route_groups(l, 6, score="sigmoid")[0], ids)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["near", "equal", "equal pairs", "tiny", "shifted"])
@pytest.mark.parametrize("t,e,k,groups,keep", [(130, 8, 3, 2, 1), (67, 64, 8, 8, 4), (33, 160, 6, 8, 3), (9, 600, 8, 4, 2)])
def test_scores_that_fp32_cannot_tell_apart(t, e, k, groups, keep, kind, dtype):
    """Scores that differ by less than an fp32 step, or not at all."""
    rng = np.random.default_rng([t, e, len(kind)])
    if kind == "near":                                       # logits a few steps apart, far out where the slope is small
        l = 6.0 + rng.integers(0, 20, (t, e)) * (2.0 ** -21 if dtype == F32 else 2.0 ** -5)
    elif kind == "equal":
        l = np.zeros((t, e))
    elif kind == "equal pairs":
        l = rng.integers(-1, 2, (t, e)) * 0.5
    elif kind == "tiny":                                     # sigmoids and softmaxes below fp32's numbers
        l = -95.0 - 0.25 * rng.integers(0, 60, (t, e))
    else:                                                    # a bias that lifts small differences
        l = -12.0 + 0.01 * rng.standard_normal((t, e))
    l = torch.from_numpy(l.astype(np.float32)).to(dtype)
    bias = (0.5 * rng.integers(-1, 2, e)).astype(np.float32)
    for b, score, top in ((bias, "sigmoid", 2), (None, "sigmoid", 2), (bias, "softmax", 1), (None, "softmax", 2),
                          (None, "softmax", 1)):
        # the gradient's tolerance is of ordinary logits
        check(l, k, b, grad=False, score=score, groups=groups, topk_groups=keep, group_top=top, renorm=kind != "tiny")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["finite", "nan", "inf", "bias"])
@pytest.mark.parametrize("t,e,k,groups,keep", [(67, 4, 1, 2, 1), (200, 8, 4, 4, 2), (130, 40, 6, 5, 2), (70, 64, 8, 8, 4),
                                               (65, 200, 7, 10, 3), (20, 600, 5, 3, 2)])
def test_special_values(t, e, k, groups, keep, kind, dtype):
    rng = np.random.default_rng([t, e, len(kind)])
    info = torch.finfo(dtype)
    pool = [0.0, -0.0, info.min, info.max, 1.0, 1.0, -2.0, 3.0, -np.inf, -np.inf, -np.inf]
    pool += [np.nan, -np.nan] if kind == "nan" else []
    pool += [np.inf, np.inf] if kind == "inf" else []
    l = rng.choice(np.array(pool), (t, e))
    for i in range(0, t, 3):                                 # rows with few open experts
        l[i, rng.permutation(e)[:max(e - 2, 0)]] = -np.inf
    l[1] = -np.inf
    l[4] = 0.5                                               # all equal
    with np.errstate(over="ignore", invalid="ignore"):
        l = torch.from_numpy(l.astype(np.float32)).to(dtype)
    bias = (0.1 * rng.standard_normal(e)).astype(np.float32)
    if kind == "bias":
        bias[rng.random(e) < 0.3] = -np.inf
        bias[rng.random(e) < 0.1] = np.inf
        bias[rng.random(e) < 0.1] = np.nan
    for b in (bias, None):
        for score, top, renorm in (("sigmoid", 2, True), ("sigmoid", 1, False), ("softmax", 2, True), ("softmax", 1, False)):
            check(l, k, b, grad=False, score=score, groups=groups, topk_groups=keep, group_top=top, renorm=renorm)
            check(l, k, b, grad=False, score=score, groups=groups, group_top=top, renorm=renorm)


def test_gradient_against_differences():
    """d sum(dw w) along a direction, by differences of the GPU's own weights:
    a step of 2^-6 leaves a truncation error of h^2 |f'''| / 6 < 5e-5 |dw| and
    rounding of 2^-17 / h < 5e-4 of the weights."""
    rng = np.random.default_rng(3)
    l = torch.from_numpy(rng.standard_normal((64, 16)).astype(np.float32)).cuda()
    l += 4.0 * (torch.arange(16, device="cuda") % 2) - 2.0   # the choice stays put under the step
    v = torch.from_numpy(rng.standard_normal((64, 16)).astype(np.float32)).cuda().clamp(-1, 1)
    dw = torch.from_numpy(rng.standard_normal((64, 8)).astype(np.float32)).cuda()
    for kw in (dict(score=s, renorm=r) for s in ("sigmoid", "softmax") for r in (True, False)):
        def weights(x):
            ids, w = av.averis_moe_route_groups(x, 8, **kw)
            return ids, torch.zeros(64, 16, device="cuda").scatter_(1, ids.long(), w)
        ids, _ = weights(l)
        h = 2.0 ** -6
        up, down = weights(l + h * v), weights(l - h * v)
        assert all(torch.equal(torch.sort(x[0], 1).values, torch.sort(ids, 1).values) for x in (up, down))
        full = torch.zeros(64, 16, device="cuda").scatter_(1, ids.long(), dw)
        slope = (full * (up[1] - down[1])).sum(1) / (2 * h)
        d = av.averis_moe_route_groups_grad(l, ids, dw, **kw)
        assert ((d * v).sum(1) - slope).abs().max() < 1e-3 * dw.abs().sum(1).max()


def test_ids_outside_the_experts_contribute_nothing():
    l = torch.randn(5, 12, device="cuda")
    ids = torch.tensor([[0, 12], [-1, -7], [3, 1 << 30], [11, -2147483648], [2, 5]], dtype=torch.int32, device="cuda")
    dw = torch.ones(5, 2, device="cuda")
    d = av.averis_moe_route_groups_grad(l, ids, dw, renorm=False)
    s = torch.sigmoid(l.double())
    ref = torch.zeros(5, 12, dtype=torch.float64, device="cuda")
    for t, e in ((0, 0), (2, 3), (3, 11), (4, 2), (4, 5)):
        ref[t, e] = s[t, e] * (1 - s[t, e])
    assert ((d.double() - ref).abs() <= 2.0 ** -20 * ref).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(dtype):
    l = torch.empty(0, 64, device="cuda", dtype=dtype)
    ids, w = av.averis_moe_route_groups(l, 8, groups=8, topk_groups=4)
    assert ids.shape == w.shape == (0, 8)
    assert av.averis_moe_route_groups_grad(l, ids, w).shape == (0, 64)


def test_more_tokens_than_one_launch_takes():
    """2^24 - 1 workgroups of 256 tokens of eight experts and fewer: the rest in another."""
    t = ((1 << 24) - 1) * 256 // 2 + 5                       # two lanes a token
    if torch.cuda.mem_get_info()[0] < t * 9 * 2 + t * 8 * 3:
        pytest.skip("not enough memory")
    t = min(t, (1 << 31) - 1)
    l = torch.zeros(t, 9, dtype=BF16, device="cuda")
    tail = torch.randn(300, 9).to(BF16)
    l[-300:] = tail.cuda()
    ids, w = av.averis_moe_route_groups(l, 1, groups=3, topk_groups=2)
    rid, rw = block.route_groups(tail.double().numpy(), 1, groups=3, topk_groups=2)
    np.testing.assert_array_equal(ids[-300:].cpu().numpy(), rid)
    assert (ids[:-300] == 0).all() and (w[:-300] == 1).all()
    d = av.averis_moe_route_groups_grad(l, ids, w, renorm=False, out=l)
    s = torch.sigmoid(tail.double())
    want = torch.zeros(300, 9, dtype=torch.float64)
    for i, e in enumerate(rid[:, 0]):
        want[i, e] = s[i, e] * (1 - s[i, e]) * float(rw[i, 0])
    assert ((d[-300:].double().cpu() - want).abs() <= 2.0 ** -8 * want + 1e-38).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_expert_alone(dtype, score):
    """Renormalised, the weight of a token's only expert is the scale, and its logit has no gradient: exactly."""
    for t, e, k in ((1000, 40, 1), (777, 256, 1), (500, 12, 4)):
        l = (6 * torch.randn(t, e, device="cuda")).to(dtype)
        if k > 1:   # one open expert
            l.masked_fill_(torch.arange(e, device="cuda") != torch.randint(0, e, (t, 1), device="cuda"), float("-inf"))
        bias = torch.randn(e, device="cuda")
        ids, w = av.averis_moe_route_groups(l, k, bias=bias, score=score, scale=2.5)
        assert (w[:, 0] == 2.5).all() and (ids[:, 0] >= 0).all() and (ids[:, 1:] == -1).all() and (w[:, 1:] == 0).all()
        d = av.averis_moe_route_groups_grad(l, ids, torch.randn(t, k, device="cuda"), score=score, scale=2.5)
        assert (d == 0).all()
