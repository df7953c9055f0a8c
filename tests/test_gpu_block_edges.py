"""Calls of the operators around a block's linears at the ends of what they take:
more rows than one launch has, sums in place of the residual, weights and logits
that are not finite, against the oracle and against the calls they are made of."""

import numpy as np
import pytest
import torch

from oracle import block
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def same_fp8(a, b):
    kb = -(-a.cols // 128)
    return torch.equal(a.codes, b.codes) and torch.equal(a.scales[:, :kb], b.scales[:, :kb])


def test_norm_of_more_rows_than_one_launch_takes():
    """2^22 workgroups of four rows: the rest in another.  rstd and y as for the rows alone."""
    rows = (1 << 24) + 5
    x = torch.empty(rows, 8, dtype=BF16, device="cuda").normal_()
    w = torch.rand(8, device="cuda") + 0.5
    h, rstd, y, _, _ = av.averis_rmsnorm(x, w, y=True, fp8=False)
    for a, b in ((0, 100), ((1 << 24) - 50, rows)):
        _, f, part, _, _ = av.averis_rmsnorm(x[a:b].contiguous(), w, y=True, fp8=False)
        assert torch.equal(rstd[a:b], f) and torch.equal(y[a:b], part)
    dh, dw = av.averis_rmsnorm_grad(y, h, w, rstd)
    part, _ = av.averis_rmsnorm_grad(y[-50:].contiguous(), h[-50:].contiguous(), w, rstd[-50:].contiguous())
    assert torch.equal(dh[-50:], part)
    ref = (y.double() * h.double() * rstd.double()[:, None]).sum(0)
    mag = (y.double() * h.double() * rstd.double()[:, None]).abs().sum(0)
    assert ((dw.double() - ref).abs() <= (rows / 4096 + 90) * U * mag).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [100, 2048, 9000])
def test_sum_in_place_of_the_residual(cols, dtype):
    x, r = torch.randn(37, cols, device="cuda").to(dtype), torch.randn(37, cols, device="cuda").to(dtype)
    w = torch.rand(cols, device="cuda")
    want = av.averis_rmsnorm(x, w, residual=r, y=True, transposed=True)
    into = r.clone()
    got = av.averis_rmsnorm(x, w, residual=into, out=into, y=True, transposed=True)
    assert got[0] is into
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))
    assert same_fp8(want[3], got[3]) and same_fp8(want[4], got[4])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weights_that_are_not_finite(dtype):
    """The codes of both copies are those of y, in columns of infinities and NaN and beside them."""
    x = torch.randn(130, 300, device="cuda").to(dtype)
    x[5, 7] = 0.0
    w = torch.ones(300, device="cuda")
    w[7], w[140], w[299] = float("inf"), float("nan"), float("-inf")
    _, _, y, q, qt = av.averis_rmsnorm(x, w, y=True, transposed=True)
    assert torch.isnan(y[5, 7]) and torch.isinf(y[6, 7]) and torch.isnan(y[:, 140]).all()
    plain, plain_t = av.averis_fp8_quant(y, transposed=True)
    assert same_fp8(q, plain) and same_fp8(qt, plain_t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
def test_softmax_of_a_nan(groups, keep, dtype):
    """Every score is NaN: by the logits, where they decide, the NaN is first; with a bias the lowest open indexes are."""
    l = torch.randn(3, 64)
    l[0, 10] = float("nan")
    l[1, [9, 40]] = float("nan")
    l[1, :9] = -float("inf")
    l = l.to(dtype)
    bias = np.linspace(-1, 1, 64).astype(np.float32)
    for b, top in ((None, 1), (bias, 1), (bias, 2), (None, 2)):
        want, wr = block.route_groups(l.double().numpy(), 6, b, score="softmax", groups=groups, topk_groups=keep,
                                      group_top=top)
        bg = None if b is None else torch.from_numpy(b).cuda()
        for i in range(3):
            ids, w = av.averis_moe_route_groups(l[i:i + 1].cuda(), 6, bias=bg, score="softmax", groups=groups,
                                                topk_groups=keep, group_top=top)
            np.testing.assert_array_equal(ids.cpu().numpy(), want[i:i + 1])
            np.testing.assert_array_equal(np.isnan(w.cpu().numpy()), np.isnan(wr[i:i + 1]))
