"""Router logits that are not ordinary numbers, in both types and many tokens a
wavefront: NaN, infinities, signed zeros, the type's lowest and largest values,
equal logits and masked experts, alone and mixed, against the oracle's order.

Weights: 2^-17 relative as for ordinary logits; NaN exactly where a chosen
logit's row has a NaN or +inf; 0 for every slot without an expert."""

import numpy as np
import pytest
import torch

from oracle import moe
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

REL_W = 2.0 ** -17
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def check(l, k):
    n = l.double().cpu().numpy()
    for renorm in (True, False):
        ids, w = av.averis_moe_route(l.cuda(), k, renorm=renorm)
        rid, rw = moe.route(n, k, renorm)
        ids, w = ids.cpu().numpy(), w.cpu().numpy()
        np.testing.assert_array_equal(ids, rid)
        np.testing.assert_array_equal(w[rid < 0], 0.0)
        np.testing.assert_array_equal(np.isnan(w), np.isnan(rw))
        ok = ~np.isnan(rw)
        assert np.all(np.abs(w[ok] - rw[ok]) <= REL_W * rw[ok] + 1e-45)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["finite", "nan", "inf", "all"])
@pytest.mark.parametrize("t,e,k", [(67, 4, 3), (200, 8, 8), (130, 40, 6), (70, 64, 8), (65, 200, 7), (40, 600, 5)])
def test_special_logits(t, e, k, kind, dtype):
    rng = np.random.default_rng([t, e, len(kind)])
    info = torch.finfo(dtype)
    pool = [0.0, -0.0, info.min, info.max, info.tiny, -info.tiny, 1.0, 1.0, -2.0, 3.0, -np.inf, -np.inf, -np.inf]
    pool += [np.nan, -np.nan] if kind in ("nan", "all") else []
    pool += [np.inf, np.inf] if kind in ("inf", "all") else []
    l = rng.choice(np.array(pool), (t, e))
    for i in range(0, t, 3):                       # rows with few open experts
        l[i, rng.permutation(e)[:max(e - 2, 0)]] = -np.inf
    l[1] = -np.inf
    l[4] = 0.5                                     # all equal
    if kind != "finite":                           # one, with too few open experts behind it
        l[5] = -np.inf
        l[5, e // 2] = np.inf if kind == "inf" else np.nan
    with np.errstate(over="ignore", invalid="ignore"):
        check(torch.from_numpy(l.astype(np.float32)).to(dtype), k)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_by_hand(dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    l = torch.tensor([[0.0, -0.0, -0.0, 0.0], [low, -inf, low, -inf], [1.0, nan, 2.0, -inf],
                      [inf, 1.0, inf, 0.0], [-nan, 1.0, nan, 0.0], [-inf, nan, -inf, -inf],
                      [-inf, -inf, inf, -inf], [-inf] * 4], device="cuda").to(dtype)
    ids, w = av.averis_moe_route(l, 3)
    assert ids.tolist() == [[0, 1, 2], [0, 2, -1], [1, 2, 0], [0, 2, 1], [0, 2, 1], [1, -1, -1], [2, -1, -1], [-1] * 3]
    w = w.cpu().numpy()
    np.testing.assert_allclose(w[0], 1 / 3, rtol=1e-6)
    np.testing.assert_array_equal(w[1], [0.5, 0.5, 0.0])
    assert np.isnan(w[2:5]).all() and np.isnan(w[5:7, 0]).all()
    np.testing.assert_array_equal(w[5:7, 1:], 0.0)
    np.testing.assert_array_equal(w[7], 0.0)
