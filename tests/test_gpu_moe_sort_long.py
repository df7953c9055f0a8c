"""The order of more slots than the scan over the chunks takes in one round
(512 chunks of 1024 slots), against a stable sort of the keys."""

import numpy as np
import pytest
import torch

from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,k,e", [(65536, 8, 64), (70000, 8, 64), (600001, 1, 1000), (140000, 8, 5), (75000, 32, 128)])
@pytest.mark.parametrize("kind", ["mixed", "one", "dropped"])
def test_long_sort(t, k, e, kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rng = np.random.default_rng([t, k, e])
    ids = rng.integers(0, e, t * k).astype(np.int32)
    if kind == "one":
        ids[:] = e // 2
    if kind == "dropped":
        ids[rng.random(t * k) < 0.3] = -1
        ids[rng.random(t * k) < 0.1] = e
    key = np.where((ids >= 0) & (ids < e), ids, e)
    src = np.argsort(key, kind="stable")
    pos = np.empty(t * k, np.int64)
    pos[src] = np.arange(t * k)
    offsets, p, s = av.averis_moe_sort(torch.from_numpy(ids.reshape(t, k)).cuda(), e)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(key, minlength=e + 1)[:e])]))
    assert np.array_equal(s.cpu().numpy(), src)
    assert np.array_equal(p.cpu().numpy().reshape(-1), np.where(key < e, pos, ~pos))
