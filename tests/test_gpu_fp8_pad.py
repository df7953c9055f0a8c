"""The pad of fp8 codes (past the columns, to whole blocks of 128) is 0 also
where the last block holds a value that is not finite."""

import numpy as np
import pytest
import torch

from oracle import fp8
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def check(q, codes, scales):
    got, kb = q.codes.cpu().numpy(), -(-q.cols // 128)
    np.testing.assert_array_equal(got[:, :q.cols], codes)
    np.testing.assert_array_equal(got[:, q.cols:], 0)
    np.testing.assert_array_equal(q.scales.cpu().numpy()[:, :kb], scales)


def values(rows, cols, dtype):
    rng = np.random.default_rng([rows, cols])
    a = rng.standard_normal((rows, cols)).astype(np.float32)
    for i, v in enumerate((np.nan, np.inf, -np.inf)):
        a[-1 - i % rows, -1 - i % cols] = v
        a[i % rows, 0] = v
    return torch.from_numpy(a).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (70, 130), (130, 70), (133, 254), (257, 300), (128, 128)])
def test_pad(rows, cols, dtype):
    a = values(rows, cols, dtype)
    n = a.double().numpy()
    check(av.averis_fp8_quant(a.cuda()), *fp8.quantize(n))
    q, qt = av.averis_fp8_quant(a.cuda(), transposed=True)
    check(q, *fp8.quantize(n))
    check(qt, *fp8.quantize(n.T))
    wt, wd = av.averis_fp8_quant_weight(a.cuda())
    check(wd, *fp8.quantize(n, True))
    check(wt, *fp8.quantize(n.T, True))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offs", [[0, 5, 5, 140, 300], [0, 129, 130, 256, 256]])
def test_pad_of_segments(offs, dtype):
    """The rest of a segment's last run."""
    rows, cols = offs[-1], 150
    a = values(rows, cols, dtype)
    for r in offs[1:]:
        a[r - 1, ::3] = float("nan")
    n = a.double().numpy()
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    q, qt = av.averis_fp8_quant(a.cuda(), transposed=True, offsets=o)
    check(q, *fp8.quantize(n))
    got, starts = qt.codes.cpu().numpy(), fp8.seg_starts(np.array(offs))
    for s in range(len(offs) - 1):
        m = offs[s + 1] - offs[s]
        codes, _ = fp8.quantize(n[offs[s]:offs[s + 1]].T)
        part = got[:, starts[s]:starts[s + 1]]
        np.testing.assert_array_equal(part[:, :m], codes)
        np.testing.assert_array_equal(part[:, m:], 0)
