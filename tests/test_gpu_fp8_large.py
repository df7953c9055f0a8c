"""fp8 quantization of more rows than one launch has threads for (a grid has
fewer than 2^32 of them, and a wavefront takes four rows)."""

import pytest
import torch

from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu


def test_rows_past_one_launch():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rows = (1 << 28) + 100
    # 2^e: the scale 2^(e - 8) and the code of 256
    e = (torch.arange(rows, device="cuda") % 7).to(torch.uint8)
    a = torch.exp2(e.float()).to(torch.bfloat16).reshape(-1, 1)
    q = av.averis_fp8_quant(a)
    ok = [bool((q.codes[:, 0] == 0x78).all()), bool((q.scales[:, 0] == e + (127 - 8)).all())]
    ok += [bool((q.codes[part, 1:] == 0).all()) for part in (slice(None, 1000), slice(-1000, None))]
    del a, q, e
    torch.cuda.empty_cache()
    assert all(ok), ok
