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


def small(*shape):
    g = torch.Generator(device="cuda").manual_seed(shape[0])
    return torch.randint(-4, 5, shape, dtype=torch.int8, device="cuda", generator=g).to(torch.bfloat16)


def test_products_of_many_rows():
    """More than 65535 tiles of 256 rows; small integers, exact."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m, n = (1 << 24) + 1000, 8
    a, b = small(m, 1), small(n, 1)
    qa = av.averis_fp8_quant(a)
    c = av.averis_fp8_gemm(qa, av.averis_fp8_quant(b), torch.float32)
    ok = [bool((c == a.float() @ b.float().t()).all())]
    cuts, w = [0, 5, (1 << 24) + 900, m], small(3 * n, 1)
    c = av.averis_fp8_gemm(qa, av.averis_fp8_quant(w), torch.float32, offsets=torch.tensor(cuts, device="cuda"))
    for s in range(3):
        ok.append(bool((c[cuts[s]:cuts[s + 1]] == a[cuts[s]:cuts[s + 1]].float() @ w[s * n:(s + 1) * n].float().t()).all()))
    del c, qa
    x, d = small(2, m), small(2, n)
    _, xt = av.averis_fp8_quant(x, transposed=True, plain=False)
    _, dt = av.averis_fp8_quant(d, transposed=True, plain=False)
    g = av.averis_fp8_gemm_wgrad(xt, dt, torch.float32)
    ok.append(bool((g == x[0].float()[:, None] * d[0].float() + x[1].float()[:, None] * d[1].float()).all()))
    del g, xt
    torch.cuda.empty_cache()
    assert all(ok), ok
