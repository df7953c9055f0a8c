"""The fp8 product with bias, activation and residual in its epilogue, on the GPU.

The sums are averis_fp8_gemm's, so z = sum + bias has to be that product in fp32
plus the bias, bit for bit, and with no activation or relu, c too.  The smooth
activations z s: the sigmoid's argument carries at most 5 x 2^-24 of itself,
exp2 and the reciprocal an ulp each, so s is off by at most 5 x 2^-24: under
2^-20 |z|, and half a step of the output's type."""

import numpy as np
import pytest
import torch

from oracle import block
from tests.parity import BF16_REL
from tests.test_gpu_fp8 import GEMMS, LARGE, exact_fp8
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def operands(rng, m, n, k):
    a, b = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(BF16) for s in ((m, k), (n, k)))
    return av.averis_fp8_quant(a), av.averis_fp8_quant(b)


def smooth(c, z, act, res):
    """c against act(z) + res in float64, z in fp32."""
    zn = z.double()
    ref = {"silu": zn * torch.sigmoid(zn),
           "gelu": 0.5 * zn * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (zn + 0.044715 * zn ** 3)))}[act]
    lim = 2.0 ** -20 * zn.abs()
    if res is not None:
        ref = ref + res.double()
        lim = lim + U * ref.abs()
    lim = lim + (BF16_REL if c.dtype == BF16 else U) * ref.abs() + 1e-38
    assert ((c.double() - ref).abs() <= lim).all()


def full(rows, cols, dtype, value):
    """(the buffer, a rows x cols part of it at an odd place)."""
    buf = torch.full((rows + 2, cols + 5), value, dtype=dtype, device="cuda")
    return buf, buf[1:1 + rows, 3:3 + cols]


@pytest.mark.parametrize("m,n,k", GEMMS + [(2000, 2000, 256), (700, 1030, 9000)])
def test_epilogue(m, n, k):
    rng = np.random.default_rng([m, n, k])
    a, b = operands(rng, m, n, k)
    plain = av.averis_fp8_gemm(a, b, F32)
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32) * k ** 0.5).cuda()
    for dt in (F32, BF16):
        res = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda().to(dt)
        for use, bv, rv in (("none", bias, res), ("relu", bias.to(BF16), None), ("silu", bias, res), ("gelu", None, res),
                            ("gelu", bias, None)):
            z32 = plain if bv is None else plain + bv.float()
            c, z = av.averis_fp8_gemm_act(a, b, bias=bv, act=use, residual=rv, save=True, out_dtype=dt)
            assert c.dtype == dt and torch.equal(z, z32.to(dt))
            if use in ("none", "relu"):
                y = z32 if use == "none" else z32.clamp(min=0.0)
                assert torch.equal(c, (y if rv is None else y + rv.float()).to(dt))
            else:
                smooth(c, z32, use, rv)
            assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bv, act=use, residual=rv, out_dtype=dt), c)
            # any strides and places; the residual in place
            buf, out = full(m, n, dt, 9.0)
            rs = None
            if rv is not None:
                rs = full(m, n, dt, 4.0)[1]
                rs.copy_(rv)
            assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bv, act=use, residual=rs, out=out), c)
            out.fill_(9.0)
            assert (buf == 9.0).all()
            if rs is not None:
                assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bv, act=use, residual=rs, out=rs), c)


# columns in whole 16-byte pieces, which the large tile's epilogue is for
WHOLE = [(3001, 3008, 3790), (12001, 2216, 800), (9000, 5008, 260), (16384, 1032, 2048), (1001, 3008, 16300)]


@pytest.mark.parametrize("m,n,k", LARGE + WHOLE)
def test_large_products_are_exact(m, n, k):
    """Both tile sizes, several tiles a workgroup and split sums, of small integers."""
    rng = np.random.default_rng([m, n, k, 2])
    a, va = exact_fp8(rng, m, k)
    b, vb = exact_fp8(rng, n, k)
    z = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda().t()
    bias = torch.from_numpy(rng.integers(-50, 50, n).astype(np.float32)).cuda()
    z = z + bias.double()
    for dt in (F32, BF16):
        res = torch.randint(-50, 50, (m, n), device="cuda").to(dt)
        c, s = av.averis_fp8_gemm_act(a, b, bias=bias, act="relu", residual=res, save=True, out_dtype=dt)
        assert torch.equal(s, z.to(dt))
        assert torch.equal(c, (z.clamp(min=0.0) + res.double()).to(dt))
        buf, out = full(m, n, dt, 9.0)
        assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bias, act="relu", residual=res, out=out), c)
        out.fill_(9.0)
        assert (buf == 9.0).all()
        # rows that start at whole pieces and end before the next one does; in place; without each part
        wide, rw = (torch.full((m + 1, n + 16), v, dtype=dt, device="cuda") for v in (9.0, 4.0))
        rw[:m, 8:8 + n] = res
        part = wide[:m, 8:8 + n]
        assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bias, act="relu", residual=rw[:m, 8:8 + n], out=part), c)
        part.fill_(9.0)
        assert (wide == 9.0).all()
        own = rw[:m, 8:8 + n]
        assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bias, act="relu", residual=own, out=own), c)
        assert (rw[:m, :8] == 4.0).all() and (rw[:m, 8 + n:] == 4.0).all() and (rw[m:] == 4.0).all()
        assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bias, out_dtype=dt), z.to(dt))
        assert torch.equal(av.averis_fp8_gemm_act(a, b, out_dtype=dt), av.averis_fp8_gemm(a, b, dt))
        smooth(av.averis_fp8_gemm_act(a, b, bias=bias, act="gelu", residual=res, out_dtype=dt), z.float(), "gelu", res)
        smooth(av.averis_fp8_gemm_act(a, b, bias=bias, act="silu", out_dtype=dt), z.float(), "silu", None)


@pytest.mark.parametrize("k,n", [(200, 96), (640, 300), (2100, 1031), (2100, 2104)])
@pytest.mark.parametrize("offs", [[0, 5], [0, 0, 3, 3, 70, 90], [0, 256, 256, 900, 1500, 1500], [0, 300, 310, 1400],
                                  [0, 1, 1, 2500, 2756, 8000, 9000]])
def test_segments_are_exact(offs, k, n):
    rng = np.random.default_rng(offs + [k])
    nseg, rows = len(offs) - 1, offs[-1] + 3                # three rows in no segment
    a, va = exact_fp8(rng, rows, k)
    b, vb = exact_fp8(rng, nseg * n, k)
    va, vb = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    bias = torch.from_numpy(rng.integers(-50, 50, (nseg, n)).astype(np.float32)).cuda()
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    z = torch.cat([va[offs[s]:offs[s + 1]] @ vb[s * n:(s + 1) * n].t() + bias[s].double() for s in range(nseg)])
    end = offs[-1]
    for dt in (F32, BF16):
        res = torch.randint(-50, 50, (rows, n), device="cuda").to(dt)
        for bv in (bias, bias.to(BF16)):
            c = torch.full((rows, n), 7.0, dtype=dt, device="cuda")
            _, s = av.averis_fp8_gemm_act(a, b, bias=bv, act="relu", residual=res, save=True, offsets=o, out=c)
            assert torch.equal(s[:end], z.to(dt))
            assert torch.equal(c[:end], (z.clamp(min=0.0) + res[:end].double()).to(dt))
            assert (c[end:] == 7).all()
        c, s = av.averis_fp8_gemm_act(a, b, bias=bias, act="gelu", save=True, offsets=o, out_dtype=dt)
        smooth(c[:end], z.float(), "gelu", None)


def test_many_segments():
    rng = np.random.default_rng(8)
    nseg, rows, k, n = 200, 600, 72, 40
    offs = [0] + sorted(int(v) for v in rng.integers(0, rows + 1, nseg - 1)) + [rows]
    a, va = exact_fp8(rng, rows, k)
    b, vb = exact_fp8(rng, nseg * n, k)
    bias = rng.integers(-50, 50, (nseg, n)).astype(np.float32)
    c = av.averis_fp8_gemm_act(a, b, bias=torch.from_numpy(bias).cuda(), offsets=torch.tensor(offs, device="cuda"),
                               out_dtype=F32)
    seg = np.searchsorted(np.array(offs[1:]), np.arange(rows), side="right")
    ref = np.einsum("ri,roi->ro", va, vb.reshape(nseg, n, k)[seg]) + bias[seg]
    np.testing.assert_array_equal(c.cpu().numpy(), ref)


def test_special_values():
    """NaN and infinities of the bias pass as the formulas have them."""
    inf, nan = float("inf"), float("nan")
    a, _ = exact_fp8(np.random.default_rng(0), 40, 128)
    b, _ = exact_fp8(np.random.default_rng(1), 300, 128)
    bias = torch.zeros(300, device="cuda")
    bias[:6] = torch.tensor([nan, inf, -inf, 1e30, -1e30, 3e38])
    for m in (40, 3):                                       # the tiled and the few-rows kernel
        q = av.FP8(a.codes[:m].contiguous(), a.scales[:m].contiguous(), m, 128)
        for act, want in (("none", [nan, inf, -inf, 1e30, -1e30, 3e38]), ("relu", [nan, inf, 0, 1e30, 0, 3e38]),
                          ("silu", [nan, inf, nan, 1e30, 0, 3e38]), ("gelu", [nan, inf, nan, 1e30, 0, 3e38])):
            c = av.averis_fp8_gemm_act(q, b, bias=bias, act=act, out_dtype=F32)
            np.testing.assert_allclose(c[:, :6].cpu().numpy(), np.tile(np.float32(want), (m, 1)), rtol=1e-5)
            assert torch.isfinite(c[:, 6:]).all()


def test_no_rows():
    b, _ = exact_fp8(np.random.default_rng(1), 300, 128)
    c, z = av.averis_fp8_gemm_act(av.FP8.empty(0, 128), b, act="gelu", save=True, bias=torch.zeros(300, device="cuda"))
    assert c.shape == z.shape == (0, 300)


def test_offsets_past_32_bits():
    rows, n = 70001, 40000
    small = lambda *s: torch.randint(-4, 5, s, dtype=torch.int8, device="cuda").to(BF16)
    x, y = small(rows, 128), small(n, 128)
    bias = torch.randint(-9, 9, (n,), device="cuda").float()
    res = torch.zeros(rows, n, dtype=F32, device="cuda")    # 11 GB
    some = [0, 255, 26843, 53687, rows - 1]
    res[some] = 5.0
    c = av.averis_fp8_gemm_act(av.averis_fp8_quant(x), av.averis_fp8_quant(y), bias=bias, act="relu", residual=res,
                               out=res)
    ref = (x[some].double() @ y.double().t() + bias.double()).clamp(min=0.0) + 5.0
    assert torch.equal(c[some].double(), ref)


@pytest.mark.parametrize("offs", [None, [0, 900, 900, 2000, 4096]])
def test_columns_in_half_a_lane(offs):
    """fp32 rows of whole 16-byte pieces, four columns past a multiple of eight: nothing is read or written
    past a row's end, whichever tile is taken."""
    m, n, k = 4096, 4092, 640
    nseg = 1 if offs is None else len(offs) - 1
    rng = np.random.default_rng(n)
    a, b = operands(rng, m, nseg * n, k)
    o = None if offs is None else torch.tensor(offs, dtype=torch.int64, device="cuda")
    bias = torch.randn(n if offs is None else (nseg, n), device="cuda")
    res = torch.randn(m, n, device="cuda")
    z = av.averis_fp8_gemm(a, b, F32, offsets=o)
    z = z + bias if offs is None else torch.cat([z[p:q] + bias[s] for s, (p, q) in enumerate(zip(offs, offs[1:]))])
    buf = torch.full((m + 1, n), 9.0, device="cuda")
    c, kept = av.averis_fp8_gemm_act(a, b, bias=bias, act="relu", residual=res, save=True, offsets=o, out=buf[:m])
    assert torch.equal(kept, z) and torch.equal(c, z.clamp(min=0.0) + res)
    assert (buf[m:] == 9.0).all()
    assert torch.equal(av.averis_fp8_gemm_act(a, b, bias=bias, offsets=o, out_dtype=F32), z)
