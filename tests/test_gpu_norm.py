"""The norm with the residual's addition and its gradient on the GPU against the
float64 oracle.

Tolerances.  rstd: an fp64 result rounded to fp32 (2^-24 relative, and 2^-40 for
fp64's own errors).  y: two fp32 products of a rounded factor, 3 x 2^-24, and
half a step of the type.  The codes are determined by y.  dh = f (t - v c) + e
with t = dy w, v = h f, c the mean of t v: t, v, their product and at most 32
fused additions a lane, 9 across a row and the mean's factor, under 60 x 2^-24
of mean |t v|; the rest 8 x 2^-24 of f |t| and 4 of |e|.  dweight: at most
(rows / 512 + 1) additions in a wavefront, 4 in a workgroup and 1024 / 16 + 16
at the end, of products with 3 roundings."""

import numpy as np
import pytest
import torch

from oracle import block, fp8
from tests.parity import BF16_REL
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def half(ref, dtype):
    return np.abs(ref) * (BF16_REL if dtype == BF16 else U) + 1e-38


def strided(a, pad, lead=0):
    """a in a buffer whose rows are `pad` elements longer, `lead` elements in."""
    buf = torch.full((a.shape[0] * (a.shape[1] + pad) + lead,), 7.0, dtype=a.dtype, device="cuda")
    v = buf[lead:].as_strided(a.shape, (a.shape[1] + pad, 1), lead)
    v.copy_(a)
    return v


def randn(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32))


def num(t):
    return t.double().cpu().numpy()


def same_fp8(a, b):
    kb = -(-a.cols // 128)
    return torch.equal(a.codes, b.codes) and torch.equal(a.scales[:, :kb], b.scales[:, :kb])


# every number of wavefronts a row and pieces a lane, and rows that end inside a piece
SHAPES = [(1, 1), (1, 7), (5, 8), (3, 129), (130, 512), (129, 520), (16, 1000), (257, 1024), (33, 2048), (7, 2049),
          (1000, 640), (5, 4096), (6, 4099), (3, 8192), (4, 8200), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_and_gradient(rows, cols, dtype):
    rng = np.random.default_rng([rows, cols])
    x, r = randn(rng, rows, cols).to(dtype), randn(rng, rows, cols, scale=3.0).to(dtype)
    x *= torch.from_numpy(np.exp(3 * rng.standard_normal((rows, 1)))).to(dtype)
    wdt = F32 if cols % 2 else BF16
    w = (1.0 + 0.3 * randn(rng, cols)).to(wdt)
    wg = w.cuda()
    for res, pad, lead in ((None, 0, 0), (r, 0, 0), (r, 3, 1)):
        xg = strided(x, pad, lead)
        rg = strided(res, pad + 2, lead) if res is not None else None
        h, rstd, y, q, qt = av.averis_rmsnorm(xg, wg, eps=1e-5, residual=rg, y=True, transposed=True)
        hs = x if res is None else (x.float() + res.float()).to(dtype)
        assert torch.equal(h.cpu(), hs)
        ref_r, ref_y = block.rmsnorm(num(hs), num(w), 1e-5)
        assert np.all(np.abs(num(rstd) - ref_r) <= ref_r * (U + 2.0 ** -40))
        assert np.all(np.abs(num(y) - ref_y) <= 3 * U * np.abs(ref_y) + half(ref_y, dtype))
        plain, plain_t = av.averis_fp8_quant(y, transposed=True)
        assert same_fp8(q, plain) and same_fp8(qt, plain_t)
        codes, scales = fp8.quantize(num(y))
        np.testing.assert_array_equal(q.codes.cpu().numpy()[:, :cols], codes)
        np.testing.assert_array_equal(q.scales.cpu().numpy()[:, :scales.shape[1]], scales)
        # each output alone, and the sum in place
        into = strided(x, pad, lead) if res is not None else None
        h2, rstd2, none, q2, qt2 = av.averis_rmsnorm(into if into is not None else xg, wg, eps=1e-5, residual=rg,
                                                     out=into)
        assert none is None and qt2 is None and torch.equal(rstd2, rstd) and same_fp8(q2, q) and torch.equal(h2, h)
        _, _, none, q3, qt3 = av.averis_rmsnorm(xg, wg, eps=1e-5, residual=rg, fp8=False, transposed=True)
        assert none is None and q3 is None and same_fp8(qt3, qt)

        dy, dres = randn(rng, rows, cols).to(dtype), randn(rng, rows, cols).to(dtype)
        e = dres if res is not None else None
        eg = strided(dres, pad, lead) if res is not None else None
        dh, dw = av.averis_rmsnorm_grad(strided(dy, pad, lead), h, wg, rstd, dres=eg)
        f = num(rstd)[:, None]
        ref_h, ref_w = block.rmsnorm_grad(num(dy), num(hs), num(w), num(rstd))
        t, v = np.abs(num(dy) * num(w)), np.abs(num(hs) * f)
        lim = U * (f * (8 * t + 64 * v * np.mean(t * v, axis=1, keepdims=True)))
        if e is not None:
            ref_h = ref_h + num(e)
            lim = lim + 4 * U * (np.abs(num(e)) + np.abs(ref_h))
        assert dh.dtype == dtype and dw.dtype == F32
        assert np.all(np.abs(num(dh) - ref_h) <= lim + half(ref_h, dtype))
        n = rows / 512 + 1 + 4 + 80 + 3
        assert np.all(np.abs(num(dw) - ref_w) <= n * U * np.sum(np.abs(num(dy)) * v, axis=0) + 1e-38)
        for target in ("dy", "dres"):                       # in place, and the same bits
            if target == "dres" and e is None:
                continue
            a = strided(dy, pad, lead)
            b = strided(dres, pad, lead) if e is not None else None
            dh2, dw2 = av.averis_rmsnorm_grad(a, h, wg, rstd, dres=b, out=a if target == "dy" else b)
            assert torch.equal(dh2, dh) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_beyond_the_rows_is_written(dtype):
    x, w = torch.randn(5, 100, device="cuda").to(dtype), torch.ones(100, device="cuda")
    buf = torch.full((7, 110), 9.0, dtype=dtype, device="cuda")
    h, rstd, _, _, _ = av.averis_rmsnorm(x, w, residual=x, out=buf[1:6, 3:103])
    dbuf = torch.full((7, 110), 9.0, dtype=dtype, device="cuda")
    av.averis_rmsnorm_grad(x, h, w, rstd, out=dbuf[1:6, 3:103])
    for b in (buf, dbuf):
        b[1:6, 3:103] = 9.0
        assert (b == 9.0).all()


@pytest.mark.parametrize("cols", [64, 2048, 6000])
def test_no_rows(cols):
    x, w = torch.empty(0, cols, device="cuda", dtype=BF16), torch.ones(cols, device="cuda")
    h, rstd, y, q, qt = av.averis_rmsnorm(x, w, residual=x, y=True, transposed=True)
    assert h.shape == y.shape == (0, cols) and rstd.shape == (0,) and qt.codes.shape == (cols, 0)
    dh, dw = av.averis_rmsnorm_grad(x, h, w, rstd)
    assert dh.shape == (0, cols) and (dw == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_small_and_special_values(dtype):
    """Squares past fp32's range and below it, a row of zeros, and rows that are not finite."""
    rng = np.random.default_rng(7)
    x = randn(rng, 8, 300).to(dtype)
    x[0] *= 1e36
    x[1] *= 1e-36
    x[2] = 0.0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    w = torch.ones(300)
    h, rstd, y, q, qt = av.averis_rmsnorm(x.cuda(), w.cuda(), eps=1e-30, y=True, transposed=True)
    ref_r, ref_y = block.rmsnorm(num(x), num(w), 1e-30)
    with np.errstate(invalid="ignore"):
        ok = np.isfinite(ref_y)
        assert (np.isnan(num(y)) == np.isnan(ref_y)).all()
        assert np.all((np.abs(num(y) - ref_y) <= 3 * U * np.abs(ref_y) + half(ref_y, dtype))[ok])
    assert np.all((num(y)[2] == 0)) and (num(y)[3, :5] == 0).all()
    plain, plain_t = av.averis_fp8_quant(y, transposed=True)
    assert same_fp8(q, plain) and same_fp8(qt, plain_t)
    _, _, y, _, _ = av.averis_rmsnorm(torch.zeros(1, 4, device="cuda"), torch.ones(4, device="cuda"), eps=0.0, y=True)
    assert torch.isnan(y).all()
    _, dw = av.averis_rmsnorm_grad(torch.ones(8, 300, device="cuda").to(dtype), h, w.cuda(), rstd)
    assert torch.isnan(dw).all()                             # the row whose factor is NaN counts in every column


def test_gradient_against_differences():
    """Along a direction, by differences of float64 norms of the same values:
    a step of 2^-12 leaves 2^-24 |f'''| / 6, far below the 2^-17 asked for."""
    rng = np.random.default_rng(8)
    x, dy, v = (randn(rng, 12, 200) for _ in range(3))
    w, u = 1 + 0.2 * randn(rng, 200), randn(rng, 200)
    h, rstd, _, _, _ = av.averis_rmsnorm(x.cuda(), w.cuda(), eps=1e-4)
    dh, dw = av.averis_rmsnorm_grad(dy.cuda(), h, w.cuda(), rstd)
    f = lambda x, w: np.sum(num(dy) * block.rmsnorm(x, w, 1e-4)[1])
    e = 2.0 ** -12
    slope = (f(num(x) + e * num(v), num(w)) - f(num(x) - e * num(v), num(w))) / (2 * e)
    assert abs(np.sum(num(dh) * num(v)) - slope) < 2.0 ** -17 * np.sum(np.abs(num(dh) * num(v)))
    slope = (f(num(x), num(w) + e * num(u)) - f(num(x), num(w) - e * num(u))) / (2 * e)
    assert abs(np.sum(num(dw) * num(u)) - slope) < 2.0 ** -17 * np.sum(np.abs(num(dw) * num(u)))


def test_many_rows_and_offsets_past_32_bits():
    """Sums over many rows, and tensors of more than 2^32 bytes: the first and the last rows."""
    rows, cols = 300_000, 8192
    x = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_()
    w = torch.rand(cols, device="cuda") + 0.5
    h, rstd, y, q, qt = av.averis_rmsnorm(x, w, residual=x, y=True, transposed=True)
    some = [0, 1, 131072, rows - 2, rows - 1]
    ref_r, ref_y = block.rmsnorm(2 * num(x[some]), num(w), 1e-6)
    assert np.all(np.abs(num(y[some]) - ref_y) <= 3 * U * np.abs(ref_y) + half(ref_y, BF16))
    assert same_fp8(av.averis_fp8_quant(y[-300:].contiguous()), av.FP8(q.codes[-300:], q.scales[-300:], 300, cols))
    last = rows - rows % 128   # the last run of the transposed copy, and one in the middle
    for a, b in ((last, rows), (150016, 150144)):
        part = av.averis_fp8_quant(y[a:b].contiguous(), transposed=True, plain=False)[1]
        assert torch.equal(qt.codes[:, a:a + 128], part.codes)
        assert torch.equal(qt.scales[:, a // 128], part.scales[:, 0])
    del q, qt, y
    dh, dw = av.averis_rmsnorm_grad(x, h, w, rstd, dres=h)
    ref_h, _ = block.rmsnorm_grad(num(x[some]), num(h[some]), num(w), num(rstd[some]))
    ref_h = ref_h + num(h[some])
    lim = 64 * U * np.max(np.abs(ref_h)) + half(ref_h, BF16)
    assert np.all(np.abs(num(dh[some]) - ref_h) <= lim)
    # a tensor of ones as dy: dw = sum of h rstd, here in float64 over the rows in pieces
    ref = sum((h[i:i + 20000].double() * rstd[i:i + 20000, None].double() * x[i:i + 20000].double()).sum(0)
              for i in range(0, rows, 20000))
    mag = sum((h[i:i + 20000].float() * rstd[i:i + 20000, None] * x[i:i + 20000].float()).abs().sum(0)
              for i in range(0, rows, 20000)).double()
    assert ((dw.double() - ref).abs() <= (rows / 512 + 90) * U * mag).all()
