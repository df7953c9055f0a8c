"""Block-scaled fp8 quantization and products on the GPU against the float64
oracle.

Codes and scale bytes are determined, so they have to be equal.  A product's
error: the matrix instruction cuts each of eight consecutive products at 2^-13
of the largest, at most 7 x 2^-13 < 2^-10 of sum |a b|; the fp32 additions of
K / 8 groups are far below (K <= 2^14: K / 8 x 2^-24 = 2^-13); together within
2^-10 + 2^-13 of sum |a b|, below tests/parity.py's GEMM_TOL plus that last
term.  bf16 output adds half an ulp.  Operands of few bits (integers up to 4,
scales 1) lose nothing in either place: those products have to be exact."""

import numpy as np
import pytest
import torch

from oracle import fp8
from tests.parity import BF16_REL
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = 2.0 ** -10 + 2.0 ** -13


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def values(rng, rows, cols, dtype):
    a = rng.standard_normal((rows, cols)) * np.exp(2.0 * rng.standard_normal((rows, 1)))
    a[rng.random((rows, cols)) < 0.05] = 0.0
    if rows > 3:
        a[1] = 0.0
        a[2] *= 1e-37                       # at the smallest scales
        a[3] *= 1e34
        a[3, cols // 2] = 448.0 * 2.0 ** 100
    return torch.from_numpy(a.astype(np.float32)).to(dtype)


def strided(a, pad):
    buf = torch.full((a.shape[0], a.shape[1] + pad), 3.0, dtype=a.dtype, device="cuda")
    buf[:, pad // 2:pad // 2 + a.shape[1]] = a.cuda()
    return buf[:, pad // 2:pad // 2 + a.shape[1]]


def check(q, codes, scales):
    kb = -(-q.cols // 128)
    got = q.codes.cpu().numpy()
    np.testing.assert_array_equal(q.scales.cpu().numpy()[:, :kb], scales)
    np.testing.assert_array_equal(got[:, :q.cols], codes)
    assert (got[:, q.cols:] == 0).all()     # the pad


def deq(q):
    kb = -(-q.cols // 128)
    return fp8.dequantize(q.codes.cpu().numpy()[:, :q.cols], q.scales.cpu().numpy()[:, :kb])


QUANTS = [(1, 1), (1, 2048), (3, 127), (5, 129), (130, 64), (128, 128), (257, 600), (64, 1000), (1000, 3)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", QUANTS)
def test_quant(rows, cols, dtype):
    a = values(np.random.default_rng([rows, cols]), rows, cols, dtype)
    n = a.double().numpy()
    for pad in (0, 7):
        g = strided(a, pad)
        check(av.averis_fp8_quant(g), *fp8.quantize(n))
        q, qt = av.averis_fp8_quant(g, transposed=True)
        check(q, *fp8.quantize(n))
        check(qt, *fp8.quantize(n.T))
        none, qt = av.averis_fp8_quant(g, transposed=True, plain=False)
        assert none is None
        check(qt, *fp8.quantize(n.T))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_every_scale(dtype):
    """Blocks whose maximum is at and next to each step of the scale, over the
    type's whole range, subnormal numbers included."""
    top = np.float64(2.0) ** np.arange(-148, 128)
    a = np.stack([top, 1.75 * top, np.minimum(1.7578125 * top, 3.38e38), 1.9921875 * top])
    a = np.clip(a, 0, 3.38e38).reshape(-1, 1) * np.linspace(1.0, -1.0, 128)[None, :] ** 3
    t = torch.from_numpy(a.astype(np.float32)).to(dtype)
    n = t.double().numpy()
    check(av.averis_fp8_quant(t.cuda()), *fp8.quantize(n))
    q, qt = av.averis_fp8_quant(t.cuda().t().contiguous(), transposed=True)
    check(qt, *fp8.quantize(n))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_values_that_are_not_finite(dtype):
    a = values(np.random.default_rng(9), 300, 300, dtype)
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        a[5 + 50 * i, 100 * i + 20] = v
    n = a.double().numpy()
    q, qt = av.averis_fp8_quant(a.cuda(), transposed=True)
    check(q, *fp8.quantize(n))
    check(qt, *fp8.quantize(n.T))
    check(av.averis_fp8_quant(a.cuda()), *fp8.quantize(n))
    wt, wd = av.averis_fp8_quant_weight(a.cuda())
    check(wd, *fp8.quantize(n, True))
    check(wt, *fp8.quantize(n.T, True))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (1, 300, 130), (3, 128, 256), (2, 77, 200)])
def test_quant_weight(batch, rows, cols, dtype):
    rng = np.random.default_rng([batch, rows, cols])
    w = torch.stack([values(rng, rows, cols, dtype) for _ in range(batch)])
    big = torch.zeros(batch, rows + 2, cols + 3, dtype=dtype, device="cuda")
    big[:, :rows, :cols] = w.cuda()
    for g in ((w.cuda(), big[:, :rows, :cols]) if batch > 1 else (w[0].cuda(), big[0, :rows, :cols])):
        wt, wd = av.averis_fp8_quant_weight(g)
        d = [fp8.quantize(m.double().numpy(), True) for m in w]
        t = [fp8.quantize(m.double().numpy().T, True) for m in w]
        check(wd, np.concatenate([x[0] for x in d]), np.concatenate([x[1] for x in d]))
        check(wt, np.concatenate([x[0] for x in t]), np.concatenate([x[1] for x in t]))


OFFSETS = [[0, 300], [0, 0, 1, 129, 129, 300], [0, 128, 256, 300], [0, 7, 7, 7, 250]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offs", OFFSETS)
def test_quant_segments(offs, dtype):
    rows, cols, nseg = 300, 200, len(offs) - 1
    a = values(np.random.default_rng(5), rows, cols, dtype)
    n = a.double().numpy()
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    q, qt = av.averis_fp8_quant(a.cuda(), transposed=True, offsets=o)
    codes, scales = fp8.quantize(n)
    end = offs[-1]                                          # the tail is in no segment
    np.testing.assert_array_equal(q.codes.cpu().numpy()[:end, :cols], codes[:end])
    np.testing.assert_array_equal(q.scales.cpu().numpy()[:end, :2], scales[:end])
    starts = fp8.seg_starts(np.array(offs))
    for s in range(nseg):
        c, sc = fp8.quantize(n[offs[s]:offs[s + 1]].T)
        m = offs[s + 1] - offs[s]
        got = qt.codes.cpu().numpy()[:, starts[s]:starts[s + 1]]
        np.testing.assert_array_equal(got[:, :m], c)
        assert (got[:, m:] == 0).all()
        np.testing.assert_array_equal(
            qt.scales.cpu().numpy()[:, starts[s] // 128:starts[s + 1] // 128], sc)


def close(c, a, b, what=""):
    r, bound = a @ b.T, np.abs(a) @ np.abs(b).T
    lim = TOL * bound + (BF16_REL * np.abs(r) if c.dtype == BF16 else 0.0) + 1e-38
    err = np.abs(c.double().cpu().numpy() - r)
    assert np.all(err <= lim), "%s max error / sum |a b| %.3g" % (what, np.max(err / np.maximum(bound, 1e-300)))


def gpu_quant(rng, rows, cols):
    return av.averis_fp8_quant(torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)
                                                * np.exp(rng.standard_normal((rows, 1)))).cuda().to(BF16))


# every kernel and its edges: single rows, the few-rows kernels, tiles that end
# inside, one to many stages, splits, wide and narrow tiles
GEMMS = [(1, 1, 1), (1, 1024, 2048), (16, 48, 128), (17, 50, 300), (33, 16, 4096), (64, 200, 640),
         (65, 64, 128), (100, 130, 256), (256, 256, 384), (257, 300, 512), (300, 96, 8192),
         (1000, 777, 1000), (2300, 520, 640), (520, 2300, 129)]


@pytest.mark.parametrize("m,n,k", GEMMS)
def test_gemm(m, n, k):
    rng = np.random.default_rng([m, n, k])
    a, b = gpu_quant(rng, m, k), gpu_quant(rng, n, k)
    da, db = deq(a), deq(b)
    for dt in (F32, BF16):
        c = av.averis_fp8_gemm(a, b, dt)
        close(c, da, db)
        assert torch.equal(av.averis_fp8_gemm(a, b, dt), c)            # the same bits
        buf = torch.full((m, n + 5), 9.0, dtype=dt, device="cuda")     # strided, unaligned output
        av.averis_fp8_gemm(a, b, dt, out=buf[:, 3:3 + n])
        assert torch.equal(buf[:, 3:3 + n], c) and (buf[:, :3] == 9).all() and (buf[:, 3 + n:] == 9).all()


def exact_fp8(rng, rows, cols):
    """An fp8 tensor of small integers with scales that differ by row and block."""
    v = rng.integers(-4, 5, (rows, cols)).astype(np.float64)
    kb = -(-cols // 128)
    e = rng.integers(-1, 2, (rows, kb))
    q = av.FP8.empty(rows, cols)
    q.codes.zero_()
    q.scales.zero_()
    q.codes[:, :cols] = torch.from_numpy(fp8.encode(v)).cuda()
    q.scales[:, :kb] = torch.from_numpy((e + 127).astype(np.uint8)).cuda()
    return q, v * np.repeat(2.0 ** e, 128, 1)[:, :cols]


@pytest.mark.parametrize("m,n,k", GEMMS)
def test_gemm_of_small_integers_is_exact(m, n, k):
    """Sums of at most 8192 products of up to 16 x 2^+-2 stay below 2^24 quarter
    units, and eight neighbours differ by less than 2^13: nothing is rounded."""
    rng = np.random.default_rng([m, n, k, 1])
    a, va = exact_fp8(rng, m, k)
    b, vb = exact_fp8(rng, n, k)
    c = av.averis_fp8_gemm(a, b, F32)
    np.testing.assert_array_equal(c.cpu().numpy(), va @ vb.T)


@pytest.mark.parametrize("k,n", [(200, 96), (640, 300)])
@pytest.mark.parametrize("offs", [[0, 5], [0, 0, 3, 3, 70, 90], [0, 256, 256, 900, 1500, 1500],
                                  [0, 300, 310, 1400]])
def test_gemm_segments(offs, k, n):
    rng = np.random.default_rng(offs + [k])
    nseg, rows = len(offs) - 1, offs[-1] + 3                # three rows in no segment
    a, va = exact_fp8(rng, rows, k)
    b, vb = exact_fp8(rng, nseg * n, k)
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    for dt in (F32, BF16):
        c = torch.full((rows, n), 7.0, dtype=dt, device="cuda")
        av.averis_fp8_gemm(a, b, dt, offsets=o, out=c)
        ref = np.concatenate([va[offs[s]:offs[s + 1]] @ vb[s * n:(s + 1) * n].T for s in range(nseg)])
        got = c.float().cpu().numpy()
        np.testing.assert_array_equal(
            got[:offs[-1]], torch.from_numpy(ref).float().to(dt).float().numpy())
        assert (got[offs[-1]:] == 7).all()


@pytest.mark.parametrize("nseg", [64, 65, 200, 1024])
def test_many_segments(nseg):
    """More segments than a wavefront has lanes, many of them empty."""
    rng = np.random.default_rng([nseg, 8])
    rows, m, n = 3 * nseg, 72, 40
    cuts = np.sort(rng.integers(0, rows + 1, nseg - 1))
    offs = [0] + [int(v) for v in cuts] + [rows]
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    x, d = (torch.from_numpy(rng.integers(-4, 5, (rows, c)).astype(np.float32)).cuda().to(BF16) for c in (m, n))
    w = torch.from_numpy(rng.integers(-4, 5, (nseg, m, n)).astype(np.float32)).cuda().to(BF16)
    xq, xt = av.averis_fp8_quant(x, transposed=True, offsets=o)
    _, dt = av.averis_fp8_quant(d, transposed=True, offsets=o)
    wt, _ = av.averis_fp8_quant_weight(w)
    y = av.averis_fp8_gemm(xq, wt, F32, offsets=o)
    g = av.averis_fp8_gemm_wgrad(xt, dt, F32, offsets=o)
    xn, dn, wn = (t.double().cpu().numpy() for t in (x, d, w))
    seg = np.searchsorted(np.array(offs[1:]), np.arange(rows), side="right")
    np.testing.assert_array_equal(y.cpu().numpy(), np.einsum("ri,rio->ro", xn, wn[seg]))
    np.testing.assert_array_equal(
        g.cpu().numpy(), np.stack([xn[a:b].T @ dn[a:b] for a, b in zip(offs, offs[1:])]))


# Sizes for the 256 x 256 tile: one tile a workgroup, several (the next one's
# loads under the output), and K cut into fp32 partial sums.  The products are
# of small integers, and the reference is theirs in float64.
LARGE = [(3001, 3003, 3790), (12001, 2203, 800), (1001, 3003, 16300)]


@pytest.mark.parametrize("m,n,k", LARGE)
def test_large_products_are_exact(m, n, k):
    rng = np.random.default_rng([m, n, k, 2])
    a, va = exact_fp8(rng, m, k)
    b, vb = exact_fp8(rng, n, k)
    ref = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda().t()
    for dt in (F32, BF16):
        c = av.averis_fp8_gemm(a, b, dt)
        assert torch.equal(c, ref.to(dt))
        buf = torch.full((m + 2, n + 5), 9.0, dtype=dt, device="cuda")   # rows that start anywhere
        av.averis_fp8_gemm(a, b, dt, out=buf[1:1 + m, 3:3 + n])
        assert torch.equal(buf[1:1 + m, 3:3 + n], c)
        buf[1:1 + m, 3:3 + n] = 9.0
        assert (buf == 9).all()
        a2 = av.averis_fp8_gemm(a, b, dt, out=torch.empty(m, n + 8, dtype=dt, device="cuda")[:, :n])
        assert torch.equal(a2, c)                                        # whole 16-byte pieces


@pytest.mark.parametrize("offs", [[0, 1, 1, 2500, 2756, 8000, 9000], [0, 0, 9000, 9000, 9000, 9000, 9000],
                                  [0, 300, 556, 556, 557, 4000, 8900]])
def test_large_row_segments_are_exact(offs):
    rng = np.random.default_rng(offs)
    nseg, rows, n, k = len(offs) - 1, 9000, 2103, 2100
    a, va = exact_fp8(rng, rows, k)
    b, vb = exact_fp8(rng, nseg * n, k)
    va, vb = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    ref = torch.full((rows, n), 7.0, dtype=torch.float64, device="cuda")
    for s in range(nseg):
        if offs[s] < offs[s + 1]:
            ref[offs[s]:offs[s + 1]] = va[offs[s]:offs[s + 1]] @ vb[s * n:(s + 1) * n].t()
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    for dt in (F32, BF16):
        c = torch.full((rows, n), 7.0, dtype=dt, device="cuda")
        av.averis_fp8_gemm(a, b, dt, offsets=o, out=c)
        assert torch.equal(c, ref.to(dt))


@pytest.mark.parametrize("m,n,offs", [
    (2101, 2055, [0, 4000, 4000, 4129, 9400]), (130, 70, [0, 100, 9000, 9000, 9200]), (256, 512, [0, 8192, 9000]),
    (300, 2048, [0, 10, 20, 4500, 4510, 9300]), (1000, 1001, [0] * 70 + [50, 100, 6000, 6001, 9400] + [9400] * 10)])
def test_wgrad_long_segments_are_exact(m, n, offs):
    rng = np.random.default_rng(offs + [m, n])
    rows, nseg = 9400, len(offs) - 1
    x, d = (torch.from_numpy(rng.integers(-4, 5, (rows, c)).astype(np.float32)).cuda().to(BF16) for c in (m, n))
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    _, xt = av.averis_fp8_quant(x, transposed=True, offsets=o, plain=False)
    _, dt = av.averis_fp8_quant(d, transposed=True, offsets=o, plain=False)
    for dtype in (F32, BF16):
        out = torch.full((nseg + 1, m, n), 9.0, dtype=dtype, device="cuda")
        av.averis_fp8_gemm_wgrad(xt, dt, dtype, offsets=o, rows=rows, out=out[:nseg])
        for s in range(nseg):
            xs, ds = x[offs[s]:offs[s + 1]].double(), d[offs[s]:offs[s + 1]].double()
            assert torch.equal(out[s], (xs.t() @ ds).to(dtype))
        assert (out[nseg] == 9).all()
        again = av.averis_fp8_gemm_wgrad(xt, dt, dtype, offsets=o, rows=rows)
        assert torch.equal(again, out[:nseg])


@pytest.mark.parametrize("offs", [[0, 4000, 4000, 4129, 9400], [0, 0, 0, 9400, 9400], [0, 2048, 4700, 7000, 9300]])
def test_large_wgrad_segments_are_exact(offs):
    rng = np.random.default_rng(offs)
    rows, m, n, nseg = 9400, 2101, 2055, len(offs) - 1
    x, d = (torch.from_numpy(rng.integers(-4, 5, (rows, c)).astype(np.float32)).cuda().to(BF16) for c in (m, n))
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    _, xt = av.averis_fp8_quant(x, transposed=True, offsets=o, plain=False)
    _, dt = av.averis_fp8_quant(d, transposed=True, offsets=o, plain=False)
    for dtype in (F32, BF16):
        w = av.averis_fp8_gemm_wgrad(xt, dt, dtype, offsets=o)
        for s in range(nseg):
            xs, ds = x[offs[s]:offs[s + 1]].double(), d[offs[s]:offs[s + 1]].double()
            assert torch.equal(w[s], (xs.t() @ ds).to(dtype))


@pytest.mark.parametrize("l,m,n", [(1, 16, 8), (300, 96, 200), (5000, 256, 300), (128, 1000, 64), (0, 20, 30)])
def test_wgrad(l, m, n):
    rng = np.random.default_rng([l, m, n])
    x = torch.from_numpy(rng.standard_normal((l, m)).astype(np.float32)).cuda().to(BF16)
    d = torch.from_numpy(rng.standard_normal((l, n)).astype(np.float32)).cuda().to(BF16)
    _, xt = av.averis_fp8_quant(x, transposed=True)
    _, dt = av.averis_fp8_quant(d, transposed=True)
    for dtype in (F32, BF16):
        w = av.averis_fp8_gemm_wgrad(xt, dt, dtype)
        assert w.shape == (m, n)
        close(w, fp8.dequantize(*fp8.quantize(x.double().cpu().numpy().T)),
              fp8.dequantize(*fp8.quantize(d.double().cpu().numpy().T)))


@pytest.mark.parametrize("offs", [[0, 300], [0, 0, 1, 129, 129, 300], [0, 700, 700, 2000], [0, 40, 80, 81]])
def test_wgrad_segments(offs):
    rng = np.random.default_rng(offs)
    rows, m, n, nseg = offs[-1], 130, 270, len(offs) - 1
    x = torch.from_numpy(rng.integers(-4, 5, (rows, m)).astype(np.float32)).cuda().to(BF16)
    d = torch.from_numpy(rng.integers(-4, 5, (rows, n)).astype(np.float32)).cuda().to(BF16)
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    _, xt = av.averis_fp8_quant(x, transposed=True, offsets=o)
    _, dt = av.averis_fp8_quant(d, transposed=True, offsets=o, plain=False)
    xn, dn = x.double().cpu().numpy(), d.double().cpu().numpy()
    for dtype in (F32, BF16):
        w = av.averis_fp8_gemm_wgrad(xt, dt, dtype, offsets=o)
        ref = np.stack([xn[a:b].T @ dn[a:b] for a, b in zip(offs, offs[1:])])   # small integers: exact
        np.testing.assert_array_equal(w.float().cpu().numpy(),
                                      torch.from_numpy(ref).float().to(dtype).float().numpy())


def test_nan_reaches_the_output():
    x = torch.randn(300, 256, device="cuda").to(BF16)
    x[7, 3] = float("inf")
    w = torch.randn(256, 512, device="cuda").to(BF16)
    wt, wd = av.averis_fp8_quant_weight(w)
    y = av.averis_fp8_gemm(av.averis_fp8_quant(x), wt)
    assert torch.isnan(y[7]).all() and torch.isfinite(y[:7]).all() and torch.isfinite(y[8:]).all()


def test_linear_step_stream_and_graph():
    """A training step on another stream, and captured and replayed with eager
    work in between: the eager results bit for bit."""
    l, m, n = 1000, 320, 200
    x, d = (torch.randn(l, c, device="cuda").to(BF16) for c in (m, n))
    w = torch.randn(m, n, device="cuda").to(BF16)

    def step():
        xq, xt = av.averis_fp8_quant(x, transposed=True)
        dq, dt = av.averis_fp8_quant(d, transposed=True)
        wt, wd = av.averis_fp8_quant_weight(w)
        return [av.averis_fp8_gemm(xq, wt), av.averis_fp8_gemm(dq, wd), av.averis_fp8_gemm_wgrad(xt, dt),
                av.averis_fp8_gemm(av.averis_fp8_quant(x[:3]), wt)]
    ref = [v.clone() for v in step()]
    y = x.double() @ w.double()
    assert float((ref[0].double() - y).norm() / y.norm()) < 0.05
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for v in out:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
        step()


def test_offsets_past_32_bits():
    """Operands and outputs of more than 2^32 bytes: products of small integers,
    exact, at the first and the last rows."""
    rows, cols, n = 70001, 65536, 17
    small = lambda *s: torch.randint(-4, 5, s, dtype=torch.int8, device="cuda").to(BF16)
    a, b, d = small(rows, cols), small(n, cols), small(rows, n)
    q, qt = av.averis_fp8_quant(a, transposed=True)
    some = [0, 1, 32767, 65536, rows - 2, rows - 1]
    c = av.averis_fp8_gemm(q, av.averis_fp8_quant(b), F32)
    assert torch.equal(c[some].double(), a[some].double() @ b.double().t())
    _, dt = av.averis_fp8_quant(d, transposed=True)
    w = av.averis_fp8_gemm_wgrad(qt, dt, F32)
    some = [0, 1, 32769, cols - 2, cols - 1]
    assert torch.equal(w[some].double(), a[:, some].double().t() @ d.double())
    del a, q, qt, c, w
    x, y = small(rows, 128), small(40000, 128)
    c = av.averis_fp8_gemm(av.averis_fp8_quant(x), av.averis_fp8_quant(y), F32)   # 11 GB
    some = [0, 255, 26843, 53687, rows - 1]
    assert torch.equal(c[some].double(), x[some].double() @ y.double().t())
