"""Back through an activation and a bias into fp8, on the GPU.

Without an activation, and with relu, dz is determined: the codes are
averis_fp8_quant's.  The smooth ones: the argument of the sigmoid carries at
most 5 x 2^-24 of itself, exp2 and the reciprocal an ulp each, so s is off by at
most 5 x 2^-24; times z (1 - 2 s) u' and the rounding of 1 - s at 2^-24 times
z s u', which is at most 33 where 1 - s is near 2^-24 (gelu, z = 4.9) and falls
after it: under 2^-17 on the slope.  A dequantized code is then within half a
step (2^-4 relative, or 2^-10 of its scale) of dz, with half a step of dz's
type before it.  dbias adds 4 rows a thread, 2 + 8 in a workgroup, rows / 2048 +
16 at the end."""

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


def num(t):
    return t.double().cpu().numpy()


def strided(a, pad, lead=0):
    buf = torch.full((a.shape[0] * (a.shape[1] + pad) + lead,), 7.0, dtype=a.dtype, device="cuda")
    v = buf[lead:].as_strided(a.shape, (a.shape[1] + pad, 1), lead)
    v.copy_(a)
    return v


def inputs(rng, rows, cols, dtype):
    dy = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))
    z = 3.0 * rng.standard_normal((rows, cols))
    z[rng.random((rows, cols)) < 0.02] = 0.0
    z[rng.random((rows, cols)) < 0.02] *= 100.0
    return tuple(torch.from_numpy(t.astype(np.float32)).to(dtype) for t in (dy, z))


def check_codes(codes, scales, dz, err):
    """codes (rows x cols) and scale bytes of dz, known to within err."""
    cols, kb = dz.shape[1], scales.shape[1]
    pad = lambda t: np.pad(t, ((0, 0), (0, 128 * kb - cols))).reshape(t.shape[0], kb, 128)
    scale = 2.0 ** (scales.astype(np.float64) - 127)
    top = np.max(np.abs(pad(dz)), axis=2)
    off = np.max(pad(err), axis=2)
    assert np.all(top - off <= 448 * scale)
    assert np.all((top + off > 224 * scale) | (scales == 0))
    s = np.repeat(scale, 128, axis=1)[:, :cols]
    got = fp8.dequantize(codes, scales)
    assert np.all(np.abs(got - dz) <= 2.0 ** -4 * (np.abs(dz) + err) + 2.0 ** -10 * s + err)


SHAPES = [(1, 1), (1, 300), (5, 8), (130, 129), (128, 128), (257, 600), (1000, 72), (3, 5000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gradient(rows, cols, act, dtype):
    dy, z = inputs(np.random.default_rng([rows, cols]), rows, cols, dtype)
    kb = -(-cols // 128)
    zg = None if act == "none" else z.cuda()
    q, qt, db = av.averis_fp8_act_grad(dy.cuda(), z=zg, act=act)
    dz = num(dy) * block.act_slope(num(z), act)
    assert db.shape == (cols,)
    if act in ("none", "relu"):
        # (relu leaves +0 where it masks, not 0 times dy)
        exact = torch.from_numpy(dz if act == "none" else np.where(num(z) > 0, dz, 0.0)).float().to(dtype).cuda()
        p, pt = av.averis_fp8_quant(exact, transposed=True)
        assert torch.equal(q.codes, p.codes) and torch.equal(qt.codes, pt.codes)
        assert torch.equal(q.scales[:, :kb], p.scales[:, :kb])
        assert torch.equal(qt.scales[:, :-(-rows // 128)], pt.scales[:, :-(-rows // 128)])
        slope = 0.0
    else:
        slope = 2.0 ** -17
        err = np.abs(num(dy)) * slope + np.abs(dz) * (BF16_REL if dtype == BF16 else U)
        check_codes(q.codes.cpu().numpy()[:, :cols], q.scales.cpu().numpy()[:, :kb], dz, err)
        check_codes(qt.codes.cpu().numpy()[:, :rows], qt.scales.cpu().numpy()[:, :-(-rows // 128)], dz.T, err.T)
        assert (q.codes[:, cols:] == 0).all() and (qt.codes[:, rows:] == 0).all()
    lim = (slope * np.sum(np.abs(num(dy)), axis=0) +
           (4 + 10 + rows / 2048 + 18) * U * np.sum(np.abs(dz), axis=0) + 1e-38)
    assert np.all(np.abs(num(db) - dz.sum(0)) <= lim)
    # unaligned rows; each output alone; the same bits
    for pad, lead in ((3, 1), (0, 5)):
        zs = None if zg is None else strided(z, pad + 1, lead)
        a, b, c = av.averis_fp8_act_grad(strided(dy, pad, lead), z=zs, act=act)
        assert torch.equal(a.codes, q.codes) and torch.equal(b.codes, qt.codes) and torch.equal(c, db)
    a, b, c = av.averis_fp8_act_grad(dy.cuda(), z=zg, act=act, transposed=False, bias=False)
    assert b is None and c is None and torch.equal(a.codes, q.codes)
    a, b, c = av.averis_fp8_act_grad(dy.cuda(), z=zg, act=act, plain=False, bias=False)
    assert a is None and c is None and torch.equal(b.codes, qt.codes)
    a, b, c = av.averis_fp8_act_grad(dy.cuda(), z=zg, act=act, plain=False, transposed=False)
    assert a is None and b is None and torch.equal(c, db)
    a, b, c = av.averis_fp8_act_grad(dy.cuda(), z=zg, act=act, transposed=False)
    assert torch.equal(a.codes, q.codes) and torch.equal(c, db)


OFFSETS = [[0, 300], [0, 0, 1, 129, 129, 300], [0, 128, 256, 300], [0, 7, 7, 7, 250], [0] * 70 + [100, 300] + [300] * 60]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("offs", OFFSETS)
def test_segments(offs, act, dtype):
    rows, cols, nseg = 300, 200, len(offs) - 1
    dy, z = inputs(np.random.default_rng(len(offs)), rows, cols, dtype)
    zg = z.cuda() if act != "none" else None
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    q, qt, db = av.averis_fp8_act_grad(dy.cuda(), z=zg, act=act, offsets=o)
    assert db.shape == (nseg, cols)
    starts = fp8.seg_starts(np.array(offs))
    for s in range(nseg):
        a, b = offs[s], offs[s + 1]
        if a == b:
            assert (db[s] == 0).all()
            continue
        p, pt, pb = av.averis_fp8_act_grad(dy[a:b].cuda(), z=None if zg is None else zg[a:b], act=act)
        assert torch.equal(q.codes[a:b], p.codes) and torch.equal(q.scales[a:b, :2], p.scales[:, :2])
        assert torch.equal(qt.codes[:, starts[s]:starts[s + 1]], pt.codes)
        k0, k1 = starts[s] // 128, starts[s + 1] // 128
        assert torch.equal(qt.scales[:, k0:k1], pt.scales[:, :k1 - k0])
        assert torch.equal(db[s], pb)


def test_malformed_offsets_address_nothing_outside():
    """Decreasing and outlying offsets, which the kernels clamp, claim rows more than once: more runs than any
    division of the rows has.  What the calls before and after wrote stays."""
    rows, cols = 300, 200
    dy = torch.randn(rows, cols, device="cuda")
    ref = av.averis_fp8_act_grad(dy)
    for offs in ([0, 300, 0, 300, 0, 300], [-5, 400, 7, 1 << 40, -(1 << 40), 300, 2, 290, 1, 300], [300, 0, 300, 0]):
        o = torch.tensor(offs, dtype=torch.int64, device="cuda")
        need = av.workspace_bytes(av.OP_FP8_ACT_GRAD, rows, cols, 0, len(offs) - 1)
        buf = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
        _, _, db = av.averis_fp8_act_grad(dy, offsets=o, ws=buf[:need])
        assert db.shape == (len(offs) - 1, cols)
        assert (buf[need:] == 77).all()
    again = av.averis_fp8_act_grad(dy)
    assert torch.equal(again[0].codes, ref[0].codes) and torch.equal(again[1].codes, ref[1].codes)
    assert torch.equal(again[2], ref[2])


def test_special_values():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[inf, -inf, nan, 1e30, -1e30, 0.0, -0.0, 200.0, -200.0]], device="cuda")
    for dtype in (F32, BF16):
        dy = torch.full_like(z, 2.0).to(dtype)
        for act in ("silu", "gelu", "relu"):
            _, _, db = av.averis_fp8_act_grad(dy, z=z.to(dtype), act=act)
            mid = 0.0 if act == "relu" else 1.0
            want = [2.0, 0.0, nan, 2.0, 0.0, mid, mid, 2.0, 0.0]
            if act == "relu":
                want[2] = 2.0                                # z <= 0 is false
            np.testing.assert_allclose(num(db), want, atol=1e-6)
        q, _, _ = av.averis_fp8_act_grad(dy, z=z.to(dtype), act="gelu")
        assert (q.codes[0, :9] == 0x7F).all()                # a run with a NaN
    # what is masked by relu stays masked, and a NaN gradient reaches the sums
    _, _, db = av.averis_fp8_act_grad(torch.tensor([[nan, nan]], device="cuda"), z=torch.tensor([[-1.0, 1.0]], device="cuda"),
                                      act="relu")
    assert db[0] == 0 and torch.isnan(db[1])


@pytest.mark.parametrize("offs", [None, [0, 0, 0]])
def test_no_rows(offs):
    dy = torch.empty(0, 40, device="cuda")
    o = None if offs is None else torch.tensor(offs, device="cuda")
    q, qt, db = av.averis_fp8_act_grad(dy, z=dy, act="gelu", offsets=o)
    assert q.codes.shape == (0, 128) and (db == 0).all() and db.shape == ((40,) if offs is None else (2, 40))


def test_offsets_past_32_bits():
    rows, cols = 300_000, 8192
    dy = torch.randint(-4, 5, (rows, cols), dtype=torch.int8, device="cuda").to(BF16)
    z = torch.ones_like(dy)
    z[-129:, ::2] = -1.0
    q, qt, db = av.averis_fp8_act_grad(dy, z=z, act="relu")
    dy[-129:, ::2] = 0.0
    p = av.averis_fp8_quant(dy[-200:].contiguous())
    assert torch.equal(q.codes[-200:], p.codes)
    a = rows - rows % 128
    pt = av.averis_fp8_quant(dy[a:].contiguous(), transposed=True, plain=False)[1]
    assert torch.equal(qt.codes[:, a:], pt.codes)
    ref = sum(dy[i:i + 20000].double().sum(0) for i in range(0, rows, 20000))
    assert torch.equal(db.double(), ref)                     # integers below 2^24: exact


@pytest.mark.parametrize("nseg", [9, 300, 4096])
def test_bias_gradient_of_many_segments(nseg):
    """Segments of none, few and many runs of 128, more than one workgroup's; their sums are those of calls on
    their own, bit for bit."""
    rng = np.random.default_rng(nseg)
    rows, cols = 9000, 70
    cuts = np.sort(rng.integers(0, 3000, nseg - 1))
    offs = [0] + cuts.tolist() + [rows]   # the last one of over 46 runs
    dy = torch.randn(rows, cols, device="cuda")
    z = torch.randn(rows, cols, device="cuda")
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    _, _, db = av.averis_fp8_act_grad(dy, z=z, act="silu", plain=False, transposed=False, offsets=o)
    filled = [s for s in range(nseg) if offs[s] < offs[s + 1]]
    for s in sorted(set(rng.choice(filled, min(len(filled), 20)).tolist() + [filled[-1]])):
        a, b = offs[s:s + 2]
        assert torch.equal(db[s], av.averis_fp8_act_grad(dy[a:b], z=z[a:b], act="silu", plain=False, transposed=False)[2])
    empty = [s for s in range(nseg) if offs[s] == offs[s + 1]]
    assert (db[empty] == 0).all()
    s64 = torch.sigmoid(z.double())
    d64 = dy.double() * s64 * (1 + z.double() * (1 - s64))
    ref = torch.zeros(nseg, cols, dtype=torch.float64, device="cuda")
    which = torch.from_numpy(np.searchsorted(np.array(offs[1:]), np.arange(rows), side="right")).cuda()
    ref.index_add_(0, which, d64)
    mag = torch.zeros_like(ref).index_add_(0, which, d64.abs())
    # a sum of n fp32 terms, each off by its slope's 2^-17 and its own rounding
    n = torch.tensor(np.diff(np.array(offs)), device="cuda").double()[:, None]
    lim = (n + 1) * U * mag + 2.0 ** -17 * torch.zeros_like(ref).index_add_(0, which, dy.double().abs())
    assert ((db.double() - ref).abs() <= lim + 1e-30).all()
