"""Rejections of the calls around a block's linears and of the grouped routing:
refused before any HIP call (no GPU needed)."""

import ctypes
import weakref

import pytest
import torch

from mean_residual_quantized_amd import averis as av

P = 0x10000   # stand-in device address: validation must reject the call before using it
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return av.lib()


def f8(rows, cols, codes=P, scales=P):
    return av._FP8(codes, scales, rows, cols)


def ref(t):
    return ctypes.byref(t) if t is not None else None


def test_rmsnorm_rejections(L):
    def n(x=P, dt=av.BF16, rows=64, cols=100, ldx=100, res=P, ldr=100, w=P, wdt=av.F32, eps=1e-6, h=P,
          ldh=100, y=P, ldy=100, rstd=P, out=f8(64, 100), out_t=f8(100, 64)):
        return L.averis_rmsnorm(x, dt, rows, cols, ldx, res, ldr, w, wdt, eps, h, ldh, y, ldy, rstd,
                                ref(out), ref(out_t), None)
    assert n(dt=4) == 3
    assert n(wdt=4) == 3
    assert n(rows=-1) == 2
    assert n(rows=(1 << 30) + 1) == 2
    assert n(cols=0, ldx=0) == 2
    assert n(cols=av.MAX_NORM_COLS + 1, ldx=BIG, ldr=BIG, ldh=BIG, ldy=BIG) == 2
    assert n(ldx=99) == 2 and n(ldr=99) == 2 and n(ldh=99) == 2 and n(ldy=99) == 2
    assert n(x=None) == 1 and n(h=None) == 1 and n(w=None) == 1 and n(rstd=None) == 1
    assert n(y=None, out=None, out_t=None) == 1
    assert n(res=None) == 6                                # h without a residual
    assert n(eps=-1e-6) == 6 and n(eps=float("nan")) == 6
    assert n(x=P + 1) == 4 and n(res=P + 1) == 4 and n(h=P + 1) == 4 and n(y=P + 1) == 4
    assert n(rstd=P + 2) == 4 and n(w=P + 2) == 4
    assert n(dt=av.F32, x=P + 2) == 4
    assert n(out=f8(64, 99)) == 2
    assert n(out_t=f8(64, 100)) == 2                       # not transposed
    assert n(out=f8(64, 100, codes=P + 8)) == 4
    assert n(out=f8(64, 100, codes=None)) == 1
    # more tiles than a launch numbers
    many = (1 << 30) - 64
    assert n(rows=many, cols=1024, ldx=1024, ldr=1024, ldh=1024, ldy=1024, out=None, out_t=f8(1024, many)) == 2


def test_rmsnorm_grad_rejections(L):
    need = av.workspace_bytes(av.OP_RMSNORM_GRAD, 64, 100)

    def n(dy=P, dt=av.BF16, rows=64, cols=100, lddy=100, h=P, ldh=100, w=P, wdt=av.F32, rstd=P, dres=P,
          ldr=100, dh=P, ldo=100, dw=P, ws=P, wsb=1 << 30):
        return L.averis_rmsnorm_grad(dy, dt, rows, cols, lddy, h, ldh, w, wdt, rstd, dres, ldr, dh, ldo,
                                     dw, ws, wsb, None)
    assert need > 0
    assert n(dt=4) == 3 and n(wdt=9) == 3
    assert n(rows=-1) == 2 and n(cols=0) == 2 and n(cols=16385, lddy=BIG, ldh=BIG, ldr=BIG, ldo=BIG) == 2
    assert n(lddy=99) == 2 and n(ldh=99) == 2 and n(ldr=99) == 2 and n(ldo=99) == 2
    assert n(dy=None) == 1 and n(h=None) == 1 and n(w=None) == 1 and n(rstd=None) == 1 and n(dh=None) == 1
    assert n(dy=P + 1) == 4 and n(h=P + 1) == 4 and n(dres=P + 1) == 4 and n(dh=P + 1) == 4 and n(dw=P + 2) == 4
    assert n(ws=None) == 5 and n(wsb=need - 1) == 5
    assert n(ws=P + 16) == 4
    assert av.workspace_bytes(av.OP_RMSNORM_GRAD, -1, 100) == 0
    assert av.workspace_bytes(av.OP_RMSNORM_GRAD, 64, 16385) == 0


def test_act_grad_rejections(L):
    need = av.workspace_bytes(av.OP_FP8_ACT_GRAD, 64, 100)

    def a(dy=P, dt=av.BF16, rows=64, cols=100, lddy=100, z=P, ldz=100, act=3, offs=None, nseg=1,
          out=f8(64, 100), out_t=f8(100, 64), db=P, ws=P, wsb=1 << 30):
        return L.averis_fp8_act_grad(dy, dt, rows, cols, lddy, z, ldz, act, offs, nseg, ref(out),
                                     ref(out_t), db, ws, wsb, None)
    assert need == 512                                      # one chunk of 100 floats, in whole 256 bytes
    assert a(dt=4) == 3
    assert a(act=4) == 6 and a(act=-1) == 6
    assert a(rows=-1) == 2 and a(cols=0) == 2 and a(lddy=99) == 2 and a(ldz=99) == 2
    assert a(cols=(1 << 27) + 1, lddy=BIG, ldz=BIG, out=None, out_t=None) == 2
    assert a(rows=1 << 30, cols=1 << 10, lddy=BIG, ldz=BIG, out=None, out_t=None) == 2   # 2^26 tiles
    assert a(dy=None) == 1 and a(z=None) == 1
    assert a(out=None, out_t=None, db=None) == 1
    assert a(dy=P + 1) == 4 and a(z=P + 1) == 4 and a(db=P + 2) == 4
    assert a(out=f8(64, 99)) == 2 and a(out_t=f8(64, 100)) == 2
    assert a(nseg=2) == 6 and a(offs=P, nseg=0) == 6 and a(offs=P + 4, nseg=2) == 4
    assert a(offs=P, nseg=2) == 2                           # out_t without room for the segments
    assert a(ws=None) == 5 and a(wsb=need - 1) == 5 and a(ws=P + 16) == 4


def test_gemm_act_rejections(L):
    def g(a=f8(64, 256), b=f8(96, 256), bias=P, bdt=av.F32, act=3, res=P, ldr=96, offs=None, nseg=1, c=P,
          dt=av.BF16, ldc=96, z=P, ldz=96, ws=P, wsb=1 << 30):
        return L.averis_fp8_gemm_act(ref(a), ref(b), bias, bdt, act, res, ldr, offs, nseg, c, dt, ldc, z,
                                     ldz, ws, wsb, None)
    assert g(act=4) == 6 and g(act=-1) == 6
    assert g(bdt=7) == 3 and g(bias=P + 2) == 4 and g(bdt=av.BF16, bias=P + 1) == 4
    assert g(ldr=95) == 2 and g(ldz=95) == 2 and g(ldc=95) == 2
    assert g(res=P + 1) == 4 and g(z=P + 1) == 4 and g(c=P + 1) == 4
    assert g(a=None) == 1 and g(b=None) == 1 and g(c=None) == 1
    assert g(b=f8(96, 255)) == 2
    assert g(dt=3) == 3
    assert g(offs=P, nseg=5) == 2                           # 96 rows are no five matrices
    assert g(nseg=2) == 6
    assert g(ws=P + 16) == 4
    big = f8(1024, 1 << 14)
    need = av.workspace_bytes(av.OP_FP8_GEMM, 1024, 1 << 14, 1024)
    assert need > 0
    assert g(a=big, b=big, ldr=1024, ldc=1024, ldz=1024, wsb=need - 1) == 5


def test_route_groups_rejections(L):
    def r(l=P, dt=av.BF16, t=4, e=16, ld=16, k=4, bias=P, score=1, groups=4, kg=2, top=2, renorm=1, ids=P, w=P):
        return L.averis_moe_route_groups(l, dt, t, e, ld, k, bias, score, groups, kg, top, renorm, 1.0, ids,
                                         w, None)
    assert r(dt=5) == 3
    assert r(t=-1) == 2 and r(ld=15) == 2 and r(t=1 << 30) == 2
    assert r(e=0) == 6 and r(e=1025, ld=1025, groups=1, kg=1) == 6
    assert r(k=0) == 6 and r(k=17) == 6 and r(k=33, e=64, ld=64) == 6
    assert r(k=9) == 6                                      # two groups hold eight
    assert r(score=2) == 6 and r(score=-1) == 6
    assert r(groups=0) == 6 and r(groups=3) == 6 and r(groups=65, e=130, ld=130) == 6
    assert r(kg=0) == 6 and r(kg=5) == 6
    assert r(top=0) == 6 and r(top=3) == 6
    assert r(renorm=2) == 6
    assert r(l=None) == 1 and r(ids=None) == 1 and r(w=None) == 1
    assert r(l=P + 1) == 4 and r(bias=P + 2) == 4 and r(ids=P + 2) == 4 and r(w=P + 2) == 4

    def g(l=P, dt=av.BF16, t=4, e=16, ld=16, k=4, score=1, renorm=1, ids=P, dw=P, dl=P, ldd=16):
        return L.averis_moe_route_groups_grad(l, dt, t, e, ld, k, score, renorm, 1.0, ids, dw, dl, ldd, None)
    assert g(dt=5) == 3 and g(t=-1) == 2 and g(ld=15) == 2 and g(ldd=15) == 2
    assert g(k=17) == 6 and g(score=2) == 6 and g(renorm=-1) == 6
    assert g(l=None) == 1 and g(ids=None) == 1 and g(dw=None) == 1 and g(dl=None) == 1
    assert g(l=P + 1) == 4 and g(ids=P + 1) == 4 and g(dw=P + 1) == 4 and g(dl=P + 1) == 4


X = torch.zeros(64, 32)
W = torch.ones(32)
OFFS = torch.tensor([0, 32, 64])


def q(rows, cols):
    return av.FP8.empty(rows, cols, "cpu")


@pytest.mark.parametrize("bad,match", [
    (lambda: av.averis_rmsnorm(X, W[:31]), "weight"),
    (lambda: av.averis_rmsnorm(X, torch.ones(64)[::2]), "weight"),
    (lambda: av.averis_rmsnorm(X, W.to("meta")), "weight"),
    (lambda: av.averis_rmsnorm(X, W, residual=X[:63]), "residual"),
    (lambda: av.averis_rmsnorm(X, W, residual=X.bfloat16()), "residual"),
    (lambda: av.averis_rmsnorm(X, W, residual=X.to("meta")), "residual"),
    (lambda: av.averis_rmsnorm(X, W, out=X), "out"),
    (lambda: av.averis_rmsnorm(X, W, residual=X, out=X.t()), "out"),
    (lambda: av.averis_rmsnorm(X.t(), torch.ones(64)), "x"),
    (lambda: av.averis_rmsnorm_grad(X, X[:, :31], W, torch.ones(64)), "h"),
    (lambda: av.averis_rmsnorm_grad(X, X, W, torch.ones(63)), "rstd"),
    (lambda: av.averis_rmsnorm_grad(X, X, W, torch.ones(64).double()), "rstd"),
    (lambda: av.averis_rmsnorm_grad(X, X, W, torch.ones(64), dres=X.bfloat16()), "dres"),
    (lambda: av.averis_rmsnorm_grad(X, X, W, torch.ones(64), out=X.t()), "out"),
    (lambda: av.averis_fp8_act_grad(X, act="gelu"), "z"),
    (lambda: av.averis_fp8_act_grad(X, z=X[:63], act="gelu"), "z"),
    (lambda: av.averis_fp8_act_grad(X, z=X, act="tanh"), "act"),
    (lambda: av.averis_fp8_act_grad(X, offsets=OFFS.int()), "offsets"),
    (lambda: av.averis_fp8_act_grad(X, offsets=OFFS[:1]), "offsets"),
    (lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), act="tanh"), "act"),
    (lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), bias=torch.zeros(15)), "bias"),
    (lambda: av.averis_fp8_gemm_act(q(64, 32), q(32, 32), bias=torch.zeros(16), offsets=OFFS), "bias"),
    (lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), bias=torch.zeros(32)[::2]), "bias"),
    (lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), residual=torch.zeros(8, 16)), "residual"),
    (lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), residual=torch.zeros(8, 15).bfloat16()), "residual"),
    (lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), out=torch.zeros(8, 15)), "out"),
    (lambda: av.averis_moe_route_groups(X, 4, score="tanh"), "score"),
    (lambda: av.averis_moe_route_groups(X, 4, bias=torch.zeros(31)), "bias"),
    (lambda: av.averis_moe_route_groups(X, 4, bias=torch.zeros(32).bfloat16()), "bias"),
    (lambda: av.averis_moe_route_groups_grad(X, torch.zeros(63, 4, dtype=torch.int32), torch.zeros(63, 4)), "ids"),
    (lambda: av.averis_moe_route_groups_grad(X, torch.zeros(64, 4, dtype=torch.int32), torch.zeros(64, 3)), "dweights"),
])
def test_binding_rejections(bad, match, monkeypatch):
    monkeypatch.setattr(av, "_stream_on", lambda t: None)
    with pytest.raises(ValueError, match=match):
        bad()


def test_binding_type_rejections(monkeypatch):
    monkeypatch.setattr(av, "_stream_on", lambda t: None)
    for bad in (lambda: av.averis_rmsnorm(X.half(), W), lambda: av.averis_rmsnorm(X, W.half()),
                lambda: av.averis_fp8_gemm_act(q(8, 32), q(16, 32), bias=torch.zeros(16).half()),
                lambda: av.averis_moe_route_groups(X.double(), 4)):
        with pytest.raises(TypeError):
            bad()


def test_host_tensors_are_refused():
    for bad in (lambda: av.averis_rmsnorm(X, W), lambda: av.averis_moe_route_groups(X, 4),
                lambda: av.averis_fp8_act_grad(X)):
        with pytest.raises(ValueError, match="current GPU"):
            bad()


CALLS = {
    "rmsnorm_grad": lambda ws: av.averis_rmsnorm_grad(X, X, W, torch.ones(64), ws=ws),
    "act_grad": lambda ws: av.averis_fp8_act_grad(X, ws=ws),
    "act_grad by segment": lambda ws: av.averis_fp8_act_grad(X, offsets=OFFS, ws=ws),
    "gemm_act": lambda ws: av.averis_fp8_gemm_act(q(1024, 1 << 14), q(1024, 1 << 14), ws=ws),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_workspace(name, monkeypatch):
    """One that the binding makes lives until the library has returned; a given
    one is checked (a stub in place of the library)."""
    real, make, made, seen = av.lib(), av._workspace, [], []

    class Stub:
        def __getattr__(self, fn):
            if fn in ("averis_workspace_bytes", "averis_status_str", "averis_fp8_seg_cols"):
                return getattr(real, fn)

            def call(*args):
                t = made[-1]()
                seen.append(t is not None and t.data_ptr() in args)
                return 0
            return call

    def workspace(nbytes, device):
        t = make(nbytes, "cpu")
        made.append(weakref.ref(t))
        return t
    monkeypatch.setattr(av, "lib", Stub)
    monkeypatch.setattr(av, "_stream_on", lambda t: None)
    monkeypatch.setattr(av, "_workspace", workspace)
    CALLS[name](None)
    assert seen == [True]
    flat = torch.zeros(1 << 27, dtype=torch.uint8)
    for bad in (flat.to("meta"), flat[::2]):
        with pytest.raises(ValueError, match="ws"):
            CALLS[name](bad)
    made.append(weakref.ref(flat))
    CALLS[name](flat)
    assert seen == [True, True]
