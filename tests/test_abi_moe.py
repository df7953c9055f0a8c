"""Rejections of the routing, token exchange and clipping calls: every bad
argument is refused before any HIP call (no GPU needed)."""

import ctypes

import pytest
import torch

from mean_residual_quantized_amd import averis as av

P = 0x10000   # stand-in device address: validation must reject the call before using it
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    return av.lib()


def test_route_rejections(L):
    def f(logits=P, dt=av.BF16, tokens=8, experts=16, ld=16, topk=4, renorm=1, ids=P, w=P):
        return L.averis_moe_route(logits, dt, tokens, experts, ld, topk, renorm, ids, w, None)

    def g(logits=P, dt=av.BF16, tokens=8, experts=16, ld=16, topk=4, renorm=1, ids=P, dw=P, dl=P,
          ldd=16):
        return L.averis_moe_route_grad(logits, dt, tokens, experts, ld, topk, renorm, ids, dw, dl,
                                       ldd, None)
    for c in (f, g):
        assert c(dt=5) == 3
        assert c(experts=0) == 6
        assert c(experts=1025, ld=1025) == 6                # AVERIS_MAX_EXPERTS
        assert c(topk=0) == 6
        assert c(topk=17) == 6                              # more choices than experts
        assert c(topk=33, experts=64, ld=64) == 6           # AVERIS_MAX_TOPK
        assert c(tokens=-1) == 2
        assert c(tokens=1 << 30) == 2                       # 2^32 slots
        assert c(ld=15) == 2
        assert c(renorm=2) == 6
        assert c(logits=None) == 1
        assert c(ids=None) == 1
        assert c(logits=P + 1) == 4
        assert c(ids=P + 2) == 4
    assert f(w=None) == 1
    assert f(w=P + 2) == 4
    assert g(dw=None) == 1
    assert g(dl=None) == 1
    assert g(ldd=15) == 2
    assert g(dl=P + 1) == 4


def test_sort_rejections(L):
    def f(ids=P, tokens=8, topk=4, experts=16, offs=P, pos=P, src=P, ws=P, wsb=0):
        return L.averis_moe_sort(ids, tokens, topk, experts, offs, pos, src, ws, wsb, None)
    assert f(ids=None) == 1
    assert f(pos=None) == 1
    assert f(offs=None) == 1
    assert f(offs=P + 4) == 4
    assert f(ids=P + 2) == 4
    assert f(pos=P + 2) == 4
    assert f(src=P + 2) == 4
    assert f(experts=0) == 6
    assert f(experts=1025) == 6
    assert f(topk=0) == 6
    assert f(tokens=-1) == 2
    assert f(tokens=1 << 29, topk=8) == 2
    assert f(tokens=1 << 20, ws=None) == 5
    assert f(tokens=1 << 20, wsb=64) == 5
    need = av.workspace_bytes(av.OP_MOE_SORT, 4 << 20, 0, 16)
    assert need >= (4 << 20) // 2048 * 17 * 4
    assert f(tokens=1 << 20, ws=P + 16, wsb=need) == 4
    assert av.workspace_bytes(av.OP_MOE_SORT, 100, 0, 16) == 0
    assert av.workspace_bytes(av.OP_MOE_SORT, 4 << 20, 0, 2000) == 0


def test_exchange_rejections(L):
    def disp(x=P, dt=av.BF16, tokens=8, cols=32, ldx=32, pos=P, topk=4, rows=P, ldr=32):
        return L.averis_moe_dispatch(x, dt, tokens, cols, ldx, pos, topk, rows, ldr, None)

    def comb(x=P, dt=av.BF16, tokens=8, cols=32, ldx=32, pos=P, topk=4, rows=P, ldr=32, w=P):
        return L.averis_moe_combine(rows, dt, tokens, cols, ldr, pos, w, topk, x, ldx, None)

    def grad(x=P, dt=av.BF16, tokens=8, cols=32, ldx=32, pos=P, topk=4, rows=P, ldr=32, w=P, dr=P,
             lddr=32, dw=P):
        return L.averis_moe_combine_grad(x, dt, tokens, cols, ldx, rows, ldr, pos, w, topk, dr,
                                         lddr, dw, None)
    for c in (disp, comb, grad):
        assert c(dt=9) == 3
        assert c(tokens=-1) == 2
        assert c(cols=0) == 2
        assert c(topk=0) == 6
        assert c(topk=33) == 6
        assert c(tokens=1 << 30) == 2
        assert c(ldx=31) == 2
        assert c(ldr=31) == 2
        assert c(x=None) == 1
        assert c(rows=None) == 1
        assert c(pos=None) == 1
        assert c(x=P + 1) == 4
        assert c(rows=P + 1) == 4
        assert c(pos=P + 2) == 4
        assert c(dt=av.F32, x=P + 2) == 4
    assert comb(w=P + 2) == 4
    assert grad(w=None) == 1
    assert grad(dr=None) == 1
    assert grad(lddr=31) == 2
    assert grad(dw=None) == 1
    assert grad(dw=P + 2) == 4


def test_clip_rejections(L):
    def call(n=2, max_norm=1.0, eps=1e-6, norm=P, ws=P, wsb=1 << 20, arr=True, **bad):
        a = (av._Grad * 2)()
        for i in range(2):
            e = dict(grad=P, out=P, numel=100, dtype=av.BF16)
            if i == 1:
                e.update(bad)
            a[i] = av._Grad(e["grad"], e["out"], e["numel"], e["dtype"])
        p = ctypes.cast(a, ctypes.c_void_p) if arr else None
        r = L.averis_grad_clip(n, p, max_norm, eps, norm, ws, wsb, None)
        if "out" not in bad and max_norm == 1.0 and eps == 1e-6:   # the norm alone: the same checks
            assert L.averis_grad_norm(n, p, norm, ws, wsb, None) == r
        return r
    assert call(n=-1) == 6
    assert call(n=(1 << 20) + 1) == 6
    assert call(arr=False) == 1
    assert call(norm=None) == 1
    assert call(norm=P + 2) == 4
    assert call(max_norm=-1.0) == 6
    assert call(max_norm=NAN) == 6
    assert call(eps=-1.0) == 6
    assert call(dtype=7) == 3
    assert call(numel=-1) == 2
    assert call(numel=1 << 41) == 2
    assert call(grad=None) == 1
    assert call(grad=P + 1) == 4
    assert call(out=None) == 1
    assert call(out=P + 1) == 4
    assert call(ws=None) == 5
    assert call(wsb=1024) == 5
    assert call(ws=P + 16) == 4
    wb = av.workspace_bytes
    assert wb(av.OP_GRAD_NORM, 0, 0, 0) > 0
    assert wb(av.OP_GRAD_NORM, 0, 0, 300) > wb(av.OP_GRAD_NORM, 0, 0, 100)
    assert wb(av.OP_GRAD_NORM, 0, 0, -1) == 0


def test_binding_checks_tensors():
    """The binding refuses tensors of another type, shape, layout or device
    before their addresses go anywhere."""
    l = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    rows, pos = torch.zeros(8, 16), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        av.averis_moe_route_grad(l, ids.long(), w)
    with pytest.raises(ValueError):
        av.averis_moe_route_grad(l, ids, w[:3])
    with pytest.raises(ValueError):
        av.averis_moe_route_grad(l, ids[:3], w)
    with pytest.raises(ValueError):
        av.averis_moe_sort(ids.t(), 8)
    with pytest.raises(ValueError):
        av.averis_moe_dispatch(rows, pos)                      # 8 rows for 4 tokens
    with pytest.raises(ValueError):
        av.averis_moe_combine(rows[:7], pos)
    with pytest.raises(ValueError):
        av.averis_moe_combine(rows.t().contiguous().t(), pos)  # column-major
    with pytest.raises(ValueError):
        av.averis_moe_combine(rows, pos, w.double())
    with pytest.raises(ValueError):
        av.averis_moe_combine_grad(torch.zeros(4, 16).bfloat16(), rows, pos, w)
    with pytest.raises(TypeError):
        av.averis_moe_route(l.double(), 2)
    for call in (lambda: av.averis_moe_route(l, 2), lambda: av.averis_moe_route_grad(l, ids, w),
                 lambda: av.averis_moe_sort(ids, 8), lambda: av.averis_moe_dispatch(rows[:4], pos),
                 lambda: av.averis_moe_combine(rows, pos),
                 lambda: av.averis_moe_combine_grad(rows[:4], rows, pos, w),
                 lambda: av.averis_grad_clip([l], 1.0), lambda: av.averis_grad_norm([l])):
        with pytest.raises(ValueError, match="current GPU"):   # host memory
            call()
    with pytest.raises(ValueError):
        av.averis_grad_clip([l, l.t()], 1.0)
    with pytest.raises(ValueError):
        av.averis_grad_clip([l], 1.0, out=[])
    with pytest.raises(ValueError):
        av.averis_grad_clip([l], 1.0, out=[l.bfloat16()])
    with pytest.raises(TypeError):
        av.averis_grad_norm([l.double()])
