"""Rejections of the fp8 calls: refused before any HIP call (no GPU needed)."""

import ctypes

import pytest
import torch

from mean_residual_quantized_amd import averis as av

P = 0x10000   # stand-in device address: validation must reject the call before using it


@pytest.fixture(scope="module")
def L():
    return av.lib()


def f8(rows, cols, codes=P, scales=P):
    return av._FP8(codes, scales, rows, cols)


def ref(t):
    return ctypes.byref(t) if t is not None else None


def test_quant_rejections(L):
    def q(a=P, dt=av.BF16, rows=64, cols=100, lda=100, offs=None, nseg=1, out=f8(64, 100),
          out_t=f8(100, 64)):
        return L.averis_fp8_quant(a, dt, rows, cols, lda, offs, nseg, ref(out), ref(out_t), None)
    assert q(dt=4) == 3
    assert q(rows=-1) == 2
    assert q(cols=0, lda=0) == 2
    assert q(lda=99) == 2
    assert q(a=None) == 1
    assert q(a=P + 1) == 4
    assert q(dt=av.F32, a=P + 2) == 4
    assert q(out=None, out_t=None) == 1
    assert q(out=f8(64, 99)) == 2
    assert q(out_t=f8(64, 100)) == 2                       # not transposed
    assert q(out=f8(64, 100, codes=P + 8)) == 4
    assert q(out=f8(64, 100, scales=P + 2)) == 4
    assert q(out=f8(64, 100, codes=None)) == 1
    assert q(nseg=2) == 6                                  # segments without offsets
    assert q(offs=P, nseg=0) == 6
    assert q(offs=P, nseg=5000) == 6
    assert q(offs=P + 4, nseg=2) == 4
    assert q(offs=P, nseg=2) == 2                          # out_t without room for the segments
    assert L.averis_fp8_seg_cols(64, 2) == 3 * 128
    assert L.averis_fp8_seg_cols(64, 1) == 128
    assert L.averis_fp8_seg_cols(0, 3) == 3 * 128
    assert L.averis_fp8_seg_cols(-1, 3) == -1
    assert L.averis_fp8_seg_cols(64, 0) == -1


def test_quant_weight_rejections(L):
    def q(w=P, dt=av.BF16, batch=2, rows=64, cols=100, ld=100, bs=6400, out=f8(128, 100),
          out_t=f8(200, 64)):
        return L.averis_fp8_quant_weight(w, dt, batch, rows, cols, ld, bs, ref(out), ref(out_t),
                                         None)
    assert q(dt=4) == 3
    assert q(batch=0) == 6
    assert q(rows=0) == 2
    assert q(cols=0) == 2
    assert q(ld=99) == 2
    assert q(bs=6399) == 2                                 # overlapping matrices
    assert q(w=None) == 1
    assert q(w=P + 1) == 4
    assert q(out=None, out_t=None) == 1
    assert q(out=f8(64, 100)) == 2
    assert q(out_t=f8(100, 64)) == 2


def test_gemm_rejections(L):
    def g(a=f8(64, 256), b=f8(96, 256), offs=None, nseg=1, c=P, dt=av.BF16, ldc=96, ws=P, wsb=1 << 30):
        return L.averis_fp8_gemm(ref(a), ref(b), offs, nseg, c, dt, ldc, ws, wsb, None)
    assert g(a=None) == 1
    assert g(b=None) == 1
    assert g(b=f8(96, 255)) == 2
    assert g(a=f8(64, 0), b=f8(96, 0)) == 2
    assert g(a=f8(-1, 256)) == 2
    assert g(a=f8(64, 256, codes=P + 4)) == 4
    assert g(b=f8(96, 256, scales=None)) == 1
    assert g(offs=P, nseg=5) == 2                          # 96 rows are no five matrices
    assert g(offs=P + 4, nseg=2, ldc=48) == 4
    assert g(nseg=2) == 6
    assert g(c=None) == 1
    assert g(c=P + 1) == 4
    assert g(dt=3) == 3
    assert g(ldc=95) == 2
    assert g(ws=P + 16) == 4
    big = dict(a=f8(1024, 1 << 14), b=f8(1024, 1 << 14), ldc=1024)
    need = av.workspace_bytes(av.OP_FP8_GEMM, 1024, 1 << 14, 1024)
    assert need >= 2 * 1024 * 1024 * 4                     # the contraction is split
    assert g(ws=None, **big) == 5
    assert g(wsb=need - 1, **big) == 5


def test_wgrad_rejections(L):
    def g(x=f8(64, 300), d=f8(96, 300), rows=300, offs=None, nseg=1, c=P, dt=av.BF16, ld=96, ws=P,
          wsb=1 << 30):
        return L.averis_fp8_gemm_wgrad(ref(x), ref(d), rows, offs, nseg, c, dt, ld, ws, wsb, None)
    assert g(x=None) == 1
    assert g(d=f8(96, 299)) == 2
    assert g(rows=299) == 2
    assert g(rows=-1) == 2
    assert g(offs=P, nseg=2) == 2                          # not the segments' columns
    assert g(nseg=2) == 6
    assert g(offs=P + 4, nseg=2) == 4
    assert g(c=None) == 1
    assert g(dt=8) == 3
    assert g(ld=95) == 2
    assert g(ws=P + 8) == 4
    need = av.workspace_bytes(av.OP_FP8_WGRAD, 1024, 1 << 14, 1024)
    big = dict(x=f8(1024, 1 << 14), d=f8(1024, 1 << 14), rows=1 << 14, ld=1024)
    assert need > 0 and g(wsb=need - 1, **big) == 5


def test_binding_checks_tensors():
    a = torch.zeros(4, 8)
    q = av.FP8.empty(4, 200, "cpu")
    assert q.codes.shape == (4, 256) and q.scales.shape == (4, 4)
    with pytest.raises(ValueError):
        av.FP8(q.codes[:, :200], q.scales, 4, 200)
    with pytest.raises(ValueError):
        av.FP8(q.codes, q.scales[:2], 4, 200)
    with pytest.raises(ValueError):
        av.FP8(q.codes.int(), q.scales, 4, 200)
    with pytest.raises(ValueError, match="current GPU"):
        av.averis_fp8_quant(a)                             # host memory
    with pytest.raises(ValueError, match="column stride"):
        av.averis_fp8_quant(a.t())
    with pytest.raises(ValueError):
        av.averis_fp8_quant(a, transposed=True, offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        av.averis_fp8_quant_weight(a.t())
    with pytest.raises(TypeError):
        av.averis_fp8_quant(a.double())
    with pytest.raises(ValueError):
        av.averis_fp8_gemm(q, q, out=torch.zeros(4, 5))
    with pytest.raises(ValueError):
        av.averis_fp8_gemm_wgrad(q, q, out=torch.zeros(4, 8)[:, :4])
