"""Sizes past the limits of the fp8 calls are refused as shapes, before any HIP
call (no GPU needed)."""

import ctypes

import pytest

from mean_residual_quantized_amd import averis as av

P = 0x10000   # stand-in device address: validation must reject the call before using it


@pytest.fixture(scope="module")
def L():
    return av.lib()


def f8(rows, cols):
    return ctypes.byref(av._FP8(P, P, rows, cols))


def test_quant(L):
    def q(rows, cols, t):
        return L.averis_fp8_quant(P, av.BF16, rows, cols, cols, None, 1, f8(rows, cols), f8(cols, rows) if t else None, None)
    assert q((1 << 30) + 1, 1, False) == 2
    assert q(1, (1 << 30) + 1, False) == 2
    assert q(1 << 30, 1, True) == 2                         # 2^23 tiles
    assert q(1 << 21, 1 << 16, True) == 2


def test_gemm(L):
    def g(m, n, k, nseg=1):
        return L.averis_fp8_gemm(f8(m, k), f8(nseg * n, k), P if nseg > 1 else None, nseg, P, av.BF16, n, P, 1 << 40, None)
    assert g((1 << 30) + 1, 1, 128) == 2
    assert g(1, (1 << 30) + 1, 128) == 2
    assert g(16, 16, (1 << 22) + 1) == 2
    assert g(1 << 23, 1 << 22, 128) == 2                    # 2^31 tiles
    assert g(1 << 23, 1 << 22, 128, 4) == 2


def test_wgrad(L):
    def g(m, n, rows, nseg=1):
        cols = L.averis_fp8_seg_cols(rows, nseg) if nseg > 1 else rows
        return L.averis_fp8_gemm_wgrad(f8(m, cols), f8(n, cols), rows, P if nseg > 1 else None, nseg, P, av.BF16, n, P,
                                       1 << 40, None)
    assert g((1 << 30) + 1, 1, 128) == 2
    assert g(1, (1 << 30) + 1, 128) == 2
    assert g(16, 16, (1 << 22) + 1) == 2
    assert g(16, 16, 1 << 22, 4) == 2                       # 2^22 rows and a run a segment
    assert g(1 << 23, 1 << 22, 128) == 2                    # 2^31 tiles
    assert g(1 << 19, 1, 0, 4096) == 2                      # 2^24 workgroups
    assert g(1, 1 << 19, 0, 4096) == 2
