"""Pins of oracle/fp8.py: torch's E4M3 cast, scales at the binade edges, exact
round trips, and that a linear step's three products fit together."""

import numpy as np
import pytest
import torch

from oracle import fp8


def torch_codes(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def test_codes_are_torchs_cast():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(fp8.decode(codes), t)
    fin = t[np.isfinite(t)]
    mid = (np.sort(fin)[1:] + np.sort(fin)[:-1]) / 2          # every tie
    rng = np.random.default_rng(0)
    v = np.concatenate([fin, mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9),
                        np.clip(rng.standard_normal(100000) * np.exp(3 * rng.standard_normal(100000)),
                                -448, 448)])
    v = np.clip(v, -448, 448).astype(np.float32)
    np.testing.assert_array_equal(fp8.encode(v), torch_codes(v))


def test_exponent_edges():
    assert fp8.exponent(0.0) == -127
    assert fp8.exponent(448.0) == 0
    assert fp8.exponent(np.nextafter(448.0, 1e9)) == 1
    assert fp8.exponent(224.0) == -1
    assert fp8.exponent(1.0) == -8                # 448 / 256 = 1.75
    assert fp8.exponent(1.75) == -8
    assert fp8.exponent(1.75 + 2 ** -20) == -7
    assert fp8.exponent(2.0 ** -149) == -127
    assert fp8.exponent(float(np.finfo(np.float32).max)) == 120
    for k in range(-126, 128):
        assert fp8.exponent(2.0 ** k) == max(-127, k - 8)


@pytest.mark.parametrize("tile", [False, True])
def test_round_trip_of_exact_values(tile):
    rng = np.random.default_rng(1)
    v = rng.choice(fp8.GRID, (200, 300)) * rng.choice([-1, 1], (200, 300))
    v[:, ::64] = 448.0                             # every block's scale is 1
    codes, scales = fp8.quantize(v, tile)
    assert (scales == 127).all()
    np.testing.assert_array_equal(fp8.dequantize(codes, scales), v)
    codes, scales = fp8.quantize(v * 2.0 ** -30, tile)
    np.testing.assert_array_equal(fp8.dequantize(codes, scales), v * 2.0 ** -30)


def test_relative_error_and_nan_blocks():
    rng = np.random.default_rng(2)
    a = rng.standard_normal((64, 500))
    q = fp8.dequantize(*fp8.quantize(a))
    # half a step of 2^-3 relative for normal codes, 2^-10 of the block's scale below
    amax = np.repeat(np.stack([np.abs(a[:, i:i + 128]).max(1) for i in range(0, 500, 128)], 1), 128, 1)[:, :500]
    assert np.all(np.abs(q - a) <= np.maximum(np.abs(a) / 16, amax / 224 * 2.0 ** -10))
    a[3, 130] = np.inf
    a[4, 0] = np.nan
    codes, scales = fp8.quantize(a)
    assert (codes[3, 128:256] == 0x7F).all() and scales[3, 1] == 127 and np.isfinite(fp8.decode(codes[3, :128])).all()
    assert (codes[4, :128] == 0x7F).all()


def test_tiles_transpose():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((300, 200))
    c, s = fp8.quantize(w, True)
    ct, st = fp8.quantize(w.T, True)
    np.testing.assert_array_equal(fp8.dequantize(c, s), fp8.dequantize(ct, st).T)


def test_linear_gradients_are_the_products():
    """With y = x w: the loss <d, y> has the gradients d w^T and x^T d (a
    difference of a bilinear form is exact)."""
    rng = np.random.default_rng(4)
    x, w, d = rng.standard_normal((9, 5)), rng.standard_normal((5, 7)), rng.standard_normal((9, 7))
    dx, dw = d @ w.T, x.T @ d
    for i, j in ((0, 0), (8, 4), (3, 2)):
        p = x.copy()
        p[i, j] += 1.0
        assert abs(np.sum(d * (p @ w)) - np.sum(d * (x @ w)) - dx[i, j]) < 1e-12
    for i, j in ((0, 0), (4, 6), (2, 3)):
        p = w.copy()
        p[i, j] += 1.0
        assert abs(np.sum(d * (x @ p)) - np.sum(d * (x @ w)) - dw[i, j]) < 1e-12


def test_segment_starts():
    assert fp8.seg_starts(np.array([0, 1, 1, 130, 258])).tolist() == [0, 128, 128, 384, 512]
