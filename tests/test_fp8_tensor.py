"""What the fp8 calls hand to the library for a tensor of codes and scales (a
stub in place of the library: no GPU needed)."""

import copy
import pickle

import pytest
import torch

from mean_residual_quantized_amd import averis as av

REAL = av.lib


@pytest.fixture
def sent(monkeypatch):
    """The descriptors of the last product."""
    got = []

    class Stub:
        def __getattr__(self, name):
            if name in ("averis_workspace_bytes", "averis_fp8_seg_cols"):
                return getattr(REAL(), name)

            def call(*args):
                got[:] = [(a.codes, a.scales, a.rows, a.cols) for a in args if isinstance(a, av._FP8)]
                return 0
            return call
    monkeypatch.setattr(av, "lib", lambda: Stub())
    monkeypatch.setattr(av, "_stream_on", lambda t: None)
    return got


def describe(q):
    return q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols


@pytest.mark.parametrize("call", [av.averis_fp8_gemm, av.averis_fp8_gemm_wgrad])
def test_replaced_codes_and_scales_are_the_ones_used(sent, call):
    a, b = av.FP8.empty(4, 200, "cpu"), av.FP8.empty(8, 200, "cpu")
    call(a, b)
    assert sent == [describe(a), describe(b)]
    a.codes, b.scales = a.codes.clone(), b.scales.clone()
    call(a, b)
    assert sent == [describe(a), describe(b)]
    a.scales.data = a.scales.clone()          # the same tensor, its memory elsewhere
    call(a, b)
    assert sent == [describe(a), describe(b)]


def test_replacements_are_checked():
    q = av.FP8.empty(4, 200, "cpu")
    for bad in (q.codes[:3], q.codes.int(), torch.zeros(4, 512, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError):
            q.codes = bad
    for bad in (q.scales[:3], q.scales.int(), torch.zeros(4, 8, dtype=torch.uint8)[:, :4]):
        with pytest.raises(ValueError):
            q.scales = bad
    for field in ("rows", "cols"):
        with pytest.raises(AttributeError):
            setattr(q, field, 100)
    assert (q.rows, q.cols) == (4, 200)


def test_codes_and_scales_on_one_device(sent):
    """(meta stands for another device than the CPU.)"""
    q, far = av.FP8.empty(4, 200, "cpu"), av.FP8.empty(4, 200, "meta")
    with pytest.raises(ValueError, match="one device"):
        av.FP8(q.codes, far.scales, 4, 200)
    half = av.FP8.empty(4, 200, "cpu")
    half.scales = far.scales
    for call in (av.averis_fp8_gemm, av.averis_fp8_gemm_wgrad):
        for a, b in ((half, q), (q, half), (q, far), (far, q)):
            with pytest.raises(ValueError, match="one device"):
                call(a, b)
    assert sent == []


def test_copies(sent):
    q = av.FP8.empty(4, 200, "cpu")
    q.codes.fill_(3)
    q.scales.fill_(5)
    shallow, deep, loaded = copy.copy(q), copy.deepcopy(q), pickle.loads(pickle.dumps(q))
    assert describe(shallow) == describe(q)
    for other in (deep, loaded):
        assert (other.rows, other.cols) == (4, 200) and describe(other)[0] != describe(q)[0]
        assert torch.equal(other.codes, q.codes) and torch.equal(other.scales, q.scales)
        av.averis_fp8_gemm(other, q)
        assert sent == [describe(other), describe(q)]


@pytest.mark.parametrize("shape,strides", [((1, 40), (1, 1)), ((1, 1), (7, 9)), ((40, 1), (3, 5)), ((5, 40), (48, 1)),
                                           ((1, 1, 40), (2, 1, 1)), ((2, 1, 40), (64, 1, 1)), ((2, 3, 1), (9, 3, 2))])
def test_weight_of_one_row_or_column(monkeypatch, shape, strides):
    """A dimension of one element has no stride that matters."""
    sent = []

    class Stub:
        @staticmethod
        def averis_fp8_quant_weight(w, dtype, batch, rows, cols, ld, batch_stride, out, out_t, stream):
            sent.append((batch, rows, cols, ld, batch_stride))
            return 0
    monkeypatch.setattr(av, "lib", lambda: Stub)
    monkeypatch.setattr(av, "_stream_on", lambda t: None)
    w = torch.zeros(4096).as_strided(shape, strides)
    av.averis_fp8_quant_weight(w)
    (batch, rows, cols, ld, batch_stride), = sent
    assert (batch, rows, cols) == ((1,) * (3 - len(shape)) + shape)
    assert ld >= cols and (batch == 1 or batch_stride >= rows * ld)
    if rows > 1:
        assert ld == strides[-2]
    if batch > 1:
        assert batch_stride == strides[0]
