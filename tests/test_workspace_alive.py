"""A workspace that the binding makes lives until the library call that uses it
has returned (a stub in place of the library: no GPU needed)."""

import ctypes
import gc
import weakref

import pytest
import torch

from mean_residual_quantized_amd import averis as av

REAL = av.lib


class Stub:
    """The library, whose calls with a workspace only note whether it is alive."""

    def __init__(self):
        self.made, self.alive = [], []

    def __getattr__(self, name):
        real = getattr(REAL(), name)
        if name in ("averis_workspace_bytes", "averis_status_str", "averis_fp8_seg_cols"):
            return real

        def call(*args):
            gc.collect()
            assert self.made, "%s: no workspace was made" % name
            addresses = [a.value if isinstance(a, ctypes.c_void_p) else a for a in args]
            for r in self.made:
                t = r()
                self.alive.append(t is not None and t.data_ptr() in addresses)
            return 0
        return call


@pytest.fixture
def stub(monkeypatch):
    s = Stub()
    monkeypatch.setattr(av, "lib", lambda: s)
    monkeypatch.setattr(av, "_stream", lambda: None)
    monkeypatch.setattr(av, "_stream_on", lambda t: None)
    make = av._workspace

    def workspace(nbytes, device):
        t = make(nbytes, "cpu")
        s.made.append(weakref.ref(t))
        return t
    monkeypatch.setattr(av, "_workspace", workspace)
    return s


def fp8(rows, cols):
    return av.FP8.empty(rows, cols, "cpu")


def nvfp4(rows, cols, nseg=1):
    return av.NVFP4.empty(rows, cols, nseg, "cpu")


X = torch.zeros(64, 64)
OFFS = torch.tensor([0, 32, 64])

CALLS = {
    "averis_fp8_gemm": lambda: av.averis_fp8_gemm(fp8(1024, 1 << 14), fp8(1024, 1 << 14)),
    "averis_fp8_gemm_wgrad": lambda: av.averis_fp8_gemm_wgrad(fp8(1024, 1 << 14), fp8(1024, 1 << 14)),
    "averis_moe_sort": lambda: av.averis_moe_sort(torch.zeros(5000, 4, dtype=torch.int32), 16),
    "averis_grad_norm": lambda: av.averis_grad_norm([X]),
    "averis_grad_clip": lambda: av.averis_grad_clip([X], 1.0),
    "averis_split_quant": lambda: av.averis_split_quant(X),
    "averis_split_quant_grouped": lambda: av.averis_split_quant_grouped(X, OFFS),
    "averis_quant": lambda: av.averis_quant(X),
    "averis_quant_batched": lambda: av.averis_quant_batched(X.reshape(2, 32, 64)),
    "averis_quant_grouped": lambda: av.averis_quant_grouped(X, OFFS),
    "averis_quant_pair": lambda: av.averis_quant_pair(X),
    "averis_quant_pair_multi": lambda: av.averis_quant_pair_multi([X, X]),
    "averis_quant_pair_2d": lambda: av.averis_quant_pair_2d(X),
    "averis_split_quant_ratio": lambda: av.averis_split_quant_ratio(X),
    "averis_split_quant_rank1": lambda: av.averis_split_quant_rank1(X, nvfp4(64, 64)),
    "averis_split_quant_rank1_multi": lambda: av.averis_split_quant_rank1_multi(X, [nvfp4(64, 64)]),
    "averis_split_quant_grouped_rank1": lambda: av.averis_split_quant_grouped_rank1(
        X, OFFS, nvfp4(128, 64, 2)),
    "averis_gemm_rank1_stats": lambda: av.averis_gemm_rank1_stats(nvfp4(64, 64), torch.zeros(64),
                                                                  nvfp4(64, 64)),
    "averis_gemm_wgrad": lambda: av.averis_gemm_wgrad(nvfp4(64, 64), nvfp4(64, 64), torch.zeros(64),
                                                      torch.zeros(64)),
    "averis_gemm_fwd": lambda: av.averis_gemm_fwd(nvfp4(64, 64), nvfp4(1, 64), nvfp4(64, 64)),
    "averis_gemm_dgrad": lambda: av.averis_gemm_dgrad(nvfp4(64, 64), nvfp4(1, 64), nvfp4(64, 64)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_workspace_lives_through_the_call(stub, name):
    CALLS[name]()
    assert stub.alive and all(stub.alive)


GIVEN = {
    "averis_fp8_gemm": lambda ws: av.averis_fp8_gemm(fp8(1024, 1 << 14), fp8(1024, 1 << 14), ws=ws),
    "averis_fp8_gemm_wgrad": lambda ws: av.averis_fp8_gemm_wgrad(fp8(1024, 1 << 14), fp8(1024, 1 << 14), ws=ws),
    "averis_moe_sort": lambda ws: av.averis_moe_sort(torch.zeros(5000, 4, dtype=torch.int32), 16, ws=ws),
    "averis_grad_norm": lambda ws: av.averis_grad_norm([X], ws=ws),
    "averis_grad_clip": lambda ws: av.averis_grad_clip([X], 1.0, ws=ws),
}


@pytest.mark.parametrize("name", sorted(GIVEN))
def test_given_workspace_is_checked(stub, name):
    """The caller's workspace: contiguous memory where the other tensors are
    (meta stands for another device), or a refusal before the library call."""
    flat = torch.zeros(1 << 20, dtype=torch.uint8)
    stub.made.append(weakref.ref(flat))
    for bad in (flat.to("meta"), flat[::2], flat[:1].expand(1 << 20)):
        with pytest.raises(ValueError, match="ws"):
            GIVEN[name](bad)
    assert not stub.alive
    GIVEN[name](flat)
    assert stub.alive == [True]
