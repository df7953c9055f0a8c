"""Thin ctypes binding of libaveris (include/averis.h), same names as the C ABI.

Argument marshalling only: torch supplies device memory (outputs and
workspace are allocated with torch.empty) and the current HIP stream; every
step of the computation runs in the library's kernels.  The library must be
built (``python -m mean_residual_quantized_amd.build``); if it is missing,
loading fails with an error -- there is no fallback.
"""

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libaveris.so")

AVERIS_OK = 0
STATUS_NAMES = {0: "OK", 1: "E_NULL", 2: "E_SHAPE", 3: "E_DTYPE", 4: "E_ALIGN",
                5: "E_WORKSPACE", 6: "E_ARG", 7: "E_HIP"}
F32, BF16 = 0, 1
RN, SR = 0, 1
OP_SPLIT_QUANT, OP_QUANT, OP_GEMM, OP_WGRAD, OP_QUANT_PAIR_MULTI = 0, 1, 2, 3, 4
OP_MOE_SORT, OP_GRAD_NORM, OP_FP8_GEMM, OP_FP8_WGRAD = 5, 6, 7, 8
MAX_WEIGHTS = 16
MAX_RANK1 = 4
MAX_EXPERTS, MAX_TOPK, MAX_GRADS = 1024, 32, 1 << 20
STREAM_ACT, STREAM_MEAN, STREAM_WEIGHT, STREAM_RESIDUAL_T = 0, 1, 2, 3

# every symbol include/averis.h declares
EXPORTS = [
    "averis_split_quant", "averis_split_quant_grouped", "averis_quant", "averis_quant_batched",
    "averis_quant_grouped", "averis_quant_pair", "averis_quant_pair_2d",
    "averis_quant_pair_multi", "averis_gemm_fwd", "averis_gemm_dgrad",
    "averis_gemm_vanilla", "averis_gemm_grouped", "averis_residual_t_quant", "averis_gemm_wgrad",
    "averis_split_quant_ratio", "averis_split_quant_rank1", "averis_split_quant_rank1_multi",
    "averis_gemm_rank1",
    "averis_split_quant_grouped_rank1", "averis_gemm_grouped_rank1",
    "averis_split_quant_noalloc", "averis_gemm_rank1_stats", "averis_split_quant_from_stats",
    "averis_moe_route", "averis_moe_route_grad", "averis_moe_sort", "averis_moe_dispatch",
    "averis_moe_combine", "averis_moe_combine_grad", "averis_grad_norm", "averis_grad_clip",
    "averis_fp8_seg_cols", "averis_fp8_quant", "averis_fp8_quant_weight", "averis_fp8_gemm",
    "averis_fp8_gemm_wgrad",
    "averis_workspace_bytes", "averis_status_str",
    "averis_abi_version", "averis_last_error",
]


class AverisError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__("%s failed: %s (%s)" % (fn, STATUS_NAMES.get(status, status), msg))
        self.status = status


class _NVFP4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tscale", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _Weight(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("out", ctypes.POINTER(_NVFP4)), ("out_t", ctypes.POINTER(_NVFP4))]


class _FP8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _Grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


_lib = None


def lib():
    """Load libaveris.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libaveris.so not built at %s; run "
                               "`python -m mean_residual_quantized_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I64, U64, I, U32, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int,
                                   ctypes.c_uint32, ctypes.c_size_t)
        T, F8 = ctypes.POINTER(_NVFP4), ctypes.POINTER(_FP8)
        sig = {
            "averis_split_quant": [P, I, I64, I64, I64, U64, I, T, T, P, P, SZ, P],
            "averis_split_quant_grouped": [P, I, I64, I64, I64, P, I, U64, I, T, T, P, P, SZ, P],
            "averis_quant": [P, I, I64, I64, I64, I, U64, I, U32, T, P, SZ, P],
            "averis_quant_batched": [P, I, I, I64, I64, I64, I64, I, U64, I, U32, T, P, SZ, P],
            "averis_quant_grouped": [P, I, I64, I64, I64, P, I, U64, I, U32, T, P, SZ, P],
            "averis_quant_pair": [P, I, I, I64, I64, I64, I64, U64, I, U32, T, T, P, SZ, P],
            "averis_quant_pair_2d": [P, I, I, I64, I64, I64, I64, U64, I, U32, T, T, P, SZ, P],
            "averis_quant_pair_multi": [I, P, I, I, U32, P, SZ, P],
            "averis_gemm_fwd": [T, T, T, P, I, I64, P, SZ, P],
            "averis_gemm_dgrad": [T, T, T, P, I, I64, P, SZ, P],
            "averis_gemm_vanilla": [T, T, P, I, I64, P, SZ, P],
            "averis_gemm_grouped": [T, T, T, P, I, P, I, I64, P, SZ, P],
            "averis_residual_t_quant": [P, I, I64, I64, I64, P, P, U64, I, T, P],
            "averis_gemm_wgrad": [T, T, P, P, P, I, I64, P, SZ, P],
            "averis_split_quant_ratio": [P, I, I64, I64, I64, P, I, U64, I, T, T, P, P, P, SZ, P],
            "averis_split_quant_rank1": [P, I, I64, I64, I64, U64, I, T, T, P, T, P, P, SZ, P],
            "averis_gemm_rank1": [T, P, T, P, I, I64, P],
            "averis_split_quant_rank1_multi": [P, I, I64, I64, I64, U64, I, T, T, P, I, P, P, P,
                                               SZ, P],
            "averis_split_quant_grouped_rank1": [P, I, I64, I64, I64, P, I, U64, I, T, T, P, T, P,
                                                 P, SZ, P],
            "averis_gemm_grouped_rank1": [T, P, T, P, I, P, I, I64, P],
            "averis_split_quant_noalloc": [P, I, I64, I64, I64, U64, I, T, T, P, P],
            "averis_gemm_rank1_stats": [T, P, T, P, I64, P, SZ, P],
            "averis_split_quant_from_stats": [P, I64, I64, I64, U64, I, T, T, P, T, P, P, SZ, P],
            "averis_moe_route": [P, I, I64, I, I64, I, I, P, P, P],
            "averis_moe_route_grad": [P, I, I64, I, I64, I, I, P, P, P, I64, P],
            "averis_moe_sort": [P, I64, I, I, P, P, P, P, SZ, P],
            "averis_moe_dispatch": [P, I, I64, I64, I64, P, I, P, I64, P],
            "averis_moe_combine": [P, I, I64, I64, I64, P, P, I, P, I64, P],
            "averis_moe_combine_grad": [P, I, I64, I64, I64, P, I64, P, P, I, P, I64, P, P],
            "averis_fp8_quant": [P, I, I64, I64, I64, P, I, F8, F8, P],
            "averis_fp8_quant_weight": [P, I, I, I64, I64, I64, I64, F8, F8, P],
            "averis_fp8_gemm": [F8, F8, P, I, P, I, I64, P, SZ, P],
            "averis_fp8_gemm_wgrad": [F8, F8, I64, P, I, P, I, I64, P, SZ, P],
            "averis_grad_norm": [I, P, P, P, SZ, P],
            "averis_grad_clip": [I, P, ctypes.c_double, ctypes.c_double, P, P, SZ, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.averis_workspace_bytes.argtypes = [I, I64, I64, I64, I64]
        L.averis_workspace_bytes.restype = SZ
        L.averis_fp8_seg_cols.argtypes = [I64, I64]
        L.averis_fp8_seg_cols.restype = I64
        L.averis_status_str.argtypes = [I]
        L.averis_status_str.restype = ctypes.c_char_p
        L.averis_abi_version.argtypes = []
        L.averis_abi_version.restype = I
        L.averis_last_error.argtypes = []
        L.averis_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(fn, status):
    if status != AVERIS_OK:
        msg = lib().averis_status_str(status).decode()
        if status == 7:
            msg += ": " + lib().averis_last_error().decode()
        raise AverisError(fn, status, msg)


def workspace_bytes(op, rows, cols, n=0, nseg=0):
    return int(lib().averis_workspace_bytes(op, rows, cols, n, nseg))


# --------------------------------------------------------------------------
# tensors
# --------------------------------------------------------------------------

@dataclass
class NVFP4:
    """Device NVFP4-style tensor: codes u8[rows, cols/2], scales u8[rows, cols/16]
    (E4M3), tscale f32[2*nseg] = [S_enc, S_dec] per segment."""
    codes: torch.Tensor
    scales: torch.Tensor
    tscale: torch.Tensor
    rows: int
    cols: int

    @staticmethod
    def empty(rows, cols, nseg=1, device="cuda"):
        return NVFP4(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                     torch.empty((rows, cols // 16), dtype=torch.uint8, device=device),
                     torch.empty((2 * nseg,), dtype=torch.float32, device=device), rows, cols)

    def c(self):
        return _NVFP4(self.codes.data_ptr(), self.scales.data_ptr(), self.tscale.data_ptr(),
                      self.rows, self.cols)

    def cpu(self):
        return dict(codes=self.codes.cpu().numpy(), scales=self.scales.cpu().numpy(),
                    tscale=self.tscale.cpu().numpy())


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("libaveris takes float32 or bfloat16 inputs, got %s" % t.dtype)


def _stream():
    # the raw handle: torch.cuda.current_stream() builds an object around it
    # (2.9 us against 0.2 us, as much as a launch)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _stream_on(t):
    """The current stream, for a call on tensors that are where t is: t must be
    on the current GPU."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("expected tensors on the current GPU, got %s" % t.device)
    return torch._C._cuda_getCurrentRawStream(dev)


def _workspace(nbytes, device):
    return torch.empty((max(int(nbytes), 1),), dtype=torch.uint8, device=device)


def _lda(a):
    if a.dim() != 2 or a.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return a.stride(0)


# --------------------------------------------------------------------------
# entry points
# --------------------------------------------------------------------------

def averis_split_quant(a, seed=0, rnd=SR, ws=None):
    """Q4(a - 1 mu) and Q4(mu); returns (residual, mean, mu_f32)."""
    rows, cols = a.shape
    res = NVFP4.empty(rows, cols, 1, a.device)
    mean = NVFP4.empty(1, cols, 1, a.device)
    mu = torch.empty((cols,), dtype=torch.float32, device=a.device)
    need = workspace_bytes(OP_SPLIT_QUANT, rows, cols)
    ws = ws if ws is not None else _workspace(need, a.device)
    r, m = res.c(), mean.c()
    _check("averis_split_quant", lib().averis_split_quant(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), seed, rnd, ctypes.byref(r),
        ctypes.byref(m), mu.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return res, mean, mu


def averis_split_quant_noalloc(a, seed=0, rnd=SR):
    """averis_split_quant with the library's own device array as the
    workspace (no workspace argument); returns (residual, mean, mu_f32)."""
    rows, cols = a.shape
    res = NVFP4.empty(rows, cols, 1, a.device)
    mean = NVFP4.empty(1, cols, 1, a.device)
    mu = torch.empty((cols,), dtype=torch.float32, device=a.device)
    r, m = res.c(), mean.c()
    _check("averis_split_quant_noalloc", lib().averis_split_quant_noalloc(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), seed, rnd, ctypes.byref(r),
        ctypes.byref(m), mu.data_ptr(), _stream()))
    return res, mean, mu


def averis_split_quant_grouped(a, offsets, seed=0, rnd=SR, ws=None):
    """Per-segment split-quant; offsets: int64 device tensor [nseg+1]."""
    rows, cols = a.shape
    nseg = offsets.numel() - 1
    res = NVFP4.empty(rows, cols, nseg, a.device)
    mean = NVFP4.empty(nseg, cols, nseg, a.device)
    mu = torch.empty((nseg, cols), dtype=torch.float32, device=a.device)
    need = workspace_bytes(OP_SPLIT_QUANT, rows, cols, 0, nseg)
    ws = ws if ws is not None else _workspace(need, a.device)
    r, m = res.c(), mean.c()
    _check("averis_split_quant_grouped", lib().averis_split_quant_grouped(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), offsets.data_ptr(), nseg, seed, rnd,
        ctypes.byref(r), ctypes.byref(m), mu.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return res, mean, mu


def averis_quant(a, transpose=False, seed=0, rnd=SR, sr_stream=STREAM_ACT, ws=None, out=None):
    """Plain Q4.  transpose=True quantizes a^T (blocks along a's rows).  out:
    an NVFP4 of the output's shape to write into (else a new one)."""
    srows, scols = a.shape
    rows, cols = (scols, srows) if transpose else (srows, scols)
    out = out if out is not None else NVFP4.empty(rows, cols, 1, a.device)
    need = workspace_bytes(OP_QUANT, rows, cols)
    ws = ws if ws is not None else _workspace(need, a.device)
    o = out.c()
    _check("averis_quant", lib().averis_quant(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), int(transpose), seed, rnd, sr_stream,
        ctypes.byref(o), ws.data_ptr(), ws.numel(), _stream()))
    return out


def averis_quant_batched(a, transpose=False, seed=0, rnd=RN, sr_stream=STREAM_WEIGHT, ws=None):
    """Plain Q4 of each matrix a[b] (3-D tensor), one tensor scale each."""
    batch, srows, scols = a.shape
    if a.stride(2) != 1:
        raise ValueError("expected unit innermost stride")
    rows, cols = (scols, srows) if transpose else (srows, scols)
    out = NVFP4.empty(batch * rows, cols, batch, a.device)
    need = workspace_bytes(OP_QUANT, rows, cols, 0, batch)
    ws = ws if ws is not None else _workspace(need, a.device)
    o = out.c()
    _check("averis_quant_batched", lib().averis_quant_batched(
        a.data_ptr(), _dtype_code(a), batch, rows, cols, a.stride(1), a.stride(0),
        int(transpose), seed, rnd, sr_stream, ctypes.byref(o), ws.data_ptr(), ws.numel(),
        _stream()))
    return out


def averis_quant_pair(w, seed=0, rnd=RN, sr_stream=STREAM_WEIGHT, ws=None):
    """Both quantized copies of a weight in one call: returns (wt, wd) with
    wt = Q4(w^T) (blocks along w's rows; the forward operand) and wd = Q4(w)
    (blocks along w's cols; the dgrad operand).  w: 2-D, or 3-D (batch of
    matrices, one tensor scale each)."""
    a = w if w.dim() == 3 else w.unsqueeze(0)
    batch, rows, cols = a.shape
    if a.stride(2) != 1:
        raise ValueError("expected unit innermost stride")
    wd = NVFP4.empty(batch * rows, cols, batch, w.device)
    wt = NVFP4.empty(batch * cols, rows, batch, w.device)
    need = workspace_bytes(OP_QUANT, rows, cols, 0, batch)
    ws = ws if ws is not None else _workspace(need, w.device)
    o, ot = wd.c(), wt.c()
    _check("averis_quant_pair", lib().averis_quant_pair(
        a.data_ptr(), _dtype_code(a), batch, rows, cols, a.stride(1), a.stride(0), seed, rnd,
        sr_stream, ctypes.byref(o), ctypes.byref(ot), ws.data_ptr(), ws.numel(), _stream()))
    return wt, wd


def averis_quant_pair_multi(ws_list, seeds=None, rnd=RN, sr_stream=STREAM_WEIGHT, ws=None):
    """Both quantized copies of several 2-D weights (one dtype, shapes of their
    own) in two launches: returns [(wt, wd), ...] in order, each as
    averis_quant_pair(w, seed) returns it."""
    n = len(ws_list)
    if not 1 <= n <= MAX_WEIGHTS:
        raise ValueError("expected 1 .. %d weights" % MAX_WEIGHTS)
    seeds = [0] * n if seeds is None else list(seeds)
    dev = ws_list[0].device
    dt = _dtype_code(ws_list[0])
    outs, keep = [], []
    arr = (_Weight * n)()
    for i, w in enumerate(ws_list):
        if w.dim() != 2 or w.stride(1) != 1:
            raise ValueError("expected 2-D weights with unit innermost stride")
        if _dtype_code(w) != dt:
            raise ValueError("expected weights of one dtype")
        rows, cols = w.shape
        wd = NVFP4.empty(rows, cols, 1, dev)
        wt = NVFP4.empty(cols, rows, 1, dev)
        o, ot = wd.c(), wt.c()
        keep += [o, ot]
        arr[i] = _Weight(w.data_ptr(), rows, cols, w.stride(0), seeds[i],
                         ctypes.pointer(o), ctypes.pointer(ot))
        outs.append((wt, wd))
    need = workspace_bytes(OP_QUANT_PAIR_MULTI, 0, 0, n)
    ws = ws if ws is not None else _workspace(need, dev)
    _check("averis_quant_pair_multi", lib().averis_quant_pair_multi(
        n, ctypes.cast(arr, ctypes.c_void_p), dt, rnd, sr_stream, ws.data_ptr(), ws.numel(),
        _stream()))
    return outs


def averis_quant_pair_2d(w, seed=0, rnd=RN, sr_stream=STREAM_WEIGHT, ws=None):
    """Both GEMM copies of a weight from one quantization in 16 x 16 tiles:
    returns (wt, wd) as averis_quant_pair does, with deq(wt) = deq(wd)^T."""
    a = w if w.dim() == 3 else w.unsqueeze(0)
    batch, rows, cols = a.shape
    if a.stride(2) != 1:
        raise ValueError("expected unit innermost stride")
    wd = NVFP4.empty(batch * rows, cols, batch, w.device)
    wt = NVFP4.empty(batch * cols, rows, batch, w.device)
    need = workspace_bytes(OP_QUANT, rows, cols, 0, batch)
    ws = ws if ws is not None else _workspace(need, w.device)
    o, ot = wd.c(), wt.c()
    _check("averis_quant_pair_2d", lib().averis_quant_pair_2d(
        a.data_ptr(), _dtype_code(a), batch, rows, cols, a.stride(1), a.stride(0), seed, rnd,
        sr_stream, ctypes.byref(o), ctypes.byref(ot), ws.data_ptr(), ws.numel(), _stream()))
    return wt, wd


def averis_quant_grouped(a, offsets, seed=0, rnd=SR, sr_stream=STREAM_ACT, ws=None, out=None):
    """Grouped plain Q4, one tensor scale per segment.  out: an NVFP4 of the
    output's shape (nseg tensor scales) to write into (else a new one)."""
    rows, cols = a.shape
    nseg = offsets.numel() - 1
    out = out if out is not None else NVFP4.empty(rows, cols, nseg, a.device)
    need = workspace_bytes(OP_QUANT, rows, cols, 0, nseg)
    ws = ws if ws is not None else _workspace(need, a.device)
    o = out.c()
    _check("averis_quant_grouped", lib().averis_quant_grouped(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), offsets.data_ptr(), nseg, seed, rnd,
        sr_stream, ctypes.byref(o), ws.data_ptr(), ws.numel(), _stream()))
    return out


def _out(m, n, dtype, device, out):
    if out is not None:
        return out
    return torch.empty((m, n), dtype=dtype, device=device)


def _gemm(fn, a, mean, b, out_dtype, out, nseg=1, offsets=None, ws=None):
    m, k = a.rows, a.cols
    n = b.rows // (nseg if offsets is not None else 1)
    c = _out(m, n, out_dtype, a.codes.device, out)
    need = workspace_bytes(OP_GEMM, m, k, n, nseg if offsets is not None else 0)
    ws = ws if ws is not None else _workspace(need, a.codes.device)
    ca, cb = a.c(), b.c()
    cm = mean.c() if mean is not None else None
    pm = ctypes.byref(cm) if cm is not None else None
    cd = _dtype_code(c)
    if fn == "averis_gemm_vanilla":
        st = lib().averis_gemm_vanilla(ctypes.byref(ca), ctypes.byref(cb), c.data_ptr(), cd,
                                       c.stride(0), ws.data_ptr(), ws.numel(), _stream())
    elif fn == "averis_gemm_grouped":
        st = lib().averis_gemm_grouped(ctypes.byref(ca), pm, ctypes.byref(cb),
                                       offsets.data_ptr(), nseg, c.data_ptr(), cd, c.stride(0),
                                       ws.data_ptr(), ws.numel(), _stream())
    else:
        st = getattr(lib(), fn)(ctypes.byref(ca), pm, ctypes.byref(cb), c.data_ptr(), cd,
                                c.stride(0), ws.data_ptr(), ws.numel(), _stream())
    _check(fn, st)
    return c


def averis_gemm_fwd(xr, mean, wt, out_dtype=torch.float32, out=None, ws=None):
    """Y = 1 (mean W) + X_R W with wt = Q4(W^T) (n x m)."""
    return _gemm("averis_gemm_fwd", xr, mean, wt, out_dtype, out, ws=ws)


def averis_gemm_dgrad(dr, mean_d, w, out_dtype=torch.float32, out=None, ws=None):
    """dX = 1 (mean_D W^T) + D_R W^T with w = Q4(W) (m x n)."""
    return _gemm("averis_gemm_dgrad", dr, mean_d, w, out_dtype, out, ws=ws)


def averis_gemm_vanilla(a, b, out_dtype=torch.float32, out=None, ws=None):
    return _gemm("averis_gemm_vanilla", a, None, b, out_dtype, out, ws=ws)


def averis_gemm_grouped(a, mean, b, offsets, out_dtype=torch.float32, out=None, ws=None):
    nseg = offsets.numel() - 1
    return _gemm("averis_gemm_grouped", a, mean, b, out_dtype, out, nseg=nseg, offsets=offsets,
                 ws=ws)


def averis_residual_t_quant(a, mu, residual, seed=0, rnd=SR, out=None):
    """Q4((a - 1 mu)^T) (cols x rows, blocks along the tokens, SR stream 3);
    mu and residual are the fp32 mean and the residual tensor
    averis_split_quant returned for the same a."""
    rows, cols = a.shape
    out = out if out is not None else NVFP4.empty(cols, rows, 1, a.device)
    o = out.c()
    _check("averis_residual_t_quant", lib().averis_residual_t_quant(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), mu.data_ptr(),
        residual.tscale.data_ptr(), seed, rnd, ctypes.byref(o), _stream()))
    return out


def averis_gemm_wgrad(xt, dt, mu_x, mu_d, out_dtype=torch.float32, out=None, ws=None):
    """dW = deq(xt) deq(dt)^T + l mu_x mu_d^T (m x n) from the transposed
    residuals xt (m x l) and dt (n x l) and the fp32 means."""
    m, n, l = xt.rows, dt.rows, xt.cols
    c = _out(m, n, out_dtype, xt.codes.device, out)
    need = workspace_bytes(OP_WGRAD, m, l, n)
    ws = ws if ws is not None else _workspace(need, xt.codes.device)
    cx, cd = xt.c(), dt.c()
    _check("averis_gemm_wgrad", lib().averis_gemm_wgrad(
        ctypes.byref(cx), ctypes.byref(cd), mu_x.data_ptr(), mu_d.data_ptr(), c.data_ptr(),
        _dtype_code(c), c.stride(0), ws.data_ptr(), ws.numel(), _stream()))
    return c


def averis_split_quant_ratio(a, seed=0, rnd=SR, offsets=None, ws=None):
    """averis_split_quant (or its grouped form with offsets) plus the
    mean-energy ratio of each segment; returns (residual, mean, mu_f32, ratio)."""
    rows, cols = a.shape
    nseg = 1 if offsets is None else offsets.numel() - 1
    res = NVFP4.empty(rows, cols, nseg, a.device)
    mean = NVFP4.empty(nseg, cols, nseg, a.device)
    mu = torch.empty((nseg, cols) if offsets is not None else (cols,), dtype=torch.float32,
                     device=a.device)
    ratio = torch.empty((nseg,), dtype=torch.float32, device=a.device)
    need = workspace_bytes(OP_SPLIT_QUANT, rows, cols, 0, 0 if offsets is None else nseg)
    ws = ws if ws is not None else _workspace(need, a.device)
    r, m = res.c(), mean.c()
    _check("averis_split_quant_ratio", lib().averis_split_quant_ratio(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a),
        offsets.data_ptr() if offsets is not None else None, nseg, seed, rnd, ctypes.byref(r),
        ctypes.byref(m), mu.data_ptr(), ratio.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return res, mean, mu, ratio


def averis_split_quant_rank1(a, b, seed=0, rnd=SR, ws=None, rho=None, out=None):
    """averis_split_quant plus the rank-one row rho = deq(mean) deq(b)^T for
    the GEMM's B operand b; returns (residual, mean, mu_f32, rho).  out:
    (residual, mean, mu_f32) to write into (else new ones)."""
    rows, cols = a.shape
    if out is not None:
        res, mean, mu = out
    else:
        res = NVFP4.empty(rows, cols, 1, a.device)
        mean = NVFP4.empty(1, cols, 1, a.device)
        mu = torch.empty((cols,), dtype=torch.float32, device=a.device)
    rho = rho if rho is not None else torch.empty((b.rows,), dtype=torch.float32, device=a.device)
    need = workspace_bytes(OP_SPLIT_QUANT, rows, cols)
    ws = ws if ws is not None else _workspace(need, a.device)
    r, m, cb = res.c(), mean.c(), b.c()
    _check("averis_split_quant_rank1", lib().averis_split_quant_rank1(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), seed, rnd, ctypes.byref(r),
        ctypes.byref(m), mu.data_ptr(), ctypes.byref(cb), rho.data_ptr(), ws.data_ptr(),
        ws.numel(), _stream()))
    return res, mean, mu, rho


def averis_split_quant_rank1_multi(a, bs, seed=0, rnd=SR, ws=None, rhos=None):
    """averis_split_quant plus the rank-one rows of several GEMMs that take
    the split (B operands bs, at most MAX_RANK1); returns (residual, mean,
    mu_f32, [rho per operand])."""
    nb = len(bs)
    if not 1 <= nb <= MAX_RANK1:
        raise ValueError("expected 1 .. %d B operands" % MAX_RANK1)
    rows, cols = a.shape
    res = NVFP4.empty(rows, cols, 1, a.device)
    mean = NVFP4.empty(1, cols, 1, a.device)
    mu = torch.empty((cols,), dtype=torch.float32, device=a.device)
    rhos = list(rhos) if rhos is not None else [
        torch.empty((b.rows,), dtype=torch.float32, device=a.device) for b in bs]
    need = workspace_bytes(OP_SPLIT_QUANT, rows, cols)
    ws = ws if ws is not None else _workspace(need, a.device)
    r, m = res.c(), mean.c()
    cbs = [b.c() for b in bs]
    barr = (ctypes.POINTER(_NVFP4) * nb)(*[ctypes.pointer(cb) for cb in cbs])
    rarr = (ctypes.c_void_p * nb)(*[rho.data_ptr() for rho in rhos])
    _check("averis_split_quant_rank1_multi", lib().averis_split_quant_rank1_multi(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), seed, rnd, ctypes.byref(r),
        ctypes.byref(m), mu.data_ptr(), nb, ctypes.cast(barr, ctypes.c_void_p),
        ctypes.cast(rarr, ctypes.c_void_p), ws.data_ptr(), ws.numel(), _stream()))
    return res, mean, mu, rhos


def averis_gemm_rank1(a, rho, b, out_dtype=torch.float32, out=None):
    """c = deq(a) deq(b)^T + 1 rho^T."""
    c = _out(a.rows, b.rows, out_dtype, a.codes.device, out)
    ca, cb = a.c(), b.c()
    _check("averis_gemm_rank1", lib().averis_gemm_rank1(
        ctypes.byref(ca), rho.data_ptr(), ctypes.byref(cb), c.data_ptr(), _dtype_code(c),
        c.stride(0), _stream()))
    return c


def averis_split_quant_grouped_rank1(a, offsets, b, seed=0, rnd=SR, ws=None, out=None, rho=None):
    """Grouped split-quant plus rho[s] = deq(mean_s) deq(b_s)^T per segment
    (b: nseg stacked matrices); returns (residual, mean, mu_f32, rho).  out:
    (residual, mean, mu_f32) and rho: buffers to write into (else new ones)."""
    rows, cols = a.shape
    nseg = offsets.numel() - 1
    if out is not None:
        res, mean, mu = out
    else:
        res = NVFP4.empty(rows, cols, nseg, a.device)
        mean = NVFP4.empty(nseg, cols, nseg, a.device)
        mu = torch.empty((nseg, cols), dtype=torch.float32, device=a.device)
    rho = rho if rho is not None else torch.empty((b.rows,), dtype=torch.float32, device=a.device)
    need = workspace_bytes(OP_SPLIT_QUANT, rows, cols, 0, nseg)
    ws = ws if ws is not None else _workspace(need, a.device)
    r, m, cb = res.c(), mean.c(), b.c()
    _check("averis_split_quant_grouped_rank1", lib().averis_split_quant_grouped_rank1(
        a.data_ptr(), _dtype_code(a), rows, cols, _lda(a), offsets.data_ptr(), nseg, seed, rnd,
        ctypes.byref(r), ctypes.byref(m), mu.data_ptr(), ctypes.byref(cb), rho.data_ptr(),
        ws.data_ptr(), ws.numel(), _stream()))
    return res, mean, mu, rho


def averis_gemm_grouped_rank1(a, rho, b, offsets, out_dtype=torch.float32, out=None):
    """c[rows of s] = deq(a_s) deq(b_s)^T + 1 rho_s^T."""
    nseg = offsets.numel() - 1
    c = _out(a.rows, b.rows // nseg, out_dtype, a.codes.device, out)
    ca, cb = a.c(), b.c()
    _check("averis_gemm_grouped_rank1", lib().averis_gemm_grouped_rank1(
        ctypes.byref(ca), rho.data_ptr(), ctypes.byref(cb), offsets.data_ptr(), nseg,
        c.data_ptr(), _dtype_code(c), c.stride(0), _stream()))
    return c


def averis_gemm_rank1_stats(a, rho, b, ws=None, out=None):
    """averis_gemm_rank1 with bf16 output that also writes the column
    statistics of the output into ws, the split workspace of that output;
    returns (c, ws) for averis_split_quant_from_stats."""
    m, n = a.rows, b.rows
    c = _out(m, n, torch.bfloat16, a.codes.device, out)
    need = workspace_bytes(OP_SPLIT_QUANT, m, n)
    ws = ws if ws is not None else _workspace(need, a.codes.device)
    ca, cb = a.c(), b.c()
    _check("averis_gemm_rank1_stats", lib().averis_gemm_rank1_stats(
        ctypes.byref(ca), rho.data_ptr(), ctypes.byref(cb), c.data_ptr(), c.stride(0),
        ws.data_ptr(), ws.numel(), _stream()))
    return c, ws


def averis_split_quant_from_stats(c, ws, seed=0, rnd=SR, b=None, rho=None):
    """averis_split_quant of the bf16 output c of averis_gemm_rank1_stats from
    the statistics it left in ws; with b, also the rank-one row for the GEMM
    that takes this split.  Returns (residual, mean, mu_f32) or, with b,
    (residual, mean, mu_f32, rho)."""
    rows, cols = c.shape
    res = NVFP4.empty(rows, cols, 1, c.device)
    mean = NVFP4.empty(1, cols, 1, c.device)
    mu = torch.empty((cols,), dtype=torch.float32, device=c.device)
    if b is not None and rho is None:
        rho = torch.empty((b.rows,), dtype=torch.float32, device=c.device)
    r, m = res.c(), mean.c()
    cb = b.c() if b is not None else None
    _check("averis_split_quant_from_stats", lib().averis_split_quant_from_stats(
        c.data_ptr(), rows, cols, _lda(c), seed, rnd, ctypes.byref(r), ctypes.byref(m),
        mu.data_ptr(), ctypes.byref(cb) if cb is not None else None,
        rho.data_ptr() if rho is not None else None, ws.data_ptr(), ws.numel(), _stream()))
    return (res, mean, mu) if b is None else (res, mean, mu, rho)


# --------------------------------------------------------------------------
# mixture-of-experts routing and token exchange
# --------------------------------------------------------------------------

def _like(t, ref, dtype, what, shape=None):
    """t, checked to be a contiguous tensor of `dtype` (and shape) on ref's device."""
    if t.dtype != dtype or not t.is_contiguous() or t.device != ref.device:
        raise ValueError("%s: expected a contiguous %s tensor on %s" % (what, dtype, ref.device))
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (what, shape, tuple(t.shape)))
    return t


def _matrix(t, ref, what, shape=None):
    """Row stride of t, checked to be a 2-D tensor of ref's type (and shape) with unit column
    stride on ref's device."""
    sh = t.shape
    if len(sh) != 2 or (t is not ref and (t.dtype != ref.dtype or t.device != ref.device)):
        raise ValueError("%s: expected a 2-D %s tensor on %s" % (what, ref.dtype, ref.device))
    if shape is not None and sh != shape:
        raise ValueError("%s: expected shape %s, got %s" % (what, shape, tuple(sh)))
    rows, cols = sh
    if rows == 0 or cols == 0:
        return max(cols, 1)
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError("%s: expected unit column stride" % what)
    return ld if rows > 1 else max(ld, cols)


def _new(rows, cols, dtype, device):
    # a row-major matrix: with its strides given it is made 0.4 us sooner than by
    # torch.empty, an eighth of a launch
    return torch.empty_strided((rows, cols), (cols or 1, 1), dtype=dtype, device=device)


def _ws(ws, op, dims, dev):
    """A call's workspace: the caller's, checked to be contiguous memory on dev,
    a new one, or None where none is needed.  The tensor itself, which the caller
    holds until its call has returned."""
    if ws is None:
        need = workspace_bytes(op, *dims)
        return _workspace(need, dev) if need else None
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous tensor on %s" % dev)
    return ws


def averis_moe_route(logits, topk, renorm=True):
    """Top-k experts of each token and their softmax weights; returns
    (expert_ids int32 [tokens, topk], weights float32 [tokens, topk]).  -inf
    masks an expert; a slot without an open expert has id -1 and weight 0."""
    ld = _matrix(logits, logits, "logits")
    tokens, experts = logits.shape
    ids = _new(tokens, topk, torch.int32, logits.device)
    weights = torch.empty_like(ids, dtype=torch.float32)
    _check("averis_moe_route", lib().averis_moe_route(
        logits.data_ptr(), _dtype_code(logits), tokens, experts, ld, topk, int(bool(renorm)),
        ids.data_ptr(), weights.data_ptr(), _stream_on(logits)))
    return ids, weights


def averis_moe_route_grad(logits, ids, dweights, renorm=True, out=None):
    """The logits' gradient (their type) from dweights, for the ids that
    averis_moe_route returned for the same logits and renorm."""
    ld = _matrix(logits, logits, "logits")
    tokens, experts = logits.shape
    _like(ids, logits, torch.int32, "ids")
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids: expected shape (%d, topk)" % tokens)
    topk = ids.shape[1]
    _like(dweights, logits, torch.float32, "dweights", (tokens, topk))
    out = out if out is not None else _new(tokens, experts, logits.dtype, logits.device)
    ldd = _matrix(out, logits, "out", (tokens, experts))
    _check("averis_moe_route_grad", lib().averis_moe_route_grad(
        logits.data_ptr(), _dtype_code(logits), tokens, experts, ld, topk, int(bool(renorm)),
        ids.data_ptr(), dweights.data_ptr(), out.data_ptr(), ldd, _stream_on(logits)))
    return out


def averis_moe_sort(ids, experts, ws=None):
    """The slots' stable order by expert; returns (offsets int64 [experts + 1],
    pos int32 [tokens, topk], src int32 [tokens * topk]): offsets as the
    grouped calls take them, pos[t, j] slot (t, j)'s row (~row if its id is
    outside [0, experts): a tail row), src[row] the row's slot."""
    _like(ids, ids, torch.int32, "ids")
    if ids.dim() != 2:
        raise ValueError("ids: expected shape (tokens, topk)")
    tokens, topk = ids.shape
    dev = ids.device
    offsets = ids.new_empty(experts + 1, dtype=torch.int64)
    pos = torch.empty_like(ids)
    src = ids.new_empty(tokens * topk)
    ws = _ws(ws, OP_MOE_SORT, (tokens * topk, 0, experts), dev)
    _check("averis_moe_sort", lib().averis_moe_sort(
        ids.data_ptr(), tokens, topk, experts, offsets.data_ptr(), pos.data_ptr(), src.data_ptr(),
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
        _stream_on(ids)))
    return offsets, pos, src


def _slots(pos, ref):
    _like(pos, ref, torch.int32, "pos")
    if pos.dim() != 2:
        raise ValueError("pos: expected shape (tokens, topk)")
    return pos.shape


def averis_moe_dispatch(x, pos, out=None):
    """Each token's row copied to its topk rows (tail rows zero); returns
    rows [tokens * topk, cols].  Its gradient is averis_moe_combine(drows, pos)."""
    tokens, topk = _slots(pos, x)
    cols = x.shape[-1]
    ldx = _matrix(x, x, "x", (tokens, cols))
    out = out if out is not None else _new(tokens * topk, cols, x.dtype, x.device)
    ldr = _matrix(out, x, "out", (tokens * topk, cols))
    _check("averis_moe_dispatch", lib().averis_moe_dispatch(
        x.data_ptr(), _dtype_code(x), tokens, cols, ldx, pos.data_ptr(), topk, out.data_ptr(), ldr,
        _stream_on(x)))
    return out


def averis_moe_combine(rows, pos, weights=None, out=None):
    """y[t] = sum_j weights[t, j] rows[pos[t, j]] (weights None: all 1)."""
    tokens, topk = _slots(pos, rows)
    cols = rows.shape[-1]
    ldr = _matrix(rows, rows, "rows", (tokens * topk, cols))
    if weights is not None:
        _like(weights, rows, torch.float32, "weights", (tokens, topk))
    out = out if out is not None else _new(tokens, cols, rows.dtype, rows.device)
    ldy = _matrix(out, rows, "out", (tokens, cols))
    _check("averis_moe_combine", lib().averis_moe_combine(
        rows.data_ptr(), _dtype_code(rows), tokens, cols, ldr, pos.data_ptr(),
        weights.data_ptr() if weights is not None else None, topk, out.data_ptr(), ldy,
        _stream_on(rows)))
    return out


def averis_moe_combine_grad(dy, rows, pos, weights, out=None):
    """The gradients of averis_moe_combine: returns (drows, dweights)."""
    tokens, topk = _slots(pos, dy)
    cols = dy.shape[-1]
    ldy = _matrix(dy, dy, "dy", (tokens, cols))
    ldr = _matrix(rows, dy, "rows", (tokens * topk, cols))
    _like(weights, dy, torch.float32, "weights", (tokens, topk))
    out = out if out is not None else _new(tokens * topk, cols, dy.dtype, dy.device)
    lddr = _matrix(out, dy, "out", (tokens * topk, cols))
    dweights = torch.empty_like(weights)
    _check("averis_moe_combine_grad", lib().averis_moe_combine_grad(
        dy.data_ptr(), _dtype_code(dy), tokens, cols, ldy, rows.data_ptr(), ldr, pos.data_ptr(),
        weights.data_ptr(), topk, out.data_ptr(), lddr, dweights.data_ptr(), _stream_on(dy)))
    return out, dweights


# --------------------------------------------------------------------------
# linears in block-scaled fp8
# --------------------------------------------------------------------------

class FP8:
    """Device fp8 tensor with one power-of-two scale for 128 elements along the
    columns: codes u8[rows, cols rounded up to 128] (E4M3, zero past cols),
    scales u8[rows, ceil(cols / 128) rounded up to 4] (E8M0)."""
    __slots__ = ("codes", "scales", "rows", "cols", "_c")

    def __init__(self, codes, scales, rows, cols):
        pitch, spitch = FP8.pitches(cols)
        _fp8_bytes(codes, "codes", (rows, pitch))
        _fp8_bytes(scales, "scales", (rows, spitch))
        if codes.device != scales.device:
            raise ValueError("expected codes and scales on one device")
        self._set(codes, scales, rows, cols)

    def _set(self, codes, scales, rows, cols):
        _set_codes(self, codes)
        _set_scales(self, scales)
        _set_rows(self, rows)
        _set_cols(self, cols)
        _set_c(self, _FP8(None, None, rows, cols))

    def __setattr__(self, name, t):
        # codes and scales may be replaced by others of their form
        if name not in ("codes", "scales"):
            raise AttributeError("%s cannot be set" % name)
        _fp8_bytes(t, name, (self.rows, FP8.pitches(self.cols)[name == "scales"]))
        object.__setattr__(self, name, t)

    def __reduce__(self):   # copies and pickles
        return FP8, (self.codes, self.scales, self.rows, self.cols)

    def c(self):
        # the addresses of this call: the tensors may have been replaced since the last
        c = self._c
        c.codes, c.scales = self.codes.data_ptr(), self.scales.data_ptr()
        return c

    @staticmethod
    def pitches(cols):
        blocks = (cols + 127) // 128
        return 128 * blocks, (blocks + 3) // 4 * 4

    @staticmethod
    def empty(rows, cols, device="cuda"):
        p, s = FP8.pitches(cols)
        q = FP8.__new__(FP8)
        q._set(_new(rows, p, torch.uint8, device), _new(rows, s, torch.uint8, device), rows, cols)
        return q


def _fp8_bytes(t, what, shape):
    if t.shape != shape or t.dtype != torch.uint8 or not t.is_contiguous():
        raise ValueError("%s: expected a contiguous uint8 tensor of shape %s" % (what, shape))


# the fields' own setters, for what has been checked or made to fit
_set_codes, _set_scales, _set_rows, _set_cols, _set_c = (
    getattr(FP8, name).__set__ for name in FP8.__slots__)


def _segments(offsets, ref):
    """(address or None, number of segments) of the offsets of a grouped call."""
    if offsets is None:
        return None, 1
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets: expected nseg + 1 values")
    _like(offsets, ref, torch.int64, "offsets")
    return offsets.data_ptr(), offsets.numel() - 1


def averis_fp8_quant(a, transposed=False, offsets=None, plain=True):
    """a quantized along its columns, and (transposed=True) its transpose along
    a's rows too; returns q, or (q, qt) with q None unless plain.  offsets:
    the rows' segments (each starts a run of its own in qt)."""
    lda = _matrix(a, a, "a")
    rows, cols = a.shape
    offs, nseg = _segments(offsets, a)
    q = FP8.empty(rows, cols, a.device) if plain else None
    qt = None
    if transposed:
        tc = rows if offsets is None else int(lib().averis_fp8_seg_cols(rows, nseg))
        qt = FP8.empty(cols, tc, a.device)
    _check("averis_fp8_quant", lib().averis_fp8_quant(
        a.data_ptr(), _dtype_code(a), rows, cols, lda, offs, nseg,
        q.c() if q is not None else None, qt.c() if qt is not None else None, _stream_on(a)))
    return (q, qt) if transposed else q


def averis_fp8_quant_weight(w):
    """Both copies of a weight from one quantization in 128 x 128 tiles:
    returns (wt, wd) as averis_quant_pair does, wt = Q(w)^T (the forward
    operand) and wd = Q(w) (the dgrad operand).  w: 2-D, or 3-D (a stack)."""
    a = w if w.dim() == 3 else w.unsqueeze(0)
    batch, rows, cols = a.shape
    bstride, ld, step = a.stride()
    if cols > 1 and step != 1:
        raise ValueError("expected unit innermost stride")
    if rows == 1:
        ld = cols   # (the stride of a single row does not matter)
    wd = FP8.empty(batch * rows, cols, w.device)
    wt = FP8.empty(batch * cols, rows, w.device)
    _check("averis_fp8_quant_weight", lib().averis_fp8_quant_weight(
        a.data_ptr(), _dtype_code(a), batch, rows, cols, ld, bstride, wd.c(), wt.c(), _stream_on(w)))
    return wt, wd


def _one_device(a, b):
    dev = a.codes.device
    if a.scales.device != dev or b.codes.device != dev or b.scales.device != dev:
        raise ValueError("expected the operands' codes and scales on one device")
    return dev


def averis_fp8_gemm(a, b, out_dtype=torch.bfloat16, offsets=None, out=None, ws=None):
    """c = deq(a) deq(b)^T; with offsets the rows of segment s times the s-th
    of the matrices stacked in b.  Up to 2^30 rows, and 2^22 columns (k)."""
    dev = _one_device(a, b)
    offs, nseg = _segments(offsets, a.codes)
    m, k, n = a.rows, a.cols, b.rows // nseg
    c, ldc = out, n
    if out is None:
        c = _new(m, n, out_dtype, dev)
    else:
        ldc = _matrix(c, c, "out", (m, n))
        if c.device != dev:
            raise ValueError("out: expected a tensor on %s" % dev)
    ws = _ws(ws, OP_FP8_GEMM, (m, k, n, 0 if offsets is None else nseg), dev)
    _check("averis_fp8_gemm", lib().averis_fp8_gemm(
        a.c(), b.c(), offs, nseg, c.data_ptr(), _dtype_code(c), ldc,
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
        _stream_on(c)))
    return c


def averis_fp8_gemm_wgrad(xt, dt, out_dtype=torch.bfloat16, offsets=None, rows=None, out=None,
                          ws=None):
    """dw = deq(xt) deq(dt)^T over the tokens (m x n), from averis_fp8_quant's
    transposed copies; with the offsets of the quantization and its number of
    rows (by default the largest that the copies can hold) one matrix a
    segment (nseg x m x n).  Up to 2^22 tokens, each segment's last run of 128
    counted whole (fewer than averis_fp8_quant takes)."""
    dev = _one_device(xt, dt)
    offs, nseg = _segments(offsets, xt.codes)
    m, n = xt.rows, dt.rows
    if rows is None:
        # seg_cols(rows) = (ceil(rows / 128) + nseg) * 128 for more than one segment
        rows = xt.cols - (128 * nseg if offsets is not None and nseg > 1 else 0)
    shape = (m, n) if offsets is None else (nseg, m, n)
    c = out if out is not None else torch.empty(shape, dtype=out_dtype, device=dev)
    if out is not None and (c.shape != shape or not c.is_contiguous() or c.device != dev):
        raise ValueError("out: expected a contiguous tensor of shape %s on %s" % (shape, dev))
    ws = _ws(ws, OP_FP8_WGRAD, (m, rows, n, 0 if offsets is None else nseg), dev)
    _check("averis_fp8_gemm_wgrad", lib().averis_fp8_gemm_wgrad(
        xt.c(), dt.c(), rows, offs, nseg, c.data_ptr(), _dtype_code(c), n,
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
        _stream_on(c)))
    return c


# --------------------------------------------------------------------------
# the global gradient norm, and clipping
# --------------------------------------------------------------------------

def _grad_list(grads, out):
    """The C descriptors (averis_grad_t, four 8-byte words each) of the list."""
    dev = grads[0].device if len(grads) else None
    words = []
    for i, g in enumerate(grads):
        n, o = g.numel(), g
        if out is not None:
            o = out[i]
            if o.dtype != g.dtype or o.numel() != n or o.device != dev or not o.is_contiguous():
                raise ValueError("out[%d]: expected a contiguous tensor of the gradient's type, "
                                 "size and device" % i)
        if g.device != dev or not g.is_contiguous():
            raise ValueError("expected contiguous gradients on one device")
        words += (g.data_ptr(), o.data_ptr(), n, _dtype_code(g))
    return (ctypes.c_uint64 * len(words))(*words)


def _grad_call(grads, out, ws):
    arr = _grad_list(grads, out)
    dev = grads[0].device if len(grads) else "cuda"
    norm = torch.empty((), dtype=torch.float32, device=dev)
    return arr, norm, _ws(ws, OP_GRAD_NORM, (0, 0, len(grads)), norm.device)


def averis_grad_norm(grads, ws=None):
    """The 2-norm over every element of the tensors in the list (a float32
    tensor of no dimensions, on their device)."""
    arr, norm, ws = _grad_call(grads, None, ws)
    _check("averis_grad_norm", lib().averis_grad_norm(
        len(grads), arr, norm.data_ptr(), ws.data_ptr(), ws.numel(), _stream_on(norm)))
    return norm


def averis_grad_clip(grads, max_norm, eps=1e-6, out=None, ws=None):
    """Each gradient times min(1, max_norm / (norm + eps)), in place or into
    the tensors of the list out; returns the norm as averis_grad_norm does."""
    if out is not None and len(out) != len(grads):
        raise ValueError("out: expected %d tensors" % len(grads))
    arr, norm, ws = _grad_call(grads, out, ws)
    _check("averis_grad_clip", lib().averis_grad_clip(
        len(grads), arr, max_norm, eps, norm.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream_on(norm)))
    return norm
