"""Microscaled 4-bit floating point (MXFP4) and counter-based dropout: binding.

MXFP4 is the 4-bit format the sm_100 tensor cores multiply natively: E2M1
codes and one power-of-two scale for each 32 elements of a row.

    w = mx_weight(W)                                   # W^ for the forward, W^T's form for the backward
    Y, T = mx_linear_fwd(X, w, L1, L2, s, dropout=Dropout(0.1, seed, offset))
    dX, dL1, dL2 = mx_linear_bwd(dY, X, T, w, L1, L2, s, dropout=Dropout(0.1, seed, offset))
    C = mx_matmul(mx_quantize(A), mx_quantize(B))      # A.B^T, both sides in 4 bits

Calls are asynchronous on the current stream of their tensors' device and do
not depend on which device is current.
"""

from __future__ import annotations

import ctypes
import functools
import operator
from dataclasses import dataclass

import torch

import bit_nf4_quantized_15_b200 as _q

__all__ = ["MXTensor", "MXWeight", "Dropout", "mx_storage_bytes", "mx_quantize", "mx_dequant", "mx_matmul", "mx_weight",
           "mx_linear_fwd", "mx_linear_bwd", "mx_linear_workspace_bytes", "dropout"]

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_U64 = (1 << 64) - 1


class qlora_mx_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class qlora_dropout_config(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("offset_dev", ctypes.c_void_p)]


_P, _I64, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_T, _D, _SZ = ctypes.POINTER(qlora_mx_tensor), ctypes.POINTER(qlora_dropout_config), ctypes.c_size_t
SIGS = {
    "qlora_mx_storage_bytes": (_INT, [_I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "qlora_mx_quantize": (_INT, [_P, _INT, _I64, _I64, _INT, _T, _P, _P]),
    "qlora_mx_dequant": (_INT, [_T, _P, _INT, _P]),
    "qlora_mx_matmul": (_INT, [_T, _T, _P, _INT, _P, _P]),
    "qlora_dropout": (_INT, [_P, _INT, _I64, _D, _P, _P]),
    "qlora_mx_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "qlora_mx_linear_fwd": (_INT, [_P, _I64, _T, _P, _P, _INT, ctypes.c_float, _D, _P, _P, _P, _SZ, _P, _P]),
    "qlora_mx_linear_bwd": (_INT, [_P, _P, _I64, _P, _T, _I64, _I64, _P, _P, _INT, ctypes.c_float, _D, _P, _P, _P, _P,
                                   _SZ, _P, _P]),
}


def _bad(what):
    raise _q.QLoRAError(what)


def _name(dtype):
    return str(dtype).removeprefix("torch.")


def _tensor(t, name, shape, dtype, device):
    """`t` is a contiguous tensor of this shape, type and device."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device and t.is_cuda
            and t.is_contiguous()):
        _bad(f"{name} must be a contiguous {_name(dtype)} CUDA tensor of shape {tuple(shape)} on {device}")
    return t


def _matrix(t, name, dtypes):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.dtype in dtypes and t.is_contiguous()):
        _bad(f"{name} must be a contiguous CUDA matrix of " + " or ".join(map(_name, dtypes)))
    return t


# The current stream's handle; the binding's own accessor where torch has it
# (the public one builds a Stream object, 2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, f, *args):
    """f(*args, stream) with the device of its tensors current."""
    index = device.index
    if index == torch.cuda.current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc:
        _q._check(rc)


def _status_ptr(status, device):
    if status is None:
        status = _q._status_bufs.get(device.index)
        if status is None:
            status = _q._status(device)
    elif not (isinstance(status, torch.Tensor) and status.dtype == torch.int32 and status.device == device
              and status.numel()):
        _bad(f"status must be an int32 CUDA tensor on {device}")
    return status.data_ptr()


def mx_storage_bytes(rows: int, cols: int):
    """(codes, scales) bytes of an MXFP4 matrix: 4.25 bits an element, the
    scales padded to tiles of 128 x 128."""
    a, b = _SZ(), _SZ()
    _q._check(_q.lib().qlora_mx_storage_bytes(rows, cols, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


@dataclass
class MXTensor:
    """An MXFP4 matrix [rows, cols]: codes uint8 [rows * cols / 2] and tiled
    E8M0 scales uint8 (layout: qlora_mx_tensor in include/qlora_nf4.h)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @staticmethod
    def empty(rows: int, cols: int, device="cuda") -> "MXTensor":
        nc, ns = mx_storage_bytes(rows or 1, cols)
        if rows == 0:
            nc = ns = 0
        return MXTensor(torch.empty(nc, dtype=torch.uint8, device=device),
                        torch.empty(ns, dtype=torch.uint8, device=device), rows, cols)

    @property
    def device(self):
        return self.codes.device

    def descriptor(self) -> qlora_mx_tensor:
        c, s = self.codes, self.scales
        tiles = ((self.rows + 127) // 128) * ((self.cols + 127) // 128)
        if not (c.is_cuda and c.dtype == torch.uint8 and s.dtype == torch.uint8 and s.device == c.device
                and c.is_contiguous() and s.is_contiguous() and 2 * c.numel() >= self.rows * self.cols
                and s.numel() >= 512 * tiles):
            _bad("codes and scales must be contiguous uint8 CUDA tensors on one device that hold "
                 f"{self.rows} x {self.cols}")
        return qlora_mx_tensor(c.data_ptr(), s.data_ptr(), self.rows, self.cols)


@dataclass
class MXWeight:
    """A frozen weight [N, K] in MXFP4: ``fwd`` quantised along K for
    X.W^T, ``bwd`` (its transpose [K, N], quantised along N) for dY.W."""
    fwd: MXTensor
    bwd: MXTensor | None = None


@dataclass
class Dropout:
    """Dropout of probability p from the counter-based generator; (seed,
    offset) names the mask.  ``offset`` may be an int64 CUDA tensor of one
    element, read when the kernel runs (advance it between the replays of a
    captured graph)."""
    p: float
    seed: int
    offset: int | torch.Tensor = 0

    def config(self, device) -> qlora_dropout_config:
        off, dev_ptr = self.offset, None
        if isinstance(off, torch.Tensor):
            _tensor(off.reshape(-1), "offset", (1,), torch.int64, device)
            off, dev_ptr = 0, off.data_ptr()
        try:
            seed, off = operator.index(self.seed), operator.index(off)
        except TypeError:
            seed = off = -1
        if not (0 <= seed <= _U64 and 0 <= off <= _U64):
            _bad("seed and offset must be 64-bit unsigned integers")
        return qlora_dropout_config(float(self.p), seed, off, dev_ptr)


def mx_quantize(X, transpose: bool = False, out: MXTensor | None = None, status=None) -> MXTensor:
    """MXFP4 form of a bf16, fp16 or fp32 CUDA matrix [R, C], blocks of 32
    along its rows (C % 32 == 0); ``transpose``: of X^T, [C, R] (R % 32 == 0,
    C % 8 == 0).  A matrix without rows has an empty form."""
    _matrix(X, "X", DTYPES)
    R, C = X.shape
    shape = (C, R) if transpose else (R, C)
    if out is None:
        out = MXTensor.empty(*shape, device=X.device)
    if (out.rows, out.cols) != shape or out.device != X.device:
        _bad(f"out must be {shape[0]} x {shape[1]} on {X.device}")
    d = out.descriptor()
    if out.rows == 0:
        return out
    _call(X.device, _q.lib().qlora_mx_quantize, X.data_ptr(), DTYPES[X.dtype], R, C, int(transpose), ctypes.byref(d),
          _status_ptr(status, X.device))
    return out


def _values_dtype(dtype):
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        _bad("dtype must be bfloat16 or float32")
    return DTYPES[dtype]


def mx_dequant(t: MXTensor, dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """The values of an MXFP4 matrix, [rows, cols] in bf16 or fp32 (both exact)."""
    kind, d, dev = _values_dtype(dtype), t.descriptor(), t.device
    if out is None:
        out = t.codes.new_empty((t.rows, t.cols), dtype=dtype)
    else:
        _tensor(out, "out", (t.rows, t.cols), dtype, dev)
    if t.rows == 0:
        return out
    _call(dev, _q.lib().qlora_mx_dequant, ctypes.byref(d), out.data_ptr(), kind)
    return out


def mx_matmul(a: MXTensor, b: MXTensor, dtype=torch.bfloat16, out=None, status=None) -> torch.Tensor:
    """A.B^T of two MXFP4 matrices with equal cols, [a.rows, b.rows] in bf16
    or fp32; accumulated in fp32 (b.rows % 8 == 0)."""
    kind, dev = _values_dtype(dtype), a.device
    if b.device != dev:
        _bad("a and b must be on one device")
    da, db = a.descriptor(), b.descriptor()
    if out is None:
        out = a.codes.new_empty((a.rows, b.rows), dtype=dtype)
    else:
        _tensor(out, "out", (a.rows, b.rows), dtype, dev)
    if a.cols != b.cols or b.rows % 8:
        _bad("a and b must have equal cols, b a multiple of 8 rows")
    if a.rows == 0 or b.rows == 0:
        return out
    _call(dev, _q.lib().qlora_mx_matmul, ctypes.byref(da), ctypes.byref(db), out.data_ptr(), kind,
          _status_ptr(status, dev))
    return out


def mx_weight(W, backward: bool = True, status=None) -> MXWeight:
    """The MXFP4 forms of a weight [N, K] (bf16, fp16 or fp32) that the linear
    layer multiplies with; backward=False leaves out the one of dX (4.25 bits
    a weight)."""
    return MXWeight(mx_quantize(W, status=status), mx_quantize(W, transpose=True, status=status) if backward else None)


def mx_linear_workspace_bytes(M: int, N: int, K: int, r: int = 0) -> int:
    """Workspace of mx_linear_fwd and mx_linear_bwd (the larger of the two); it
    does not fall with M, so one for the largest batch serves smaller ones."""
    n = _q.lib().qlora_mx_linear_workspace_bytes(M, N, K, r)
    if not n:
        _bad("invalid shape or rank for mx_linear_workspace_bytes")
    return n


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(M, N, K, r, index):
    with torch.cuda.device(index):
        return mx_linear_workspace_bytes(M, N, K, r)


def _linear_args(M, N, K, L1, L2, dropout, ws, like):
    """(r, dropout config or None, workspace) after checking the adapter."""
    if (L1 is None) != (L2 is None):
        _bad("L1 and L2 come together")
    r, device = 0, like.device
    if L1 is not None:
        r = _matrix(L1, "L1", (torch.bfloat16,)).shape[1]
        _tensor(L1, "L1", (K, r), torch.bfloat16, device)
        _tensor(L2, "L2", (r, N), torch.bfloat16, device)
    cfg = None if dropout is None else ctypes.byref(dropout.config(device))
    need = _workspace_bytes(M, N, K, r, device.index)
    if ws is None:
        ws = like.new_empty(need, dtype=torch.uint8)
    elif not (ws.is_cuda and ws.device == device and ws.is_contiguous() and ws.numel() * ws.element_size() >= need):
        _bad(f"ws must be a contiguous CUDA tensor of {need} bytes on {device}")
    return r, cfg, ws


def _ptr(t):
    return None if t is None else t.data_ptr()


def _output(t, name, shape, dtype, like):
    return like.new_empty(shape, dtype=dtype) if t is None else _tensor(t, name, shape, dtype, like.device)


def mx_linear_fwd(X, w: MXWeight, L1=None, L2=None, s: float = 1.0, dropout: Dropout | None = None, ws=None, Y=None,
                  T=None, status=None):
    """Y = Q(X).W^T + s.T.L2 and T = drop(X).L1 (fp32, for the backward; None
    without an adapter).  X bf16 [M, K], quantised to MXFP4 on the way."""
    _matrix(X, "X", (torch.bfloat16,))
    M, K = X.shape
    dev, wf = X.device, w.fwd
    if wf.cols != K or wf.device != dev:
        _bad(f"the weight must have {K} columns and be on {dev}")
    N = wf.rows
    Y = _output(Y, "Y", (M, N), torch.bfloat16, X)
    T = None if L1 is None else _output(T, "T", (M, _matrix(L1, "L1", (torch.bfloat16,)).shape[1]), torch.float32, X)
    if M == 0:
        return Y, T
    r, cfg, ws = _linear_args(M, N, K, L1, L2, dropout, ws, X)
    d = wf.descriptor()
    _call(dev, _q.lib().qlora_mx_linear_fwd, X.data_ptr(), M, ctypes.byref(d), _ptr(L1), _ptr(L2), r, float(s), cfg,
          Y.data_ptr(), _ptr(T), ws.data_ptr(), ws.numel() * ws.element_size(), _status_ptr(status, dev))
    return Y, T


def mx_linear_bwd(dY, X, T, w: MXWeight, L1=None, L2=None, s: float = 1.0, dropout: Dropout | None = None, ws=None,
                  need_dX=True, need_dL1=True, need_dL2=True, status=None, dX=None, dL1=None, dL2=None):
    """dX = Q(dY).W + drop(s.dT.L1^T), dL1 = s.drop(X)^T.dT, dL2 = s.T^T.dY
    with dT = dY.L2^T; ``dropout`` names the forward's mask.  Without an
    adapter: dX alone.  dX needs ``w.bwd``; it must not share memory with X
    where dL1 is asked for, nor with dY where dL2 is."""
    _matrix(dY, "dY", (torch.bfloat16,))
    M, N = dY.shape
    dev, K = dY.device, w.fwd.cols
    if w.fwd.rows != N or w.fwd.device != dev:
        _bad(f"the weight must have {N} rows and be on {dev}")
    adapter = L1 is not None
    r = _matrix(L1, "L1", (torch.bfloat16,)).shape[1] if adapter else 0
    d = None
    if need_dX or dX is not None:
        wb = w.bwd
        if wb is None or (wb.rows, wb.cols) != (K, N) or wb.device != dev:
            _bad("dX needs the weight's backward form (mx_weight(W), w.bwd)")
        d = ctypes.byref(wb.descriptor())
        dX = _output(dX, "dX", (M, K), torch.bfloat16, dY)
    if adapter and (need_dL1 or dL1 is not None):
        _tensor(X, "X", (M, K), torch.bfloat16, dev)
        dL1 = _output(dL1, "dL1", (K, r), torch.float32, dY)
    if adapter and (need_dL2 or dL2 is not None):
        _tensor(T, "T", (M, r), torch.float32, dev)
        dL2 = _output(dL2, "dL2", (r, N), torch.float32, dY)
    if not adapter:
        dL1 = dL2 = None
    if M == 0:
        for g in (dL1, dL2):
            if g is not None:
                g.zero_()
        return dX, dL1, dL2
    r, cfg, ws = _linear_args(M, N, K, L1, L2, dropout, ws, dY)
    _call(dev, _q.lib().qlora_mx_linear_bwd, dY.data_ptr(), _ptr(X) if dL1 is not None else None, M,
          _ptr(T) if dL2 is not None else None, d, N, K, _ptr(L1), _ptr(L2), r, float(s), cfg, _ptr(dX), _ptr(dL1),
          _ptr(dL2), ws.data_ptr(), ws.numel() * ws.element_size(), _status_ptr(status, dev))
    return dX, dL1, dL2


def dropout(X, p: float, seed: int, offset=0, out=None) -> torch.Tensor:
    """X with elements zeroed with probability p and the others scaled by
    1 / (1 - p) (p in steps of 2^-16), the mask named by (seed, offset) and
    never stored; the gradient is the same call on the upstream gradient.
    X: contiguous bf16, fp16 or fp32 CUDA tensor of any shape; out may be X,
    but not overlap it otherwise."""
    if not (isinstance(X, torch.Tensor) and X.is_cuda and X.dtype in DTYPES and X.is_contiguous()):
        _bad("X must be a contiguous bfloat16, float16 or float32 CUDA tensor")
    dev = X.device
    cfg = Dropout(p, seed, offset).config(dev)
    if out is None:
        out = torch.empty_like(X)
    else:
        _tensor(out, "out", X.shape, X.dtype, dev)
    if X.numel():
        _call(dev, _q.lib().qlora_dropout, X.data_ptr(), DTYPES[X.dtype], X.numel(), ctypes.byref(cfg), out.data_ptr())
    return out
