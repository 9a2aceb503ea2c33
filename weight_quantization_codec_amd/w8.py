"""8-bit integer linear layers (include/qamw_w8.h): rows as int8 codes with a scale each, the norm in
front of a linear layer with its output in that form, and the product of two matrices in that form.

The binding marshals arguments as the rest of the package does; ordinary calls (matrices on the current
device, outputs made here) take a short way through the compiled module _w8_host, with the same checks,
and every other call, all errors among them, the way through this file.  Work is queued on the current stream
of the tensors' device.  Codes are int8 tensors whose rows start on 16-byte boundaries; the functions
that make codes return rows x d views of buffers with rows of q8_stride(d) bytes, and write zeros up to the next
multiple of 16 bytes behind each row, in a given out too.

Nothing here has a backward: codes, row scales, values read back and products carry no gradient, whatever their
inputs require.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

try:
    from . import _w8_host as _host
except ImportError:   # not built: every call takes the long way
    _host = None

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "qamw_q8_stride": ([_i32], _sz),
    "qamw_quant8": ([_vp, ctypes.c_int, _i32, _i32, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp], ctypes.c_int),
    "qamw_dequant8": ([_vp, _i32, _i32, _i64, _vp, _vp, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "qamw_rmsnorm8": ([_vp, ctypes.c_int, _i32, _i32, _i64, _vp, _i64, _vp, ctypes.c_float, _vp, _i64, _vp, _i64, _vp,
                       _vp, _vp], ctypes.c_int),
    "qamw_gemm8_workspace": ([_i32, _i32, _i32], _sz),
    "qamw_gemm8": ([_vp, _i64, _vp, _i32, _vp, _i64, _vp, _i32, _i32, _vp, ctypes.c_int, _i64, _vp, _sz, _vp],
                   ctypes.c_int),
}

_INT_MAX = 2**31 - 1
_VALUES = (torch.bfloat16, torch.float32)
# limits of include/qamw_w8.h
W8_MAX_COLS = 32768
GEMM8_MAX_ROWS = 1 << 24
GEMM8_MAX_COLS = 131071
GEMM8_MAX_LD = 1 << 22
GEMM8_MAX_OUT = 1 << 38


# The current stream's handle without a Stream object around it: a tenth of the time, in calls that take
# a few microseconds in all.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _not_there(index: int, **tensors):
    """The error of a call with a tensor that is not on device `index`, the first one's."""
    if index < 0:
        raise ValueError("%s must be a device tensor" % next(iter(tensors)))
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s is on %s, not on device %d" % (name, t.device, index))


def _rows(t, name: str, like: Optional[torch.Tensor] = None) -> int:
    """A 2-D bf16 or fp32 matrix with contiguous rows, of the size and type of `like`; its row pitch."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _VALUES or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor of bfloat16 or float32" % name)
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError("%s must be %s of %s, got %s of %s"
                         % (name, tuple(like.shape), like.dtype, tuple(t.shape), t.dtype))
    n, d = t.shape
    if n > _INT_MAX or d > _INT_MAX:
        raise ValueError("%s is too large: %d x %d" % (name, n, d))
    if t.is_contiguous():
        return d
    s0, s1 = t.stride()
    if d > 1 and s1 != 1:
        raise ValueError("%s rows must be contiguous" % name)
    if n > 1 and s0 < d:
        raise ValueError("%s rows overlap" % name)
    return s0 if n > 1 else d


def _codes(t, name: str, rows: Optional[int] = None, d: Optional[int] = None) -> int:
    """A code matrix: rows on 16-byte boundaries, each with the bytes up to the next one in its storage;
    its row pitch."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int8 or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor of int8" % name)
    n, k = t.shape
    if (rows is not None and n != rows) or (d is not None and k != d):
        raise ValueError("%s must be %s x %s, got %s" % (name, rows, d, tuple(t.shape)))
    if n > _INT_MAX or k > _INT_MAX:
        raise ValueError("%s is too large: %d x %d" % (name, n, k))
    padded = (k + 15) // 16 * 16
    if k == padded and t.is_contiguous():
        ld = k
    elif n == 0 or k == 0:
        return padded
    else:
        s0, s1 = t.stride()
        if k > 1 and s1 != 1:
            raise ValueError("%s rows must be contiguous" % name)
        ld = s0 if n > 1 else padded
        if k != padded and t.storage_offset() + (n - 1) * ld + padded > t.untyped_storage().nbytes():
            raise ValueError("%s ends inside its last row's 16-byte chunk" % name)
    if ld % 16 or ld < k or t.data_ptr() % 16:
        raise ValueError("%s rows must start on 16-byte boundaries and not overlap" % name)
    return ld


def _vec(t, name: str, n: int, dtype=torch.float32):
    """A contiguous vector of at least n elements of dtype."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise ValueError("%s must be a tensor of %s" % (name, dtype))
    if t.numel() < n:
        raise ValueError("%s needs at least %d elements, got %d" % (name, n, t.numel()))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _out(out: Optional[torch.Tensor], dtype, rows: int, d: int) -> int:
    """The output matrix of a call, given or to be made; its row pitch."""
    if out is None:
        if dtype not in _VALUES:
            raise ValueError("out_dtype must be bfloat16 or float32")
        return d
    ld = _rows(out, "out")
    if tuple(out.shape) != (rows, d):
        raise ValueError("out must be %d x %d, got %s" % (rows, d, tuple(out.shape)))
    return ld


def _ptr(t):
    return None if t is None else t.data_ptr()


def bind(lib):
    """Gives the compiled module the functions of the loaded library."""
    if _host is not None:
        names = ("qamw_quant8", "qamw_dequant8", "qamw_rmsnorm8", "qamw_gemm8_workspace", "qamw_gemm8")
        _host.bind(*[ctypes.cast(getattr(lib, n), _vp).value for n in names], _failed)


class _Fns(dict):
    """The library's functions by name, from the first use on."""

    def __missing__(self, name):
        from . import load
        fn = self[name] = getattr(load(), name)
        return fn


_fns = _Fns()
_current = torch.cuda.current_device


def _elsewhere(fn, index: int, args) -> int:
    """A call on a device that is not the current one."""
    with torch.cuda.device(index):
        return fn(*args, _raw_stream(index))


def _failed(rc: int, name: str):
    from . import _check
    _check(rc, name)


def q8_stride(d: int) -> int:
    """Bytes from one row of codes to the next when rows are packed: d rounded up to 16."""
    return (d + 15) // 16 * 16 if d > 0 else 0


def _empty_codes(x: torch.Tensor, rows: int, d: int, pitch: int) -> torch.Tensor:
    t = x.new_empty(rows, pitch, dtype=torch.int8)
    return t if pitch == d else t[:, :d]


def quant8(x: torch.Tensor, scale: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, row_scale: Optional[torch.Tensor] = None,
           status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of x (rows x d, bf16 or fp32) as (int8 codes, fp32 row scales): of x, of x silu(gate) with a
    gate, times the channel scale (d fp32) with one.  See qamw_quant8."""
    if out is None and row_scale is None and status is None and _host is not None:
        made = _host.quant8(x, scale, gate)
        if made is not None:
            return made
    ld_x = _rows(x, "x")
    rows, d = x.shape
    ld_g = _rows(gate, "gate", like=x) if gate is not None else 0
    if scale is not None:
        _vec(scale, "scale", d)
    if row_scale is not None:
        _vec(row_scale, "row_scale", rows)
    if status is not None:
        _vec(status, "status", 1, torch.int32)
    ld_q = _codes(out, "out", rows, d) if out is not None else q8_stride(d)
    index = x.get_device()
    if index < 0 or (gate is not None and gate.get_device() != index) or (
            scale is not None and scale.get_device() != index) or (out is not None and out.get_device() != index) or (
            row_scale is not None and row_scale.get_device() != index) or (
            status is not None and status.get_device() != index):
        _not_there(index, x=x, gate=gate, scale=scale, out=out, row_scale=row_scale, status=status)
    if out is None:
        out = _empty_codes(x, rows, d, ld_q)
    if row_scale is None:
        row_scale = x.new_empty(rows, dtype=torch.float32)
    args = (x.data_ptr(), 1 if x.dtype is torch.bfloat16 else 0, rows, d, ld_x, _ptr(gate), ld_g, _ptr(scale),
            out.data_ptr(), ld_q, row_scale.data_ptr(), _ptr(status))
    fn = _fns["qamw_quant8"]
    rc = fn(*args, _raw_stream(index)) if index == _current() else _elsewhere(fn, index, args)
    if rc:
        _failed(rc, "qamw_quant8")
    return out, row_scale


def dequant8(codes: torch.Tensor, row_scale: torch.Tensor, scale: Optional[torch.Tensor] = None,
             out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that codes stand for (rows x d, bf16 or fp32), with the channel scale that quant8
    multiplied in divided out.  See qamw_dequant8."""
    if out is None and out_dtype in _VALUES and _host is not None:
        out = _host.dequant8(codes, row_scale, scale, out_dtype is torch.bfloat16)
        if out is not None:
            return out
    ld_q = _codes(codes, "codes")
    rows, d = codes.shape
    _vec(row_scale, "row_scale", rows)
    if scale is not None:
        _vec(scale, "scale", d)
    ld_out = _out(out, out_dtype, rows, d)
    index = codes.get_device()
    if index < 0 or row_scale.get_device() != index or (scale is not None and scale.get_device() != index) or (
            out is not None and out.get_device() != index):
        _not_there(index, codes=codes, row_scale=row_scale, scale=scale, out=out)
    if out is None:
        out = codes.new_empty(rows, d, dtype=out_dtype)
    args = (codes.data_ptr(), rows, d, ld_q, row_scale.data_ptr(), _ptr(scale), out.data_ptr(),
            1 if out.dtype is torch.bfloat16 else 0, ld_out)
    fn = _fns["qamw_dequant8"]
    rc = fn(*args, _raw_stream(index)) if index == _current() else _elsewhere(fn, index, args)
    if rc:
        _failed(rc, "qamw_dequant8")
    return out


def rmsnorm8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
             residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, row_scale: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Residual addition and root-mean-square norm: (int8 codes of the normalized rows, their fp32 row
    scales, h = x + residual).  Without a residual h is x itself, and sum_out (if given) a copy of it;
    sum_out may be x or residual (h in place).  h carries no gradient: but where it is x itself, x or residual
    that requires one is refused while gradients are recorded.  See qamw_rmsnorm8."""
    if sum_out is None and out is None and row_scale is None and status is None and _host is not None:
        made = _host.rmsnorm8(x, weight, eps, residual)
        if made is not None:
            return made
    ld_x = _rows(x, "x")
    rows, d = x.shape
    ld_r = _rows(residual, "residual", like=x) if residual is not None else 0
    ld_s = _rows(sum_out, "sum_out", like=x) if sum_out is not None else d
    if (residual is not None or sum_out is not None) and torch.is_grad_enabled() and (
            x.requires_grad or (residual is not None and residual.requires_grad)):
        raise ValueError("%s requires a gradient, which h would cut off: call under torch.no_grad()"
                         % ("x" if x.requires_grad else "residual"))
    if weight is not None:
        _vec(weight, "weight", d)
    if row_scale is not None:
        _vec(row_scale, "row_scale", rows)
    if status is not None:
        _vec(status, "status", 1, torch.int32)
    ld_q = _codes(out, "out", rows, d) if out is not None else q8_stride(d)
    index = x.get_device()
    if index < 0 or (residual is not None and residual.get_device() != index) or (
            sum_out is not None and sum_out.get_device() != index) or (
            weight is not None and weight.get_device() != index) or (
            out is not None and out.get_device() != index) or (
            row_scale is not None and row_scale.get_device() != index) or (
            status is not None and status.get_device() != index):
        _not_there(index, x=x, residual=residual, sum_out=sum_out, weight=weight, out=out, row_scale=row_scale,
                   status=status)
    if residual is not None and sum_out is None:
        sum_out = x.new_empty(rows, d)
    if out is None:
        out = _empty_codes(x, rows, d, ld_q)
    if row_scale is None:
        row_scale = x.new_empty(rows, dtype=torch.float32)
    args = (x.data_ptr(), 1 if x.dtype is torch.bfloat16 else 0, rows, d, ld_x, _ptr(residual), ld_r, _ptr(weight), eps,
            _ptr(sum_out), ld_s, out.data_ptr(), ld_q, row_scale.data_ptr(), _ptr(status))
    fn = _fns["qamw_rmsnorm8"]
    rc = fn(*args, _raw_stream(index)) if index == _current() else _elsewhere(fn, index, args)
    if rc:
        _failed(rc, "qamw_rmsnorm8")
    return out, row_scale, x if sum_out is None else sum_out


def gemm8_workspace(M: int, d_out: int, d_in: int) -> int:
    """Bytes of workspace that gemm8 uses (0 for most sizes, and for those that it refuses)."""
    if not all(-_INT_MAX <= size <= _INT_MAX for size in (M, d_out, d_in)):   # ctypes would cut them to 32 bits
        return 0
    return _fns["qamw_gemm8_workspace"](M, d_out, d_in)


def gemm8(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, out_dtype=torch.bfloat16,
          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x w^T of 8-bit activations (M x d_in codes, a scale for each token) and weights (d_out x d_in
    codes, a scale for each output channel): M x d_out, bf16 or fp32.  Calls that may overlap need a
    workspace each, or none given.  See qamw_gemm8."""
    if out is None and workspace is None and out_dtype in _VALUES and _host is not None:
        out = _host.gemm8(xq, x_scale, wq, w_scale, out_dtype is torch.bfloat16)
        if out is not None:
            return out
    ld_x, ld_w = _codes(xq, "xq"), _codes(wq, "wq")
    M, K = xq.shape
    N, wk = wq.shape
    if wk != K:
        raise ValueError("xq has %d columns, wq %d" % (K, wk))
    _vec(x_scale, "x_scale", M)
    _vec(w_scale, "w_scale", N)
    ld_y = _out(out, out_dtype, M, N)
    need = _fns["qamw_gemm8_workspace"](M, N, K)
    if workspace is not None:
        _vec(workspace, "workspace", need, torch.uint8)
    index = xq.get_device()
    if index < 0 or x_scale.get_device() != index or wq.get_device() != index or w_scale.get_device() != index or (
            out is not None and out.get_device() != index) or (
            workspace is not None and workspace.get_device() != index):
        _not_there(index, xq=xq, x_scale=x_scale, wq=wq, w_scale=w_scale, out=out, workspace=workspace)
    if out is None:
        out = xq.new_empty(M, N, dtype=out_dtype)
    if workspace is None and need:
        workspace = xq.new_empty(need, dtype=torch.uint8)
    args = (xq.data_ptr(), ld_x, x_scale.data_ptr(), M, wq.data_ptr(), ld_w, w_scale.data_ptr(), N, K, out.data_ptr(),
            1 if out.dtype is torch.bfloat16 else 0, ld_y, _ptr(workspace),
            0 if workspace is None else workspace.numel())
    fn = _fns["qamw_gemm8"]
    rc = fn(*args, _raw_stream(index)) if index == _current() else _elsewhere(fn, index, args)
    if rc:
        _failed(rc, "qamw_gemm8")
    return out
