"""Microscaled 4-bit linear layers (include/qamw_mx4.h): rows as 4-bit floating-point codes with a power of two for
every 32 columns, the norm in front of a linear layer with its output in that form, the product of two matrices in
that form, and the same product for rows in groups with weights of their own (the experts of a mixture).

The binding marshals arguments as the rest of the package does; ordinary calls (matrices on the current device,
outputs made here) take a short way through the compiled module _w8_host, with the same checks, and every other call,
all errors among them, the way through this file.  Work is queued on the current stream of the tensors' device.

A matrix of rows x d values is a pair of uint8 tensors: codes, rows x mx4_stride(d) (two columns a byte, whole groups
of 256 columns), and scales, mx4_groups(d) x rows x 8.  Rows first to last of it are codes[first:last] and
scales[:, first:last].  The products take whole groups: columns behind d are zeros, as quant4 and rmsnorm4 leave them.
Codes and scale bytes that stand by rows (rows x ceil(d / 2) and rows x ceil(d / 32)) come into this form by

    pad = torch.nn.functional.pad
    codes = pad(codes, (0, mx4_stride(d) - codes.shape[1]))
    scales = pad(scales, (0, 8 * mx4_groups(d) - scales.shape[1])).view(rows, -1, 8).transpose(0, 1).contiguous()

Nothing here has a backward: codes, scales, values read back and products carry no gradient, whatever their inputs
require.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .w8 import _INT_MAX, _VALUES, _current, _elsewhere, _failed, _fns, _host, _out, _ptr, _raw_stream, _rows, _vec

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "qamw_mx4_stride": ([_i32], _sz),
    "qamw_mx4_groups": ([_i32], _i32),
    "qamw_quant4": ([_vp, ctypes.c_int, _i32, _i32, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp], ctypes.c_int),
    "qamw_dequant4": ([_vp, _i32, _i32, _i64, _vp, _i64, _vp, _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
    "qamw_rmsnorm4": ([_vp, ctypes.c_int, _i32, _i32, _i64, _vp, _i64, _vp, ctypes.c_float, _vp, _i64, _vp, _i64, _vp,
                       _i64, _vp, _vp], ctypes.c_int),
    "qamw_gemm4_workspace": ([_i32, _i32, _i32], _sz),
    "qamw_gemm4": ([_vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _i32, _i32, _vp, ctypes.c_int, _i64, _vp, _sz, _vp],
                   ctypes.c_int),
    "qamw_gemm4_grouped": ([_vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i32, _i32, _i32,
                            _vp, ctypes.c_int, _i64, _vp], ctypes.c_int),
}


def bind(lib):
    """Gives the compiled module the functions of the loaded library."""
    if _host is not None:
        names = ("qamw_quant4", "qamw_dequant4", "qamw_rmsnorm4", "qamw_gemm4_workspace", "qamw_gemm4", "qamw_gemm4_grouped")
        _host.bind4(*[ctypes.cast(getattr(lib, n), _vp).value for n in names])


# limits of include/qamw_mx4.h
MX4_MAX_NORM_COLS = 32768
MX4_MAX_COLS = 1 << 23
GEMM4_MAX_ROWS = 1 << 24
GEMM4_MAX_LD = 1 << 22
GEMM4_MAX_OUT = 1 << 38
GEMM4_MAX_EXPERTS = 1024
GEMM4_MAX_EXPERT_ROWS = 1 << 30
GEMM4_MAX_INDEXED = 1 << 31


def mx4_groups(d: int) -> int:
    """Groups of 256 columns."""
    return (d + 255) // 256 if d > 0 else 0


def mx4_stride(d: int) -> int:
    """Bytes of a row of codes: 128 for every group."""
    return mx4_groups(d) * 128


def _codes4(t, name: str, rows: Optional[int] = None, groups: Optional[int] = None) -> int:
    """A matrix of codes with contiguous rows of whole groups, on 16-byte boundaries; its row pitch."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor of uint8" % name)
    n, b = t.shape
    if (rows is not None and n != rows) or (groups is not None and b != 128 * groups):
        raise ValueError("%s must be %s x %s, got %s" % (name, rows, None if groups is None else 128 * groups, tuple(t.shape)))
    if b % 128 or b == 0:
        raise ValueError("%s rows must be whole groups of 128 bytes, got %d" % (name, b))
    if n > _INT_MAX or b > _INT_MAX:
        raise ValueError("%s is too large: %d x %d" % (name, n, b))
    if n == 0:
        return b
    s0, s1 = t.stride()
    if s1 != 1:
        raise ValueError("%s rows must be contiguous" % name)
    ld = s0 if n > 1 else b
    if ld % 16 or ld < b or t.data_ptr() % 16:
        raise ValueError("%s rows must start on 16-byte boundaries and not overlap" % name)
    return ld


def _scales4(t, name: str, groups: int, rows: int) -> int:
    """The scales of `rows` rows of `groups` groups: groups x rows x 8 with contiguous rows; the pitch of a group."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 3:
        raise ValueError("%s must be a 3-D tensor of uint8" % name)
    if tuple(t.shape) != (groups, rows, 8):
        raise ValueError("%s must be %d x %d x 8, got %s" % (name, groups, rows, tuple(t.shape)))
    if rows == 0:
        return 0
    s0, s1, s2 = t.stride()
    if s2 != 1 or (rows > 1 and s1 != 8):
        raise ValueError("%s must have the 8 bytes of a row, and the rows of a group, one behind the other" % name)
    ld = s0 if groups > 1 else 8 * rows
    if ld % 8 or ld < 8 * rows or t.data_ptr() % 8:
        raise ValueError("%s groups must start on 8-byte boundaries and not overlap" % name)
    return ld


def _made(rows: int, d: int, out, scales) -> Tuple[int, int]:
    """The pitches of the codes and scales of a call, given or to be made."""
    groups = mx4_groups(d)
    if (out is None) != (scales is None):
        raise ValueError("give out and scales together, or neither")
    if out is None:
        return 128 * groups, 8 * rows
    return _codes4(out, "out", rows, groups), _scales4(scales, "scales", groups, rows)


def _make(x: torch.Tensor, rows: int, d: int):
    groups = mx4_groups(d)
    return x.new_empty(rows, 128 * groups, dtype=torch.uint8), x.new_empty(groups, rows, 8, dtype=torch.uint8)


def _device(**tensors) -> int:
    """The device of the first of them, which all are on that are not None."""
    first, t = next(iter(tensors.items()))
    device = t.get_device()
    if device < 0:
        raise ValueError("%s must be a device tensor" % first)
    for name, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise ValueError("%s is on %s, not on device %d" % (name, t.device, device))
    return device


def _call(name: str, index: int, args):
    fn = _fns[name]
    rc = fn(*args, _raw_stream(index)) if index == _current() else _elsewhere(fn, index, args)
    if rc:
        _failed(rc, name)


def _bf(t) -> int:
    return 1 if t.dtype is torch.bfloat16 else 0


def quant4(x: torch.Tensor, scale: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
           status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of x (rows x d, bf16 or fp32) as (codes, scales): of x, of x silu(gate) with a gate, times the channel
    scale (d fp32) with one.  See qamw_quant4."""
    if out is None and scales is None and status is None and _host is not None:
        made = _host.quant4(x, scale, gate)
        if made is not None:
            return made
    ld_x = _rows(x, "x")
    rows, d = x.shape
    ld_g = _rows(gate, "gate", like=x) if gate is not None else 0
    if scale is not None:
        _vec(scale, "scale", d)
    if status is not None:
        _vec(status, "status", 1, torch.int32)
    ld_q, ld_e = _made(rows, d, out, scales)
    index = _device(x=x, gate=gate, scale=scale, out=out, scales=scales, status=status)
    if out is None:
        out, scales = _make(x, rows, d)
    _call("qamw_quant4", index, (x.data_ptr(), _bf(x), rows, d, ld_x, _ptr(gate), ld_g, _ptr(scale), out.data_ptr(), ld_q,
                                 scales.data_ptr(), ld_e, _ptr(status)))
    return out, scales


def dequant4(codes: torch.Tensor, scales: torch.Tensor, d: int, scale: Optional[torch.Tensor] = None,
             out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that codes stand for (rows x d, bf16 or fp32), with the channel scale that quant4 multiplied in
    divided out.  See qamw_dequant4."""
    if out is None and out_dtype in _VALUES and _host is not None:
        out = _host.dequant4(codes, scales, d, scale, out_dtype is torch.bfloat16)
        if out is not None:
            return out
    groups = mx4_groups(d)
    if d < 1:
        raise ValueError("d must be at least 1, got %d" % d)
    ld_q = _codes4(codes, "codes", groups=groups)
    rows = codes.shape[0]
    ld_e = _scales4(scales, "scales", groups, rows)
    if scale is not None:
        _vec(scale, "scale", d)
    ld_out = _out(out, out_dtype, rows, d)
    index = _device(codes=codes, scales=scales, scale=scale, out=out)
    if out is None:
        out = codes.new_empty(rows, d, dtype=out_dtype)
    _call("qamw_dequant4", index, (codes.data_ptr(), rows, d, ld_q, scales.data_ptr(), ld_e, _ptr(scale), out.data_ptr(),
                                   _bf(out), ld_out))
    return out


def rmsnorm4(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-5,
             residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Residual addition and root-mean-square norm: (codes of the normalized rows, their scales,
    h = x + residual).  Without a residual h is x itself, and sum_out (if given) a copy of it; sum_out may be x or
    residual (h in place).  h carries no gradient: but where it is x itself, x or residual that requires one is
    refused while gradients are recorded.  See qamw_rmsnorm4."""
    if sum_out is None and out is None and scales is None and status is None and _host is not None:
        made = _host.rmsnorm4(x, weight, eps, residual)
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
    if status is not None:
        _vec(status, "status", 1, torch.int32)
    ld_q, ld_e = _made(rows, d, out, scales)
    index = _device(x=x, residual=residual, sum_out=sum_out, weight=weight, out=out, scales=scales, status=status)
    if residual is not None and sum_out is None:
        sum_out = x.new_empty(rows, d)
    if out is None:
        out, scales = _make(x, rows, d)
    _call("qamw_rmsnorm4", index, (x.data_ptr(), _bf(x), rows, d, ld_x, _ptr(residual), ld_r, _ptr(weight), eps,
                                   _ptr(sum_out), ld_s, out.data_ptr(), ld_q, scales.data_ptr(), ld_e, _ptr(status)))
    return out, scales, x if sum_out is None else sum_out


def gemm4_workspace(M: int, d_out: int, groups: int) -> int:
    """Bytes of workspace that gemm4 uses (0 for most sizes, and for those that it refuses)."""
    if not all(-_INT_MAX <= size <= _INT_MAX for size in (M, d_out, groups)):   # ctypes would cut them to 32 bits
        return 0
    return _fns["qamw_gemm4_workspace"](M, d_out, groups)


def gemm4(xq: torch.Tensor, x_scales: torch.Tensor, wq: torch.Tensor, w_scales: torch.Tensor, out_dtype=torch.bfloat16,
          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x w^T of activations (M rows) and weights (d_out rows) in 4 bits: M x d_out, bf16 or fp32.  Calls that may
    overlap need a workspace each, or none given.  See qamw_gemm4."""
    if out is None and workspace is None and out_dtype in _VALUES and _host is not None:
        out = _host.gemm4(xq, x_scales, wq, w_scales, out_dtype is torch.bfloat16)
        if out is not None:
            return out
    ld_x, ld_w = _codes4(xq, "xq"), _codes4(wq, "wq")
    M, b = xq.shape
    N, groups = wq.shape[0], b // 128
    if wq.shape[1] != b:
        raise ValueError("xq has %d groups of columns, wq %d" % (groups, wq.shape[1] // 128))
    ld_xe, ld_we = _scales4(x_scales, "x_scales", groups, M), _scales4(w_scales, "w_scales", groups, N)
    ld_y = _out(out, out_dtype, M, N)
    need = _fns["qamw_gemm4_workspace"](M, N, groups)
    if workspace is not None:
        _vec(workspace, "workspace", need, torch.uint8)
    index = _device(xq=xq, x_scales=x_scales, wq=wq, w_scales=w_scales, out=out, workspace=workspace)
    if out is None:
        out = xq.new_empty(M, N, dtype=out_dtype)
    if workspace is None and need:
        workspace = xq.new_empty(need, dtype=torch.uint8)
    _call("qamw_gemm4", index, (xq.data_ptr(), ld_x, x_scales.data_ptr(), ld_xe, M, wq.data_ptr(), ld_w,
                                w_scales.data_ptr(), ld_we, N, groups, out.data_ptr(), _bf(out), ld_y, _ptr(workspace),
                                0 if workspace is None else workspace.numel()))
    return out


def _experts(wq, w_scales, groups: int) -> Tuple[int, int, int, int]:
    """Weights of experts (experts x d_out x bytes) and their scales (groups x experts x d_out x 8): the pitches of a
    row, of an expert, of a group of scales and of an expert's scales."""
    if not isinstance(wq, torch.Tensor) or wq.dtype != torch.uint8 or wq.dim() != 3:
        raise ValueError("wq must be a 3-D tensor of uint8")
    if not isinstance(w_scales, torch.Tensor) or w_scales.dtype != torch.uint8 or w_scales.dim() != 4:
        raise ValueError("w_scales must be a 4-D tensor of uint8")
    E, N, b = wq.shape
    if b != 128 * groups:
        raise ValueError("xq has %d groups of columns, wq %s" % (groups, b / 128))
    if tuple(w_scales.shape) != (groups, E, N, 8):
        raise ValueError("w_scales must be %d x %d x %d x 8, got %s" % (groups, E, N, tuple(w_scales.shape)))
    if E < 1:
        raise ValueError("wq has no experts")
    if E > _INT_MAX or N > _INT_MAX:
        raise ValueError("wq is too large: %s" % (tuple(wq.shape),))
    if N == 0:
        return b, 0, 0, 0
    ld_w, ld_we = _codes4(wq[0], "wq"), _scales4(w_scales[:, 0], "w_scales", groups, N)
    by_expert, scales_by_expert = (wq.stride(0), w_scales.stride(1)) if E > 1 else (0, 0)
    if by_expert % 16 or scales_by_expert % 8:
        raise ValueError("wq experts must start on 16-byte boundaries, their scales on 8-byte ones")
    return ld_w, by_expert, ld_we, scales_by_expert


def gemm4_grouped(xq: torch.Tensor, x_scales: torch.Tensor, wq: torch.Tensor, w_scales: torch.Tensor,
                  offsets: torch.Tensor, index: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows in groups, each with an expert's weights (wq: experts x d_out x bytes, w_scales: groups x experts x d_out x
    8, as quant4 leaves them for the experts' rows one behind the other, viewed): row i of y, for
    offsets[e] <= i < offsets[e + 1], is row index[i] of x (row i without an index; zeros for an index outside x) times
    expert e's weights.  offsets (experts + 1) and index (one for each row of y) are int32 on the device; rows of y that
    no group has are left as they were, so without `out` offsets should run from 0 to the rows of y.  See
    qamw_gemm4_grouped."""
    if out is None and out_dtype in _VALUES and _host is not None:
        out = _host.gemm4_grouped(xq, x_scales, wq, w_scales, offsets, index, out_dtype is torch.bfloat16)
        if out is not None:
            return out
    ld_x = _codes4(xq, "xq")
    x_rows, b = xq.shape
    groups = b // 128
    ld_xe = _scales4(x_scales, "x_scales", groups, x_rows)
    ld_w, by_expert, ld_we, scales_by_expert = _experts(wq, w_scales, groups)
    E, N = wq.shape[:2]
    _vec(offsets, "offsets", E + 1, torch.int32)
    rows = x_rows
    if index is not None:
        _vec(index, "index", 0, torch.int32)
        rows = index.numel()
        if rows > _INT_MAX:
            raise ValueError("index is too large: %d" % rows)
    ld_y = _out(out, out_dtype, rows, N)
    dev = _device(xq=xq, x_scales=x_scales, wq=wq, w_scales=w_scales, offsets=offsets, index=index, out=out)
    if out is None:
        out = xq.new_empty(rows, N, dtype=out_dtype)
    _call("qamw_gemm4_grouped", dev, (xq.data_ptr(), ld_x, x_scales.data_ptr(), ld_xe, x_rows, _ptr(index), rows,
                                      wq.data_ptr(), ld_w, by_expert, w_scales.data_ptr(), ld_we, scales_by_expert,
                                      offsets.data_ptr(), E, N, groups, out.data_ptr(), _bf(out), ld_y))
    return out
