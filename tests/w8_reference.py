"""Plain forms of the 8-bit row operators and the 8-bit product: numpy, with the roundings that
include/qamw_w8.h names and everything else in 64 bits."""
import numpy as np

ZERO_ROW = np.float32(2.0 ** -119)


def to_bf16(x):
    """fp32 -> the nearest bf16 value (ties to even), as fp32.  Finite or infinite x."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    r = ((b >> 16) & 1) + np.uint32(0x7FFF)
    return ((b + r) & np.uint32(0xFFFF0000)).view(np.float32)


def quantize(a):
    """(codes int8, top fp32, row scale fp32) of fp32 rows."""
    a = np.asarray(a, dtype=np.float32)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(a).all(1)
        top = np.where(bad, np.float32(0), np.abs(a).max(1)).astype(np.float32)
        zero = bad | (top < ZERO_ROW)
        back = np.where(zero, np.float32(0), np.float32(127) / np.where(zero, np.float32(1), top)).astype(np.float32)
        prod = np.where(zero[:, None], np.float32(0), a * back[:, None]).astype(np.float32)
        q = np.rint(prod).astype(np.int8)
        s = np.where(zero, np.float32(0), top / np.float32(127)).astype(np.float32)
    s[bad] = np.nan
    return q, top, s


def quant8(x, scale=None):
    a = np.asarray(x, dtype=np.float32)
    if scale is not None:
        with np.errstate(all="ignore"):
            a = (a * scale.astype(np.float32)).astype(np.float32)
    q, _, s = quantize(a)
    return q, s


def rmsnorm8(x, weight=None, eps=1e-5, residual=None):
    """(codes, row scale in 64 bits, h in fp32)."""
    h = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        if residual is not None:
            h = (h + np.asarray(residual, dtype=np.float32)).astype(np.float32)
        a = h if weight is None else (h * weight.astype(np.float32)).astype(np.float32)
        q, top, s0 = quantize(a)
        ms = (h.astype(np.float64) ** 2).sum(1) / h.shape[1] + float(np.float32(eps))
        s = np.where(s0 == 0, 0.0, top.astype(np.float64) / (127.0 * np.sqrt(ms)))
    s[np.isnan(s0)] = np.nan
    return q, s, h


def dequant8(q, s, scale=None):
    with np.errstate(all="ignore"):
        v = (q.astype(np.float32) * s[:, None].astype(np.float32)).astype(np.float32)
        if scale is not None:
            v = (v * (np.float32(1) / scale.astype(np.float32))).astype(np.float32)
    return v


def sums(xq, wq):
    """Exact sums of products, int64 (by fp64 products, exact below 2^53)."""
    return (xq.astype(np.float64) @ wq.astype(np.float64).T).astype(np.int64)


def gemm8(xq, xs, wq, ws):
    c = sums(xq, wq)
    with np.errstate(all="ignore"):
        y = (c.astype(np.float32) * xs[:, None].astype(np.float32)).astype(np.float32)
        return (y * ws[None, :].astype(np.float32)).astype(np.float32)
