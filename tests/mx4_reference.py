"""Plain forms of the 4-bit row operators and products: numpy, with the roundings that include/qamw_mx4.h names and
everything else in 64 bits."""
import numpy as np

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
ZERO_BLOCK = np.float32(2.0 ** -119)


def groups(d):
    return (d + 255) // 256


def blocks(a):
    n, d = a.shape
    out = np.zeros((n, groups(d) * 256), dtype=a.dtype)
    out[:, :d] = a
    return out.reshape(n, -1, 32)


def quantize(a):
    """(codes rows x stride, scales groups x rows x 8) of fp32 rows."""
    b = blocks(np.asarray(a, dtype=np.float32))
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(b).all(2)
        top = np.where(bad, np.float32(0), np.abs(b).max(2)).astype(np.float64)
        zero = bad | (top < ZERO_BLOCK)
        # the least E with top <= 7 2^E
        E = np.ceil(np.log2(np.where(zero, 1.0, top) / 7)).astype(int)
        E = np.where(top > 7 * 2.0 ** E, E + 1, np.where(top <= 7 * 2.0 ** (E - 1), E - 1, E))
        v = np.where(zero[:, :, None], 0.0, np.abs(b).astype(np.float64) * 2.0 ** -E[:, :, None])
        # distance to every value; of two at the same distance the even code
        far = np.abs(np.minimum(v, 6.0)[..., None] - VALUES)
        near = far == far.min(-1, keepdims=True)
        even = near & (np.arange(8) % 2 == 0)
        code = np.where(even.any(-1), np.argmax(even, -1), np.argmax(near, -1)) + 8 * np.signbit(b)
    code = np.where(zero[:, :, None], 0, code).astype(np.uint8).reshape(len(b), -1)
    byte = np.where(bad, 255, np.where(zero, 0, E + 127)).astype(np.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, np.ascontiguousarray(byte.reshape(len(b), -1, 8).transpose(1, 0, 2))


def read(codes, scales, d=None):
    """The values of codes and scales in 64 bits; NaN where the scale byte is 255."""
    n = len(codes)
    c = np.empty((n, 2 * codes.shape[1]), dtype=int)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = np.where(c > 7, -1, 1) * VALUES[c % 8]
    byte = scales.transpose(1, 0, 2).reshape(n, -1).astype(int)
    unit = np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
    return (v.reshape(n, -1, 32) * unit[:, :, None]).reshape(n, -1)[:, :d]


def gate(x, g):
    """fl32(x g / (1 + exp(-g)))."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(g, dtype=np.float64)
    with np.errstate(all="ignore"):
        return (x * g / (1 + np.exp(-g))).astype(np.float32)


def norm_factors(h, eps):
    """1 / sqrt(mean square + eps) of fp32 rows in 64 bits (sums in extended precision)."""
    ms = (h.astype(np.longdouble) ** 2).sum(1) / h.shape[1] + np.longdouble(np.float32(eps))
    with np.errstate(all="ignore"):
        return (1 / np.sqrt(ms)).astype(np.float64)


def normed(h, weight, f):
    """fl32(fl32(h w) f)."""
    a = h if weight is None else (h * weight.astype(np.float32)).astype(np.float32)
    with np.errstate(all="ignore"):
        return (a * f.astype(np.float32)[:, None]).astype(np.float32)


def product(x, w):
    """(x w^T, sum of magnitudes) in 64 bits."""
    with np.errstate(all="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T
