"""The 8-bit operators on matrices whose rows lie far apart."""
import numpy as np
import pytest
import torch

import w8_reference as ref
from helpers import DEV, log
from test_gpu_w8 import _code_matrix, _product, _same, _values, _want

pytestmark = pytest.mark.gpu


def _far(n, d, dtype):
    """n x d with 2^31 bytes from a row to the next: the fourth row starts behind 2^32 bytes."""
    return torch.empty((n, 2**31 // dtype.itemsize), dtype=dtype, device=DEV)[:, :d]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_rows_far_apart(q, dtype):
    n, d = 4, 1003
    rng = np.random.default_rng(31)
    a, b = _values(rng, n, d), _values(rng, n, d)
    x, r, codes, out = (_far(n, d, t) for t in (dtype, dtype, torch.int8, dtype))
    x.copy_(torch.from_numpy(a))
    r.copy_(torch.from_numpy(b))
    xf, rf = x.float().cpu().numpy(), r.float().cpu().numpy()
    w = np.exp(0.3 * rng.standard_normal(d)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    log("rows far apart %s" % dtype)
    rounded = lambda v: ref.to_bf16(v) if dtype == torch.bfloat16 else v
    want, ws = ref.quant8(xf, w)
    c, s = q.quant8(x, scale=wd, out=codes)
    assert np.array_equal(c.cpu().numpy(), want)
    _same(s, ws)
    q.dequant8(codes, s, scale=wd, out=out)
    _same(out.float(), rounded(ref.dequant8(want, ws, w)))
    # a gate of 100 leaves 100 x exactly
    want, ws = ref.quant8(xf * np.float32(100))
    out.fill_(100)
    q.quant8(x, gate=out, out=codes, row_scale=s)
    assert np.array_equal(codes.cpu().numpy(), want)
    _same(s, ws)
    # h to a matrix of its own, and in place
    want, s64, h = ref.rmsnorm8(xf, w, 1e-5, rf)
    for sum_out in (out, r, x):
        _, s, hs = q.rmsnorm8(x, wd, residual=r, sum_out=sum_out, out=codes)
        assert np.array_equal(codes.cpu().numpy(), want)
        # one rounding, and fp64 sums of 1003 squares in another order
        assert np.all(np.abs(s.cpu().numpy() - s64) <= s64 * (2.0 ** -24 + 2.0 ** -36))
        _same(hs.float(), rounded(h))
        r.copy_(torch.from_numpy(b))


# products with one matrix at the largest pitch, 2^22 bytes, and past 2^32 bytes in all: of the kernel for few rows
# (its weights), and of 256 x 256 tiles (offsets of up to 255 rows within a tile)
FAR_FEW = [(4, 1030, 2049), (40, 1030, 2049)]
FAR_TILES = [(1100, 9000, 1000), (9000, 1100, 1000)]


@pytest.mark.parametrize("M,N,K", FAR_FEW + FAR_TILES)
def test_products_far_apart(q, M, N, K):
    rng = np.random.default_rng(M + N)
    x_far = M == 1100   # otherwise the weights
    big = M if x_far else N
    far = torch.empty((big, q.w8.GEMM8_MAX_LD), dtype=torch.int8, device=DEV)[:, :K]
    far.copy_(_code_matrix(rng, big, K))
    near = _code_matrix(rng, N if x_far else M, K)
    xq, wq = (far, near) if x_far else (near, far)
    xs, ws = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    log("gemm8 far M=%d N=%d K=%d" % (M, N, K))
    for od in (torch.bfloat16, torch.float32):
        assert torch.equal(_product(q, xq, xs, wq, ws, od), _want(xq, xs, wq, ws, od))
