"""gemm4 and gemm4_grouped with scale bytes from one end to the other: what they stand for together counts, not each alone.

A step of the matrix instruction rounds its fp32 sum once: within 2^-23 of the largest magnitude in reach, or within
2^-149, the distance of the numbers below the normal ones.  K / 64 steps and as many additions of parts of k leave the bound of
test_gpu_mx4.py and (K / 64 + 16) 2^-149.  Sums whose magnitudes pass the fp32 range may be infinite or NaN on the way and
are left out.
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import DEV, log
from test_gpu_mx4 import _exact

pytestmark = pytest.mark.gpu

# bytes of x and w: ordinary numbers from extreme scales, the largest sums, sums at and below the normal numbers, none
BYTES = [(0, 254), (254, 0), (1, 253), (10, 244), (0, 230), (254, 100), (120, 252), (127, 5), (64, 64), (0, 127), (0, 120),
         (30, 85), (40, 60), (0, 0)]


def _codes(rng, n, groups, byte):
    c = rng.integers(0, 256, (n, groups * 128), dtype=np.uint8)
    s = np.full((groups, n, 8), byte, dtype=np.uint8)
    return torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), ref.read(c, s)


def _check(y, want, mag, groups):
    y, steps = y.double().cpu().numpy(), groups * 4 + 16
    ok = (np.abs(y - want) <= steps * (2.0 ** -23 * mag + 2.0 ** -149)) | (mag >= 2.0 ** 127)
    assert ok.all(), (np.argwhere(~ok)[:4], y[~ok][:4], want[~ok][:4])


# few rows, small tiles, 256 x 256, k in parts
@pytest.mark.parametrize("M,N,groups", [(1, 64, 2), (40, 100, 2), (300, 520, 3), (2300, 4500, 1), (77, 4096, 43)])
def test_scales_from_end_to_end(q, M, N, groups):
    rng = np.random.default_rng(M)
    for bx, bw in BYTES if M < 1000 and groups < 10 else BYTES[:2] + BYTES[6:13]:
        (xq, xs, xv), (wq, ws, wv) = _codes(rng, M, groups, bx), _codes(rng, N, groups, bw)
        log("gemm4 %d x %d, bytes %d and %d" % (M, N, bx, bw))
        _check(q.gemm4(xq, xs, wq, ws, out_dtype=torch.float32), *_exact(xv, wv), groups)
    # any scales beside one another
    xs.copy_(torch.from_numpy(rng.integers(0, 128, tuple(xs.shape), dtype=np.uint8)))
    ws.copy_(torch.from_numpy(rng.integers(0, 230, tuple(ws.shape), dtype=np.uint8)))
    want, mag = _exact(ref.read(xq.cpu().numpy(), xs.cpu().numpy()), ref.read(wq.cpu().numpy(), ws.cpu().numpy()))
    _check(q.gemm4(xq, xs, wq, ws, out_dtype=torch.float32), want, mag, groups)


@pytest.mark.parametrize("sizes", [[3, 0, 5], [70, 90, 10]])
def test_groups_with_scales_from_end_to_end(q, sizes):
    rng = np.random.default_rng(sum(sizes))
    ends, N, groups = np.cumsum([0] + sizes), 72, 2
    off = torch.from_numpy(ends.astype(np.int32)).to(DEV)
    for bx, bw in BYTES:
        (xq, xs, xv), (wq, ws, wv) = _codes(rng, sum(sizes), groups, bx), _codes(rng, len(sizes) * N, groups, bw)
        y = q.gemm4_grouped(xq, xs, wq.view(len(sizes), N, -1), ws.view(groups, len(sizes), N, 8), off, out_dtype=torch.float32)
        for e, n in enumerate(sizes):
            if n:
                _check(y[ends[e]:ends[e + 1]], *_exact(xv[ends[e]:ends[e + 1]], wv[e * N:(e + 1) * N]), groups)
