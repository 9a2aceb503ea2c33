"""The 4-bit operators where offsets pass 32 bits: rows far apart, and outputs of more than 2^32 bytes."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import DEV, log
from test_gpu_mx4 import _check_product, _exact, _form, _values

pytestmark = pytest.mark.gpu


def _far(n, pitch, dtype):
    """A buffer of n rows `pitch` elements apart."""
    return torch.empty((n * pitch,), dtype=dtype, device=DEV).view(n, pitch)


def test_rows_far_apart(q):
    """Rows 2^31 bytes apart, of inputs, gates, residuals, codes and values."""
    n, d = 3, 700
    rng = np.random.default_rng(1)
    x = _far(n, 1 << 30, torch.bfloat16)[:, :d]
    out = _far(n, 1 << 31, torch.uint8)[:, :q.mx4_stride(d)]
    a, b = (torch.from_numpy(_values(rng, n, d)).to(torch.bfloat16) for _ in range(2))
    x.copy_(a.to(DEV))
    scales = torch.empty((3, n, 8), dtype=torch.uint8, device=DEV)
    want = ref.quantize(a.float().numpy())
    log("quant4 far")
    q.quant4(x, out=out, scales=scales)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    log("dequant4 far")
    back = _far(n, 1 << 30, torch.bfloat16)[:, :d]
    q.dequant4(out, scales, d, out=back)
    assert torch.equal(back.cpu().double(), torch.from_numpy(ref.read(*want, d)).to(torch.bfloat16).double())
    log("rmsnorm4 far")
    back.copy_(b.to(DEV))
    c, s, h = q.rmsnorm4(x, residual=back, sum_out=back, out=out, scales=scales)
    c2, s2, h2 = q.rmsnorm4(a.to(DEV), residual=b.to(DEV))
    assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(h, h2)


def test_scales_far_apart(q):
    """Groups of scales 2^31 bytes apart."""
    rng = np.random.default_rng(2)
    xq, xs, xv = _form(q, rng, 70, 700)
    wq, ws, wv = _form(q, rng, 300, 700)
    far = torch.empty((3 << 31,), dtype=torch.uint8, device=DEV).view(3, -1)
    fx, fw = far[:, 8:8 + 560].view(3, 70, 8), far[:, 4096:4096 + 2400].view(3, 300, 8)
    fx.copy_(xs), fw.copy_(ws)
    want, mag = _exact(xv, wv)
    log("gemm4 with far scales")
    for m in (1, 70):
        y = q.gemm4(xq[:m], fx[:, :m], wq, fw, out_dtype=torch.float32)
        _check_product(y, want[:m], mag[:m], 768, torch.float32)


def test_weights_and_output_past_32_bits(q):
    """66000 x 33000 of output (4.4 GB of bf16), from weight rows 2^18 bytes apart (8.6 GB); and the last rows of it as
    groups of their own, of experts that lie as far apart."""
    M, N, K = 66000, 33000, 300
    rng = np.random.default_rng(3)
    xq, xs, xv = _form(q, rng, M, K)
    wq, ws, wv = _form(q, rng, N, K)
    far = torch.empty((N, 1 << 18), dtype=torch.uint8, device=DEV)[:, :256]
    far.copy_(wq)
    log("gemm4 %d x %d x %d" % (M, N, K))
    y = q.gemm4(xq, xs, far, ws)
    rows, cols = [0, 1, 32541, 65535, 65536, M - 1], [0, 31, 16384, 32767, 32768, N - 1]
    want, mag = ref.product(xv[rows], wv[cols])
    _check_product(y[rows][:, cols], want, mag, 512, torch.bfloat16)
    last = q.gemm4(xq[-300:], xs[:, -300:], wq, ws)
    assert torch.equal(y[-300:], last)
    log("gemm4 of few rows")
    few = q.gemm4(xq[-5:], xs[:, -5:], far, ws, out_dtype=torch.float32)
    want, mag = ref.product(xv[-5:], wv[cols])
    _check_product(few[:, cols], want, mag, 512, torch.float32)
    log("gemm4_grouped")
    experts, es = far.view(3, N // 3, 256), ws.view(2, 3, N // 3, 8)
    off = torch.tensor([0, 30000, 65000, M], dtype=torch.int32, device=DEV)
    z = q.gemm4_grouped(xq, xs, experts, es, off)
    for r, e in ((0, 0), (29999, 0), (30000, 1), (65000, 2), (M - 1, 2)):
        some = [0, 5000, N // 3 - 1]
        want, mag = ref.product(xv[r:r + 1], wv[[e * (N // 3) + c for c in some]])
        _check_product(z[r:r + 1][:, some], want, mag, 512, torch.bfloat16)


def test_many_rows(q):
    """More rows than a launch has workgroups of."""
    n, d = 1 << 21, 40
    x = torch.randn((n, d), device=DEV)
    c, s = q.quant4(x)
    c2, s2, _ = q.rmsnorm4(x)
    for at in (0, n // 2 - 1, n - 3):
        want = ref.quantize(x[at:at + 3].cpu().numpy())
        assert np.array_equal(c[at:at + 3].cpu().numpy(), want[0]) and np.array_equal(s[:, at:at + 3].cpu().numpy(), want[1])
        part = q.rmsnorm4(x[at:at + 3])
        assert torch.equal(c2[at:at + 3], part[0]) and torch.equal(s2[:, at:at + 3], part[1])
    v = q.dequant4(c, s, d, out_dtype=torch.float32)
    assert torch.equal(v[-3:].cpu().double(), torch.from_numpy(ref.read(c[-3:].cpu().numpy(), s[:, -3:].cpu().numpy(), d)))
