"""Gated rows of quant8 on the GPU: the accuracy of silu, and a gate together with a channel scale."""
import numpy as np
import pytest
import torch

import w8_reference as ref
from helpers import DEV, log
from test_gpu_w8 import MANY, _check_codes, _code_buffer, _rows, _same, _values

pytestmark = pytest.mark.gpu


def test_silu_over_its_range(q):
    """Rows of one value, x = 2^40 (exact in the product with silu): the row scale gives silu(g) back, over the whole
    range of g, with one rounding more (the division by 127, 2^-24).  The header's bound on silu is (|g| + 8) 2^-23."""
    rng = np.random.default_rng(21)
    g = np.concatenate([rng.uniform(-87.0, 0.0, 6000), rng.uniform(0.0, 120.0, 3000), rng.standard_normal(6000),
                        np.array([-87.0, -1e-30, 1e-30, 1.0, -1.0, 88.0, 120.0, 3e38])]).astype(np.float32)
    x = np.where(g > 1e6, np.float32(0.5), np.float32(2.0 ** 40))
    _, s = q.quant8(torch.from_numpy(x[:, None]).to(DEV), gate=torch.from_numpy(g[:, None]).to(DEV))
    g64 = g.astype(np.float64)
    e = np.exp(-np.abs(g64))
    want = np.abs(g64) * np.where(g64 >= 0, 1.0, e) / (1.0 + e) * x
    keep = want >= 2.0 ** -119
    off = np.abs(s.cpu().numpy().astype(np.float64) * 127.0 - want)[keep] / want[keep]
    part = off / ((np.abs(g64[keep]) + 8) * 2.0 ** -23 + 2.0 ** -24)
    log("silu: %d values, at most %.2f of the bound" % (keep.sum(), part.max()))
    assert keep.sum() > 15000
    assert part.max() <= 1.0, g[keep][part.argmax()]


def test_silu_far_below(q):
    """Where exp(-g) exceeds 2^126, silu is 0, whatever finite value it is multiplied with."""
    g = torch.tensor([-87.4, -88.0, -89.0, -100.0, -1e4, -1e30, -3.4e38], device=DEV)[:, None]
    flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
    c, s = q.quant8(torch.full_like(g, 3.4e38), gate=g, status=flag)
    assert (s == 0).all() and (c == 0).all() and flag.item() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", [(1, 1), (5, 17), (64, 1003), (3, 5120), (9, 13824), (2, 32768), (300, 4100)])
def test_gate_and_scale(q, n, d, dtype):
    """With a the exact row x silu(g) s, the kernel's is off by the header's bound on silu, (|g| + 8) 2^-23, and by two
    roundings of products, 2^-24 each; the row scale and the codes as without a channel scale."""
    rng = np.random.default_rng(3 * n + 11 * d)
    both = np.concatenate([3 * rng.standard_normal((n, d)), _values(rng, n, d)], 1).astype(np.float32)
    scale = np.exp(rng.standard_normal(d)).astype(np.float32)
    t, f = _rows(both, dtype, 3, 1)
    log("gate and scale %d x %d %s" % (n, d, dtype))
    buf, flag = _code_buffer(n, d, 16), torch.zeros((1,), dtype=torch.int32, device=DEV)
    sd = torch.from_numpy(scale).to(DEV)
    c, s = q.quant8(t[:, d:], gate=t[:, :d], scale=sd, out=buf[:n, :d], status=flag)
    c2, s2 = q.quant8(t[:, d:], gate=t[:, :d], scale=sd)
    assert torch.equal(c, c2) and torch.equal(s, s2) and flag.item() == 0
    g, u, s64 = f[:, :d].astype(np.float64), f[:, d:].astype(np.float64), scale.astype(np.float64)
    a = u * g / (1 + np.exp(-g)) * s64
    e = ((np.abs(g) + 8) * 2.0 ** -23 + 2.0 ** -23) * np.abs(a)
    _check_codes(buf, n, d, c2.cpu().numpy())   # padding and what lies outside
    rs, codes = s.cpu().numpy().astype(np.float64), c.cpu().numpy().astype(np.float64)
    top, et = np.abs(a).max(1), e.max(1)
    assert np.all(np.abs(rs - top / 127) <= et / 127 + rs * 2.0 ** -23)
    assert np.all(np.abs(codes * rs[:, None] - a) <= e + rs[:, None] * (0.5 + 2.0 ** -15))
    _same(q.dequant8(c, s, scale=sd, out_dtype=torch.float32), ref.dequant8(c.cpu().numpy(), s.cpu().numpy(), scale))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", [(1, 5), (37, 511), (200, 5120)] + MANY)
def test_gate_and_scale_exact(q, n, d, dtype):
    """silu(0) = 0 and silu(100) = 100 exactly in fp32: codes and scales of the rows fl32(100 x) s bit for bit, at every
    number of chunks a thread, and zeros elsewhere."""
    rng = np.random.default_rng(n * 31 + d)
    x, xf = _rows(_values(rng, n, d), dtype, 1, 1)
    scale = np.exp(0.5 * rng.standard_normal(d)).astype(np.float32)
    sd = torch.from_numpy(scale).to(DEV)
    gate = torch.full((n, d), 100.0, device=DEV)
    gate[1::3] = 0
    gate[:, ::7] = 0
    log("gate and scale, exact %d x %d %s" % (n, d, dtype))
    want, ws = ref.quant8(np.where(gate.cpu().numpy() == 0, np.float32(0), xf * np.float32(100)), scale)
    buf = _code_buffer(n, d)
    c, s = q.quant8(x, gate=gate.to(dtype), scale=sd, out=buf[:n, :d])
    _check_codes(buf, n, d, want)
    _same(s, ws)
    _same(q.dequant8(c, s, scale=sd).float(), ref.to_bf16(ref.dequant8(want, ws, scale)))


def test_gate_and_bad_scale(q):
    """A channel scale that is not above 0 is reported with a gate too, wherever it stands, also where the gate closes
    its channel."""
    n, d = 3, 1003
    flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
    for at in (0, 500, d - 1):
        for v in (0.0, -2.0, float("nan")):
            scale = torch.ones((d,), device=DEV)
            scale[at] = v
            flag.zero_()
            q.quant8(torch.ones((n, d), device=DEV), gate=torch.zeros((n, d), device=DEV), scale=scale, status=flag)
            assert flag.item() & q.FLAG_BAD_SCALE, (at, v)
