"""Gated rows of quant8 on the GPU: the accuracy of silu, and a gate together with a channel scale."""
import numpy as np
import pytest
import torch

from helpers import DEV, log

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
