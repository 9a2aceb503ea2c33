"""quant4 where its inputs, or the values on the way to its codes, are below the normal fp32 numbers.

A gated value is x silu(g) to within 2^-38, rounded to fp32 once, and is multiplied by the channel scale only then; so
every block has to hold the codes of one end of that range or of the other.
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import DEV, log

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -149   # the smallest fp32 number


def _gated(q, x, g, dtype, scale=None):
    """quant4 of rows gated by g against both ends of the bound, block by block."""
    xt, gt = (torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(dtype) for v in (x, g))
    x, g = xt.double().numpy(), gt.double().numpy()
    n = len(x)
    flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
    c, s = q.quant4(xt.to(DEV), gate=gt.to(DEV), scale=None if scale is None else torch.from_numpy(scale).to(DEV), status=flag)
    c, s = c.cpu().numpy().reshape(n, -1, 16), s.cpu().numpy().transpose(1, 0, 2).reshape(n, -1)
    a = x * g / (1 + np.exp(-g))
    assert np.isfinite(a.astype(np.float32)).all()
    fits = np.zeros(s.shape, dtype=bool)
    for end in (1 - 2.0 ** -38, 1 + 2.0 ** -38):
        v = (a * end).astype(np.float32)
        wc, ws = ref.quantize(v if scale is None else (v * scale).astype(np.float32))
        fits |= (c == wc.reshape(n, -1, 16)).all(2) & (s == ws.transpose(1, 0, 2).reshape(n, -1))
    assert fits.all(), "%d of %d blocks, first %s" % ((~fits).sum(), fits.size, np.argwhere(~fits)[:4])
    assert flag.item() == 0


def _each(x, g):
    """Every x with every g, one a row (so that each has its own block)."""
    return [v.reshape(-1, 1) for v in np.meshgrid(np.float32(x), np.float32(g))]


def test_gates_below_the_normal_numbers(q):
    k = np.concatenate([np.arange(1, 40), 2 ** np.arange(6, 24), 2 ** np.arange(6, 24) + 1, [999, 2 ** 23 - 1, 2 ** 24, 2 ** 25 + 3]])
    g = np.concatenate([k, -k]) * LEAST
    x = [2.0 ** 100, -2.0 ** 127, 1.7e25, 3.3e38, 1.2345e20, 2.0 ** 29, 5e8, 2.0 ** 24, 1.0, -1e-3, 2.0 ** -126, 0.0]
    _gated(q, *_each(x, g), torch.float32)


def test_every_bf16_gate_below_the_normal_numbers(q):
    g = np.arange(1, 256) * 2.0 ** -133   # and the first normal ones
    _gated(q, *_each([2.0 ** 100, 1.7e25, 3.3e38, -2.0 ** 30], np.concatenate([g, -g])), torch.bfloat16)


@pytest.mark.parametrize("n,d", [(64, 1003), (5, 40), (300, 256)])
def test_blocks_with_small_gates(q, n, d):
    """Blocks of such gates alone, among zeros, and beside ordinary ones."""
    rng = np.random.default_rng(n + d)
    x = rng.standard_normal((n, d)) * 1e25
    g = rng.integers(1, 1000, (n, d)) * rng.choice([-1, 1], (n, d)) * LEAST
    g[1::4][rng.random(g[1::4].shape) < 0.8] = 0
    x[2::4, ::3] = 0
    g[3::4, ::7] = rng.standard_normal(g[3::4, ::7].shape)
    x[3::4, ::7] = 1e-20
    log("small gates %d x %d" % (n, d))
    _gated(q, x, g, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("power", [-3, 2, 3, 7, 20, 60, 100])
def test_small_gated_values_with_a_scale(q, power, dtype):
    """x silu(g) below the normal numbers, rounded there, and a channel scale that makes normal numbers of it."""
    rng = np.random.default_rng(abs(power))
    n, d = 96, 600
    # products from 2^-160 (zeros, or next to them) to 2^-115 (above every zero block), by a small x, by a small gate, by a gate far below 0
    size = np.exp2(rng.uniform(-160, -115, (n, d)))
    g = rng.standard_normal((n, d))
    g[1::3] = np.exp2(rng.uniform(-100, -60, g[1::3].shape))
    g[2::3] = rng.uniform(-79, -20, g[2::3].shape)
    x = size * rng.choice([-1, 1], (n, d)) / np.abs(g / (1 + np.exp(-g)))
    x[:, ::9] = 0
    g[:, ::11] = 0
    scale = (2.0 ** power * np.exp(rng.standard_normal(d))).astype(np.float32)
    log("gated values with a scale of 2^%d" % power)
    _gated(q, x, g, dtype, scale)
    # each by itself
    _gated(q, x[:, :32].reshape(-1, 1), g[:, :32].reshape(-1, 1), dtype, scale[:1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_gated_values_next_to_a_rounding_with_a_scale(q, dtype):
    """Gated values beside the middle of two subnormal numbers, closer than fp32 operations tell: the scale shows on
    which side they were rounded."""
    rng = np.random.default_rng(3)
    if dtype == torch.float32:
        g = rng.uniform(-79, -20, 4000).astype(np.float32).astype(np.float64)
        middle = (rng.integers(0, 12, 4000) + 0.5) * LEAST * (1 + rng.choice([-1, 1], 4000) * np.exp2(rng.uniform(-22, -19, 4000)))
        x = middle / (g / (1 + np.exp(-g)))
    else:   # of many, those that are there
        g, x = (torch.from_numpy(v).to(dtype).double().numpy() for v in (rng.uniform(-79, -20, 1 << 23), -np.exp2(rng.uniform(-80, -30, 1 << 23))))
        a = x * g / (1 + np.exp(-g)) / LEAST
        near = (a < 12) & (np.abs(a - np.floor(a) - 0.5) < 2.0 ** -17 * a) & (np.abs(a - np.floor(a) - 0.5) > 2.0 ** -34)
        g, x = g[near], x[near]
        assert len(g) > 20
    _gated(q, x[:, None], g[:, None], dtype, np.array([2.0 ** 80], dtype=np.float32))


def test_small_values_keep_their_sign(q):
    """Subnormal values in a block of normal ones: code 0 with their sign; in a block of their own a zero block."""
    a = np.random.default_rng(8).standard_normal((40, 300)).astype(np.float32)
    a[:, 1::3] *= np.float32(1e-41)
    a[:20, 32:64] *= np.float32(1e-39)
    c, s = q.quant4(torch.from_numpy(a).to(DEV))
    want = ref.quantize(a)
    assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    assert (want[0] & 0x88).any()
