"""The 4-bit linear layers on the GPU against plain forms (mx4_reference.py).

Codes, scales and the values they stand for follow from operations that include/qamw_mx4.h names one by one, and are
compared bit for bit; where a rounding to fp32 rests on a sum or an exponential in fp64, either neighbour is
taken if the plain form's value is within the fp64 bound of the middle between them.

Products.  Values are e2m1 numbers times powers of two, products of two are exact, and a step of the matrix
instruction adds 64 of them to an fp32 sum: with an error of at most 2^-23 of the largest magnitude in reach, the
sum's or the step's.  K / 64 steps, and as many additions more for parts of k, leave
(K / 64 + 16) 2^-23 sum |x w|; bf16 adds half a step of the result, 2^-8 (1 + that).
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from helpers import DEV, log

pytestmark = pytest.mark.gpu

GUARD = 77


def _rows(a, dtype, pad=0, offset=0):
    """fp32 array -> device matrix of dtype with `pad` more elements a row and its first element `offset`
    elements into the buffer; NaN outside.  Also the values it holds, as fp32."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype)
    n, d = a.shape
    buf = torch.full((offset + n * (d + pad),), float("nan"), dtype=dtype, device=DEV)
    v = buf[offset:].view(n, d + pad)[:, :d]
    v.copy_(t.to(DEV))
    return v, t.float().numpy()


def _values(rng, n, d):
    a = rng.standard_normal((n, d)) * np.exp(rng.standard_normal((n, 1)))
    a[:, rng.integers(0, d, max(1, d // 64))] *= 20
    return a.astype(np.float32)


def _room(q, n, d, extra=0):
    """Room for codes with `extra` more bytes a row and a guard row behind them, and for scales with a guard row."""
    codes = torch.full((n + 1, q.mx4_stride(d) + extra), GUARD, dtype=torch.uint8, device=DEV)
    scales = torch.full((q.mx4_groups(d), n + 1, 8), GUARD, dtype=torch.uint8, device=DEV)
    return codes, scales, codes[:n, :q.mx4_stride(d)], scales[:, :n]


def _check_form(room, want, n):
    codes, scales, cv, sv = room
    wc, ws = want
    got_c, got_s = cv.cpu().numpy(), sv.cpu().numpy()
    assert np.array_equal(got_s, ws), "scales differ at %s" % (np.argwhere(got_s != ws)[:4],)
    assert np.array_equal(got_c, wc), "codes differ at %s" % (np.argwhere(got_c != wc)[:4],)
    assert (codes[n] == GUARD).all() and (codes[:, wc.shape[1]:] == GUARD).all() and (scales[:, n] == GUARD).all()


def _bf16(v):
    """fp64 -> fp32 -> bf16, as fp64."""
    return torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).double().numpy()


def _same(got, want):
    got = got.double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:4]


SHAPES = [(1, 1), (3, 7), (2, 31), (5, 32), (4, 33), (6, 255), (1, 256), (33, 257), (7, 1003), (1, 5120), (300, 4100),
          (5, 13824), (2, 40000), (700, 64), (4099, 300), (20000, 40), (9000, 300), (7001, 5), (12000, 17), (3000, 1003)]
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@TYPES
@pytest.mark.parametrize("n,d", SHAPES)
def test_quant4_and_back(q, n, d, dtype):
    rng = np.random.default_rng(n * 100003 + d)
    pad, offset, extra = [(0, 0, 0), (5, 3, 16), (d % 3, 1, 0)][(n + d) % 3]
    x, xf = _rows(_values(rng, n, d), dtype, pad, offset)
    scale = np.exp(rng.standard_normal(d)).astype(np.float32)
    sd = torch.from_numpy(scale).to(DEV)
    log("quant4 %d x %d %s pad %d" % (n, d, dtype, pad))
    for sc, st in ((None, None), (scale, sd)):
        want = ref.quantize(xf if sc is None else (xf * sc).astype(np.float32))
        room = _room(q, n, d, extra)
        flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
        c, s = q.quant4(x, scale=st, out=room[2], scales=room[3], status=flag)
        torch.cuda.synchronize()
        _check_form(room, want, n)
        assert flag.item() == 0
        for od in (torch.bfloat16, torch.float32):
            out = torch.full((n + 1, d + pad), 7.0, dtype=od, device=DEV)
            q.dequant4(c, s, d, scale=st, out=out[:n, :d])
            v = ref.read(*want, d).astype(np.float32)
            if sc is not None:
                v = v * (np.float32(1) / sc)
            _same(out[:n, :d], _bf16(v) if od == torch.bfloat16 else v.astype(np.float64))
            assert (out[n] == 7).all() and (out[:n, d:] == 7).all()
    c2, s2 = q.quant4(x)   # buffers of its own
    c3, s3 = q.quant4(x.contiguous())
    assert torch.equal(c2, c3) and torch.equal(s2, s3)
    assert tuple(c2.shape) == (n, q.mx4_stride(d)) and tuple(s2.shape) == (q.mx4_groups(d), n, 8)
    _same(q.dequant4(c2, s2, d), _bf16(ref.read(*ref.quantize(xf), d)))


@TYPES
@pytest.mark.parametrize("with_scale", [False, True])
@pytest.mark.parametrize("n,d", [(1, 1), (5, 17), (64, 1003), (3, 5120), (9, 13824), (700, 300), (9000, 75)])
def test_quant4_gated(q, n, d, with_scale, dtype):
    """Gate and up as the halves of one matrix.  A gated value is within 2^-38 of itself before it is rounded to
    fp32: the roundings of both ends of that range have to give the codes, block by block."""
    rng = np.random.default_rng(n + 7 * d)
    both = np.concatenate([3 * rng.standard_normal((n, d)), _values(rng, n, d)], 1).astype(np.float32)
    both[0, 0] = 100.0   # exp(-g) below and above the fp32 range
    both[-1, d - 1] = -100.0
    t, f = _rows(both, dtype, 3, 1)
    scale = np.exp(rng.standard_normal(d)).astype(np.float32) if with_scale else None
    c, s = q.quant4(t[:, d:], gate=t[:, :d], scale=None if scale is None else torch.from_numpy(scale).to(DEV))
    g, u = f[:, :d].astype(np.float64), f[:, d:].astype(np.float64)
    a = u * g / (1 + np.exp(-g))
    log("gated %d x %d %s" % (n, d, dtype))
    c, s = c.cpu().numpy(), s.cpu().numpy()
    forms = []
    for end in (1 - 2.0 ** -38, 1 + 2.0 ** -38):
        v = (a * end).astype(np.float32)
        forms.append(ref.quantize(v if scale is None else (v * scale).astype(np.float32)))
    fits = [(c.reshape(n, -1, 16) == fc.reshape(n, -1, 16)).all(2) & (s.transpose(1, 0, 2).reshape(n, -1) == fs.transpose(1, 0, 2).reshape(n, -1))
            for fc, fs in forms]
    # a block where the two ends differ may hold values of both; there are few of those
    apart = ~((forms[0][0].reshape(n, -1, 16) == forms[1][0].reshape(n, -1, 16)).all(2))
    assert (fits[0] | fits[1] | apart).all() and apart.mean() < 0.01


@TYPES
def test_gate_far_values(q, dtype):
    """Gates far from zero: silu(g) is g to within 2^-24 above, and below a number of any size down to 0."""
    g = np.array([-1e30, -800, -750, -700, -120, -104, -90, -88, -60, 40, 88, 90, 130, 800, 1e30, 0], dtype=np.float32)
    x = np.array([1.0, 1e30, -1e37, 1e-30], dtype=np.float32)
    gg, xx = [v.ravel() for v in np.meshgrid(g, x)]
    t, f = _rows(np.stack([gg, xx]), dtype)
    gg, xx = f
    with np.errstate(all="ignore"):
        a = ref.gate(xx, gg)
    keep = np.isfinite(a)   # one value a row, so that each has its own block
    c, s = q.quant4(t[1][:, None].contiguous(), gate=t[0][:, None].contiguous())
    wc, ws = ref.quantize(a[:, None])
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(c.cpu().numpy(), wc)
    assert keep.sum() > 40 and (ws[0, ~keep, 0] == 255).all()


def test_quant4_every_border(q):
    """Every border of two codes and its fp32 neighbours, both signs, at exponents over the whole range."""
    b = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], dtype=np.float32)
    v = np.concatenate([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(9)), [0.0, -0.0, 6, 7]]).astype(np.float32)
    v = np.concatenate([v, -v, [6.0] * (64 - 2 * len(v))]).astype(np.float32)
    v[31] = 6.0   # either block's largest value is 6 or 7
    a = np.stack([v * np.float32(2.0 ** e) for e in range(-121, 126)])
    c, s = q.quant4(torch.from_numpy(a).to(DEV))
    want = ref.quantize(a)
    assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    tops = np.array([3.5, 4, 6, 7, 7.5], dtype=np.float32)
    tops = np.concatenate([tops, np.nextafter(tops, np.float32(0)), np.nextafter(tops, np.float32(9))])
    a = np.zeros((len(tops), 32), dtype=np.float32)
    a[:, 7], a[:, 20] = tops, 1.0
    c, s = q.quant4(torch.from_numpy(a).to(DEV))
    want = ref.quantize(a)
    assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])


def test_quant4_special_blocks(q):
    d = 1000
    a = np.random.default_rng(5).standard_normal((12, d)).astype(np.float32)
    a[1] = 0
    a[2, 999] = np.nan
    a[3, 0] = np.inf
    a[4, 500] = -np.inf
    a[5] *= 1e-41            # denormals: zero blocks
    a[6] *= 1e-36            # at the border of a zero block
    a[7] = np.float32(3.4e38) * np.sign(a[7])   # the largest values
    a[8] = 0
    a[8, 3] = np.float32(2.0 ** -119)
    a[9] = 0
    a[9, 3] = np.nextafter(np.float32(2.0 ** -119), np.float32(0))
    a[10, ::2] = np.nan
    a[11, 64:96] = -0.0
    want = ref.quantize(a)
    flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
    x = torch.from_numpy(a).to(DEV)
    c, s = q.quant4(x, status=flag)
    assert np.array_equal(s.cpu().numpy(), want[1]) and np.array_equal(c.cpu().numpy(), want[0])
    assert flag.item() == q.FLAG_NONFINITE
    with np.errstate(all="ignore"):
        _same(q.dequant4(c, s, d, out_dtype=torch.float32), ref.read(*want, d).astype(np.float32).astype(np.float64))
    back = q.dequant4(c, s, d).float().cpu().numpy()
    assert np.isnan(back[2, 992:]).all() and np.isfinite(back[2, :992]).all() and not np.isnan(back[4, :480]).any()
    for rows, bits in (([0, 1, 5, 6, 8, 9, 11], 0), ([2], 1), ([3], 1), ([4], 1), ([10], 1)):
        flag.zero_()
        q.quant4(x[rows], status=flag)
        assert flag.item() == bits * q.FLAG_NONFINITE
    scale = torch.ones(d, device=DEV)
    for v in (0.0, -1.0, float("nan")):
        scale[d - 1] = v
        flag.zero_()
        q.quant4(x[:2].contiguous(), scale=scale, status=flag)
        assert flag.item() & q.FLAG_BAD_SCALE


def test_dequant4_every_code_and_scale(q):
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)[:, :128].contiguous()
    codes[:, 64:] = torch.arange(192, 256, dtype=torch.uint8, device=DEV)
    codes[:, :64] = torch.arange(0, 256, 4, dtype=torch.uint8, device=DEV)
    scales = torch.arange(256, dtype=torch.uint8, device=DEV)[None, :, None].expand(1, 256, 8).contiguous()
    with np.errstate(all="ignore"):
        v = ref.read(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)
    _same(q.dequant4(codes, scales, 256, out_dtype=torch.float32), v.astype(np.float64))
    got = q.dequant4(codes, scales, 256)
    assert torch.equal(got.nan_to_num(1e30), torch.from_numpy(v).to(DEV).to(torch.bfloat16).nan_to_num(1e30))


# ---------------------------------------------------------------- the norm

def _norm_forms(xf, rf, wf, eps):
    """h, and the forms with the norm's factor rounded from either end of its fp64 bound: a sum of d squares is
    within d 2^-53 of itself, and division and square root add a few roundings."""
    h = xf if rf is None else (xf + rf).astype(np.float32)
    f, e = ref.norm_factors(h, eps), (h.shape[1] + 8) * 2.0 ** -53
    return h, [ref.quantize(ref.normed(h, wf, (f * s).astype(np.float32))) for s in (1 - e, 1 + e)]


def _check_norm(room, forms, n):
    codes, scales, cv, sv = room
    c, s = cv.cpu().numpy(), sv.cpu().numpy()
    fits = [(c == fc).all(1) & (s == fs).all((0, 2)) for fc, fs in forms]
    assert (fits[0] | fits[1]).all(), np.argwhere(~(fits[0] | fits[1]))[:4]
    assert (codes[n] == GUARD).all() and (codes[:, c.shape[1]:] == GUARD).all() and (scales[:, n] == GUARD).all()


@TYPES
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (2, 33), (5, 256), (4, 257), (33, 513), (7, 1003), (1, 4096), (300, 4100),
                                 (1100, 5120), (3, 8200), (2, 13824), (3, 16400), (2, 24576), (2, 32768), (2050, 640), (5000, 43)])
def test_rmsnorm4(q, n, d, dtype):
    rng = np.random.default_rng(n * 7919 + d)
    pad, offset, extra = [(0, 0, 0), (5, 3, 16), (d % 3, 1, 0)][(n + d) % 3]
    x, xf = _rows(_values(rng, n, d), dtype, pad, offset)
    r, rf = _rows(3 * _values(rng, n, d), dtype, pad + 1, 1)
    w = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    log("rmsnorm4 %d x %d %s pad %d" % (n, d, dtype, pad))
    for res, resf, wt, wf in ((r, rf, wd, w), (None, None, wd, w), (r, rf, None, None), (None, None, None, None)):
        h, forms = _norm_forms(xf, resf, wf, 1e-5)
        room = _room(q, n, d, extra)
        flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
        out = torch.full((n + 1, d + pad), 7.0, dtype=dtype, device=DEV)
        c, s, got_h = q.rmsnorm4(x, wt, eps=1e-5, residual=res, sum_out=out[:n, :d], out=room[2], scales=room[3], status=flag)
        _check_norm(room, forms, n)
        assert flag.item() == 0
        _same(got_h, _bf16(h) if dtype == torch.bfloat16 else h.astype(np.float64))
        assert (out[n] == 7).all() and (out[:n, d:] == 7).all()
        c2, s2, h2 = q.rmsnorm4(x, wt, eps=1e-5, residual=res)
        assert torch.equal(c2, c) and torch.equal(s2, s) and torch.equal(h2, got_h)
        assert h2 is x if res is None else h2.is_contiguous()
    for over in ("x", "residual"):   # h in place
        xc, rc = x.clone(), r.clone()
        to = xc if over == "x" else rc
        c2, s2, h2 = q.rmsnorm4(xc, wd, residual=rc, sum_out=to)
        h, forms = _norm_forms(xf, rf, w, 1e-5)
        assert h2 is to
        _same(to, _bf16(h) if dtype == torch.bfloat16 else h.astype(np.float64))
        fits = [(c2.cpu().numpy() == fc).all(1) for fc, _ in forms]
        assert (fits[0] | fits[1]).all()


def test_rmsnorm4_special_rows(q):
    d = 700
    a = np.random.default_rng(6).standard_normal((7, d)).astype(np.float32)
    a[1] = 0
    a[2, 699] = np.nan
    a[3, 0] = np.inf
    a[4] *= 1e-30
    a[5] *= 1e30
    x = torch.from_numpy(a).to(DEV)
    flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
    c, s, _ = q.rmsnorm4(x, eps=1e-5, status=flag)
    assert flag.item() == q.FLAG_NONFINITE
    h, forms = _norm_forms(a, None, None, 1e-5)
    c, s = c.cpu().numpy(), s.cpu().numpy()
    for i in (0, 1, 4, 5, 6):
        assert any(np.array_equal(c[i], fc[i]) and np.array_equal(s[:, i], fs[:, i]) for fc, fs in forms), i
    # a row with a NaN is NaN as a whole; one with an infinity has factor 0: NaN there, 0 elsewhere
    assert (s[:, 2].reshape(-1)[:22] == 255).all() and s[0, 3, 0] == 255 and not c[2].any() and not c[3].any()
    assert not s[:, 3].reshape(-1)[1:].any()
    for rows, bits in (([0, 1, 4, 5, 6], 0), ([2], 1), ([3], 1)):
        flag.zero_()
        q.rmsnorm4(x[rows], status=flag)
        assert flag.item() == bits * q.FLAG_NONFINITE
    flag.zero_()
    c, s, _ = q.rmsnorm4(x[:2].contiguous(), eps=0.0, status=flag)   # a row of zeros has no norm
    assert flag.item() == q.FLAG_NONFINITE and (s[:, 1].reshape(-1)[:22] == 255).all() and s[0, 0, 0] != 255


# ---------------------------------------------------------------- products

def _form(q, rng, n, d, spread=0, extra=0):
    """Codes and scales of n x d values on the device (scales over `spread` binades more), and the values.  Of many
    values, codes drawn as such."""
    if n * d <= 300000:
        a = rng.standard_normal((n, d)).astype(np.float32)
        if spread:
            b = ref.blocks(a)
            a = (b * np.exp2(rng.integers(-spread, spread + 1, b.shape[:2] + (1,)))).astype(np.float32).reshape(n, -1)[:, :d]
        c, s = ref.quantize(a)
    else:
        c = rng.integers(0, 256, (n, q.mx4_stride(d)), dtype=np.uint8)
        s = rng.integers(125 - spread, 128 + spread, (q.mx4_groups(d), n, 8), dtype=np.uint8)
        c[:, (d + 1) // 2:] = 0
        if d % 2:
            c[:, d // 2] &= 15
    room = _room(q, n, d, extra)
    room[2].copy_(torch.from_numpy(c).to(DEV))
    room[3].copy_(torch.from_numpy(s).to(DEV))
    return room[2], room[3], ref.read(c, s)


def _exact(x, w):
    """The product and its sum of magnitudes in 64 bits, on the device."""
    x, w = torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV)
    return (x @ w.t()).cpu().numpy(), (x.abs() @ w.abs().t()).cpu().numpy()


def _check_product(y, want, mag, K, out):
    got = y.double().cpu().numpy()
    bound = (K / 64 + 16) * 2.0 ** -23 * mag
    if out == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want).max())


def _product(q, M, N, K, seed=0, spread=0):
    rng = np.random.default_rng(seed + M * 1009 + N * 13 + K)
    extra = [0, 16, 128][(M + N + K) % 3]
    xq, xs, xv = _form(q, rng, M, K, spread, extra)
    wq, ws, wv = _form(q, rng, N, K, spread)
    want, mag = _exact(xv, wv)
    log("gemm4 %d x %d x %d" % (M, N, K))
    first = None
    for out in (torch.float32, torch.bfloat16):
        pad = (M + N) % 3
        y = torch.full((M + 1, N + pad), 7.0, dtype=out, device=DEV)
        q.gemm4(xq, xs, wq, ws, out=y[:M, :N])
        _check_product(y[:M, :N], want, mag, K, out)
        assert (y[M] == 7).all() and (y[:M, N:] == 7).all()
        y2 = q.gemm4(xq, xs, wq, ws, out_dtype=out)
        assert torch.equal(y2, y[:M, :N])
        first = y2 if first is None else first
        # bf16 is the fp32 result rounded
        assert torch.equal(y2, first.to(out))
    return xq, xs, wq, ws, first


SMALL = [(1, 1, 1), (1, 33, 300), (2, 64, 256), (3, 100, 1003), (31, 31, 512), (32, 32, 257), (33, 65, 700), (64, 63, 2048),
         (65, 129, 4100), (7, 5, 13824), (130, 40, 600), (129, 257, 1000)]


@pytest.mark.parametrize("M,N,K", SMALL)
def test_gemm4_small(q, M, N, K):
    _product(q, M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 77, 1), (5, 300, 32), (40, 64, 8192), (300, 333, 1500), (257, 700, 5120)])
def test_gemm4_scales_of_any_size(q, M, N, K):
    _product(q, M, N, K, seed=1, spread=20)


# Sizes that go to each of the kernels, in the order of their choice (test_mx4_plan.py asserts that they do): tiles of 256
# x 256, one tile a workgroup and several, with one group of columns and more; 128 x 256; 128 x 128, k whole and in
# parts; 64 x 256; 32 x 256; 64 x 64; few rows, of each width.
KERNELS = [(857, 9539, 256), (2300, 4500, 200), (5000, 5000, 100), (5000, 5700, 700), (2049, 4100, 1200),
           (979, 5570, 256), (1300, 5300, 700), (1500, 5120, 5120),
           (131, 13841, 256), (515, 5120, 4096), (68, 5633, 12200), (2609, 747, 13200), (102, 2956, 13500),
           (130, 13121, 256), (276, 6348, 14800), (39, 10656, 13300), (47, 6050, 13500),
           (132, 11089, 256), (17, 13779, 11500), (91, 2881, 10400),
           (33, 16, 256), (77, 4096, 11008), (33, 4139, 6000), (51, 2111, 5500), (80, 158, 11400), (600, 2049, 700),
           (1, 5120, 5120), (8, 300, 1000), (9, 4096, 4000), (16, 13824, 5120), (17, 5120, 5000), (32, 333, 1700)]


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_gemm4_every_kernel(q, M, N, K):
    _product(q, M, N, K)


def test_gemm4_views(q):
    """Rows first to last of a matrix of codes, and of its scales, are a matrix of codes."""
    rng = np.random.default_rng(11)
    xq, xs, xv = _form(q, rng, 90, 700)
    wq, ws, wv = _form(q, rng, 80, 700)
    y = q.gemm4(xq, xs, wq, ws, out_dtype=torch.float32)
    for m0, m1, n0, n1 in ((1, 2, 3, 80), (7, 90, 0, 1), (33, 65, 5, 70)):
        part = q.gemm4(xq[m0:m1], xs[:, m0:m1], wq[n0:n1], ws[:, n0:n1], out_dtype=torch.float32)
        want, mag = ref.product(xv[m0:m1], wv[n0:n1])
        _check_product(part, want, mag, 768, torch.float32)
        assert (part - y[m0:m1, n0:n1]).abs().max() <= 32 * 2.0 ** -23 * mag.max()


def test_gemm4_nan_blocks(q):
    """A block that is NaN makes its row of x, its column of y, NaN, and nothing else."""
    rng = np.random.default_rng(12)
    for M, N, K in ((1, 40, 300), (40, 100, 2000), (300, 520, 600)):
        xq, xs, xv = _form(q, rng, M, K)
        wq, ws, wv = _form(q, rng, N, K)
        m, n = M // 2, N - 1
        xs[(K - 1) // 256, m, (K - 1) // 32 % 8] = 255
        xq[m, (K - 1) // 32 * 16:((K - 1) // 32 + 1) * 16] = 0
        ws[0, n, 0] = 255
        y = q.gemm4(xq, xs, wq, ws, out_dtype=torch.float32).cpu().numpy()
        nan = np.zeros((M, N), dtype=bool)
        nan[m], nan[:, n] = True, True
        assert np.array_equal(np.isnan(y), nan)


# ---------------------------------------------------------------- rows in groups

def _grouped_want(xv, wv, offsets, index, rows, N):
    """The rows that groups have (others NaN), and the sums of magnitudes."""
    want, mag = np.full((rows, N), np.nan), np.zeros((rows, N))
    xz = np.concatenate([xv, np.zeros((1, xv.shape[1]))])
    for e in range(len(offsets) - 1):
        at = np.arange(offsets[e], offsets[e + 1])
        if not len(at):
            continue
        r = at if index is None else np.where((index[at] < 0) | (index[at] >= len(xv)), len(xv), index[at])
        want[at], mag[at] = _exact(xz[r], wv[e])
    return want, mag


def _grouped(q, x_rows, sizes, N, K, indexed, first=0, behind=0, seed=0, extra=0):
    rng = np.random.default_rng(seed + x_rows * 31 + N * 7 + K + len(sizes))
    E = len(sizes)
    offsets = (first + np.concatenate([[0], np.cumsum(sizes)])).astype(np.int32)
    rows = int(offsets[-1]) + behind
    xq, xs, xv = _form(q, rng, x_rows, K, extra=extra)
    wq, ws, wv = _form(q, rng, E * N, K)
    wq, ws, wv = wq.view(E, N, -1), ws.reshape(ws.shape[0], E, N, 8), wv.reshape(E, N, -1)
    index = None
    if indexed:
        index = rng.integers(0, x_rows, rows).astype(np.int32)
        if rows > 3:
            index[rows // 3], index[rows // 2], index[rows - 1] = -1, x_rows, -2 ** 31
    else:
        assert rows == x_rows
    want, mag = _grouped_want(xv, wv, offsets, index, rows, N)
    od, idx = torch.from_numpy(offsets).to(DEV), None if index is None else torch.from_numpy(index).to(DEV)
    log("gemm4_grouped %d of %d rows, %d experts, %d x %d" % (rows, x_rows, E, N, K))
    have = ~np.isnan(want[:, :1]).all(1)
    for out in (torch.float32, torch.bfloat16):
        pad = N % 3
        y = torch.full((rows + 1, N + pad), 7.0, dtype=out, device=DEV)
        q.gemm4_grouped(xq, xs, wq, ws, od, index=idx, out=y[:rows, :N])
        got = y[:rows, :N]
        _check_product(got[torch.from_numpy(have).to(DEV)], want[have], mag[have], K, out)
        assert (y[rows] == 7).all() and (y[:, N:] == 7).all() and (got[torch.from_numpy(~have).to(DEV)] == 7).all()
        y2 = q.gemm4_grouped(xq, xs, wq, ws, od, index=idx, out_dtype=out)
        assert torch.equal(y2[torch.from_numpy(have).to(DEV)], got[torch.from_numpy(have).to(DEV)])
    return xq, xs, wq, ws, od, idx


GROUPS = [(1, [1], 1, 1), (2, [0, 2], 33, 300), (9, [4, 0, 0, 5], 65, 256), (40, [0, 33, 1, 6], 100, 700),
          (200, [64, 0, 129, 7], 300, 1003), (70, [1] * 70, 40, 512), (300, [0] * 64 + [255] + [0] * 40 + [45], 64, 600)]


@pytest.mark.parametrize("indexed", [False, True], ids=["rows", "index"])
@pytest.mark.parametrize("x_rows,sizes,N,K", GROUPS)
def test_grouped_small(q, x_rows, sizes, N, K, indexed):
    _grouped(q, x_rows, sizes, N, K, indexed)


def test_grouped_rows_without_a_group(q):
    """Rows before the first group and behind the last one keep what they had."""
    _grouped(q, 30, [3, 0, 9], 50, 300, True, first=4, behind=6)
    _grouped(q, 22, [3, 0, 9], 50, 300, False, first=4, behind=6)
    _grouped(q, 300, [100, 70], 200, 300, False, first=70, behind=60)


# The same for rows in groups: 256 x 256 (one tile a workgroup and several, more than 64 groups), 128 x 256, 64 x 256,
# 32 x 256, few rows.
GROUP_KERNELS = [(3000, [2000, 3074, 600], 5200, 256), (700, [3000, 3074, 600], 5200, 600), (2000, [9, 20000] + [0] * 63 + [19991], 1500, 200),
                 (1000, [37, 500, 1, 462], 5120, 1100), (5000, [60] * 80 + [900], 500, 300),
                 (400, [40] * 90 + [333, 7], 1024, 1800), (700, [300, 90, 610, 200], 1700, 256),
                 (515, [700, 0, 100, 230], 1024, 2048), (64, [33, 31], 5120, 5000),
                 (24, [3] * 31 + [40], 512, 4096), (70, [1] * 70, 40, 512), (100, [50, 0, 17, 133], 300, 900)]


@pytest.mark.parametrize("x_rows,sizes,N,K", GROUP_KERNELS)
def test_grouped_every_kernel(q, x_rows, sizes, N, K):
    _grouped(q, x_rows, sizes, N, K, True)
    if sum(sizes) < 4000:
        _grouped(q, sum(sizes), sizes, N, K, False, seed=1)


def test_grouped_equals_products(q):
    """Groups of rows in order, expert by expert, against gemm4 on the experts' slices."""
    xq, xs, wq, ws, od, _ = _grouped(q, 170, [40, 0, 100, 30], 96, 1000, False)
    y = q.gemm4_grouped(xq, xs, wq, ws, od, out_dtype=torch.float32)
    for e, (a, b) in enumerate(((0, 40), (40, 40), (40, 140), (140, 170))):
        part = q.gemm4(xq[a:b], xs[:, a:b], wq[e], ws[:, e], out_dtype=torch.float32)
        assert (part - y[a:b]).abs().max() < 1e-3 if b > a else part.numel() == 0
    # a slice of the experts, with offsets of their own
    some = torch.tensor([40, 140, 170], dtype=torch.int32, device=DEV)
    out = torch.full_like(y, 7.0)
    q.gemm4_grouped(xq, xs, wq[2:], ws[:, 2:], some, out=out)
    assert torch.equal(out[40:], y[40:]) and (out[:40] == 7).all()


def test_grouped_offsets_out_of_range(q):
    """Offsets are held to 0 .. rows on the device, a group that ends before it begins is empty: nothing outside the
    matrices is touched, and groups that are in order are right."""
    rng = np.random.default_rng(21)
    xq, xs, xv = _form(q, rng, 50, 300)
    wq, ws, wv = _form(q, rng, 4 * 40, 300)
    wq, ws, wv = wq.view(4, 40, -1), ws.reshape(2, 4, 40, 8), wv.reshape(4, 40, -1)
    for offsets in ([-5, 10, 20, 30, 70], [-2**31, 10, 20, 30, 2**31 - 1], [60, 70, 80, 90, 100], [0, 50, 50, 20, 20]):
        held = np.clip(offsets, 0, 50)
        room = torch.full((52, 40), 7.0, device=DEV)
        q.gemm4_grouped(xq, xs, wq, ws, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=room[1:51])
        assert (room[0] == 7).all() and (room[51] == 7).all()
        want, mag = _grouped_want(xv, wv, held, None, 50, 40)
        have = ~np.isnan(want).all(1)
        _check_product(room[1:51][torch.from_numpy(have).to(DEV)], want[have], mag[have], 512, torch.float32)
        assert (room[1:51][torch.from_numpy(~have).to(DEV)] == 7).all()


def test_grouped_all_indexes_outside(q):
    """Only rows of zeros, also of an x that has none."""
    rng = np.random.default_rng(22)
    wq, ws, _ = _form(q, rng, 2 * 40, 300)
    wq, ws = wq.view(2, 40, -1), ws.reshape(2, 2, 40, 8)
    off = torch.tensor([0, 3, 9], dtype=torch.int32, device=DEV)
    for n in (0, 1):
        xq, xs, _ = _form(q, rng, n, 300) if n else (torch.empty((0, 256), dtype=torch.uint8, device=DEV),
                                                    torch.empty((2, 0, 8), dtype=torch.uint8, device=DEV), None)
        y = q.gemm4_grouped(xq, xs, wq, ws, off, index=torch.full((9,), -1, dtype=torch.int32, device=DEV))
        assert tuple(y.shape) == (9, 40) and (y == 0).all()


# ---------------------------------------------------------------- in use

def test_experts_block(q):
    """A layer of experts as it is used: norm, router's choice, gate and up projection of the chosen rows, gated
    activation, down projection, weighted sum; each step against its plain form on the step's own inputs."""
    rng = np.random.default_rng(31)
    T, D, F, E, top = 37, 512, 320, 6, 2
    x, xf = _rows(_values(rng, T, D), torch.bfloat16)
    r, rf = _rows(_values(rng, T, D), torch.bfloat16)
    w = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32)
    up = (0.05 * rng.standard_normal((E * 2 * F, D))).astype(np.float32)
    down = (0.05 * rng.standard_normal((E * D, F))).astype(np.float32)
    uq, us = q.quant4(torch.from_numpy(up).to(DEV))
    dq, ds = q.quant4(torch.from_numpy(down).to(DEV))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    prob, chosen = logits.softmax(1).topk(top, 1)
    order = chosen.reshape(-1).argsort(stable=True)
    index = (order // top).to(torch.int32)
    offsets = torch.searchsorted(chosen.reshape(-1)[order], torch.arange(E + 1, device=DEV)).to(torch.int32)
    hq, hs, h = q.rmsnorm4(x, torch.from_numpy(w).to(DEV), residual=r)
    both = q.gemm4_grouped(hq, hs, uq.view(E, 2 * F, -1), us.view(-1, E, 2 * F, 8), offsets, index=index)
    aq, as_ = q.quant4(both[:, F:], gate=both[:, :F])
    y = q.gemm4_grouped(aq, as_, dq.view(E, D, -1), ds.view(-1, E, D, 8), offsets, out_dtype=torch.float32)
    out = torch.zeros((T, D), device=DEV).index_add_(0, index.long(), y * prob.reshape(-1)[order][:, None]) + h.float()

    off, idx = offsets.cpu().numpy(), index.cpu().numpy()
    hw, forms = _norm_forms(xf, rf, w, 1e-5)
    assert any(np.array_equal(hq.cpu().numpy(), f[0]) for f in forms)
    want, mag = _grouped_want(ref.read(hq.cpu().numpy(), hs.cpu().numpy()), ref.read(*ref.quantize(up)).reshape(E, 2 * F, -1),
                              off, idx, T * top, 2 * F)
    _check_product(both, want, mag, D, torch.bfloat16)
    bf = both.float().cpu().numpy()
    wc, wsc = ref.quantize(ref.gate(bf[:, F:], bf[:, :F]))
    assert (aq.cpu().numpy() == wc).mean() > 0.9999 and (as_.cpu().numpy() == wsc).mean() > 0.9999
    want, mag = _grouped_want(ref.read(aq.cpu().numpy(), as_.cpu().numpy()), ref.read(*ref.quantize(down)).reshape(E, D, -1),
                              off, None, T * top, D)
    _check_product(y, want, mag, F, torch.float32)
    assert out.shape == (T, D) and torch.isfinite(out).all()


def test_streams_and_graphs(q):
    """The operators on a stream of their own, and captured into a graph whose inputs change between replays."""
    rng = np.random.default_rng(41)
    T, D, N, E = 40, 700, 260, 3
    x = torch.from_numpy(_values(rng, T, D)).to(DEV).to(torch.bfloat16)
    wq, ws, _ = _form(q, rng, E * N, D)
    w3, ws4 = wq.view(E, N, -1), ws.reshape(ws.shape[0], E, N, 8)
    off = torch.tensor([0, 11, 11, 40], dtype=torch.int32, device=DEV)
    index = torch.randint(0, T, (40,), dtype=torch.int32, device=DEV)

    def step():
        c, s, h = q.rmsnorm4(x, residual=x)
        y = q.gemm4(c, s, wq, ws)
        z = q.gemm4_grouped(c, s, w3, ws4, off, index=index)
        c2, s2 = q.quant4(y[:, :N], gate=y[:, N:2 * N])
        return c, s, h, y, z, q.dequant4(c2, s2, N)

    want = step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = step()
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    for k in range(4):
        x.copy_(torch.from_numpy(_values(rng, T, D)).to(DEV))
        off.copy_(torch.tensor([0, 3 * k, 20 + k, 40], dtype=torch.int32))
        index.copy_(torch.randint(0, T, (40,), dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(made, want)), k
