"""The 8-bit linear layers on the GPU against plain forms (w8_reference.py).

Almost everything is compared bit for bit: a row's codes and scale, the values they stand for and the
product follow from fp32 operations that include/qamw_w8.h names one by one, and sums of code products
are exact.  Two results are compared within a bound instead: the norm's row scale (its sum of squares is
taken in fp64 in another order: one fp32 rounding, 2^-24 relative, and far less for the order) and gated
rows (the header's bound on silu).
"""
import numpy as np
import pytest
import torch

import w8_reference as ref
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


def _code_buffer(n, d, extra=0):
    """Room for codes with `extra` more bytes a row, and a guard row behind them."""
    pitch = (d + 15) // 16 * 16 + extra
    return torch.full((n + 1, pitch), GUARD, dtype=torch.int8, device=DEV)


def _check_codes(buf, n, d, want):
    got = buf.cpu().numpy()
    padded = (d + 15) // 16 * 16
    assert np.array_equal(got[:n, :d], want), "codes differ at %s" % (np.argwhere(got[:n, :d] != want)[:4],)
    assert not got[:n, d:padded].any(), "padding bytes"
    assert (got[:n, padded:] == GUARD).all() and (got[n] == GUARD).all(), "bytes outside the rows"


def _same(got, want):
    got = got.cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:4]


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 15), (4, 16), (6, 17), (1, 511), (33, 513), (7, 1003), (1, 5120), (300, 4100),
          (2, 8192), (3, 8200), (5, 13824), (2, 16384), (3, 16400), (2, 24576), (2, 32768), (700, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", SHAPES)
def test_quant8_and_back(q, n, d, dtype):
    rng = np.random.default_rng(n * 100003 + d)
    pad, offset, extra = [(0, 0, 0), (5, 3, 16), (d % 3, 1, 0)][(n + d) % 3]
    x, xf = _rows(_values(rng, n, d), dtype, pad, offset)
    scale = np.exp(rng.standard_normal(d)).astype(np.float32)
    sd = torch.from_numpy(scale).to(DEV)
    log("quant8 %d x %d %s pad %d" % (n, d, dtype, pad))
    for sc, st in ((None, None), (scale, sd)):
        want, ws = ref.quant8(xf, sc)
        buf = _code_buffer(n, d, extra)
        rs = torch.full((n + 1,), 7.0, device=DEV)
        flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
        c, s = q.quant8(x, scale=st, out=buf[:n, :d], row_scale=rs, status=flag)
        torch.cuda.synchronize()
        _check_codes(buf, n, d, want)
        _same(rs[:n], ws)
        assert rs[n] == 7.0 and flag.item() == 0
        buf[:, d:] = 55   # bytes past the row mean nothing
        for od in (torch.bfloat16, torch.float32):
            out = torch.full((n + 1, d + pad), 7.0, dtype=od, device=DEV)
            q.dequant8(c, rs, scale=st, out=out[:n, :d])
            v = ref.dequant8(want, ws, sc)
            _same(out[:n, :d].float(), ref.to_bf16(v) if od == torch.bfloat16 else v)
            assert (out[n] == 7).all() and (out[:n, d:] == 7).all()
    c2, s2 = q.quant8(x)   # buffers of its own
    c3, s3 = q.quant8(x.contiguous())
    assert torch.equal(c2, c3) and torch.equal(s2, s3) and c2.stride(0) == q.q8_stride(d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", [(1, 1), (5, 17), (64, 1003), (3, 5120), (9, 13824), (2, 32768)])
def test_quant8_gated(q, n, d, dtype):
    """Gate and up as the halves of one matrix.  With a the exact row, the kernel's a' is off by
    e_j = ((|g_j| + 8) 2^-23 + 2^-24) |a_j| (silu, its product with x), the largest value by max e_j,
    the row scale by that / 127 and one rounding, and a value read back by half a step more."""
    rng = np.random.default_rng(n + 7 * d)
    both = np.concatenate([3 * rng.standard_normal((n, d)), _values(rng, n, d)], 1).astype(np.float32)
    both[0, 0] = 100.0   # exp(-g) below and above the fp32 range
    both[-1, d - 1] = -100.0
    t, f = _rows(both, dtype, 3, 1)
    c, s = q.quant8(t[:, d:], gate=t[:, :d])
    g, u = f[:, :d].astype(np.float64), f[:, d:].astype(np.float64)
    a = u * g / (1 + np.exp(-g))
    e = ((np.abs(g) + 8) * 2.0 ** -23 + 2.0 ** -24) * np.abs(a) + 2.0 ** -100 * np.abs(u)
    log("gated %d x %d %s" % (n, d, dtype))
    s, c = s.cpu().numpy().astype(np.float64), c.cpu().numpy().astype(np.float64)
    top, et = np.abs(a).max(1), e.max(1)
    assert np.all(np.abs(s - top / 127) <= et / 127 + s * 2.0 ** -23)
    assert np.all(np.abs(c * s[:, None] - a) <= e + s[:, None] * (0.5 + 2.0 ** -15))
    # the largest value of a row has code 127, but in a zero row (the 1 x 1 case: its gate is -100, and
    # silu(-100) = -3.7e-42 is below 2^-119, whatever x is)
    assert np.all(np.abs(c).max(1) == np.where(top < 2.0 ** -119, 0, 127))


def test_quant8_special_rows(q):
    d = 1000
    a = np.random.default_rng(5).standard_normal((12, d)).astype(np.float32)
    a[1] = 0
    a[2, 999] = np.nan
    a[3, 0] = np.inf
    a[4, 500] = -np.inf
    a[5] *= 1e-41            # denormals: a zero row
    a[6] *= 1e-36            # at the border of a zero row
    a[7] = np.float32(3.4e38) * np.sign(a[7])   # the largest values
    a[8] = 0
    a[8, 3] = np.float32(2.0 ** -119)
    a[9] = 0
    a[9, 3] = np.nextafter(np.float32(2.0 ** -119), np.float32(0))
    a[10, ::2] = np.nan
    want, ws = ref.quant8(a)
    flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
    x = torch.from_numpy(a).to(DEV)
    c, s = q.quant8(x, status=flag)
    _same(s, ws)
    assert np.array_equal(c.cpu().numpy(), want) and flag.item() == q.FLAG_NONFINITE
    assert ws[8] > 0 and ws[9] == 0
    back = q.dequant8(c, s).float().cpu().numpy()
    for i in range(12):
        assert np.isnan(back[i]).all() == bool(np.isnan(ws[i])), i
    c, s = q.quant8(x)   # no status: the same answer
    _same(s, ws)
    # a gate that is not finite marks its row as a value does
    for v in (np.nan, np.inf, -np.inf):
        g = np.zeros((2, d), dtype=np.float32)
        g[1, 77] = v
        flag.zero_()
        _, s = q.quant8(torch.ones((2, d), device=DEV), gate=torch.from_numpy(g).to(DEV), status=flag)
        assert s[0] == 0 and torch.isnan(s[1]) and flag.item() == q.FLAG_NONFINITE
    for v in (0.0, -1.0, np.nan):
        sc = torch.ones((d,), device=DEV)
        sc[d - 1] = v
        flag.zero_()
        q.quant8(torch.ones((2, d), device=DEV), scale=sc, status=flag)
        assert flag.item() & q.FLAG_BAD_SCALE


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", SHAPES)
def test_rmsnorm8(q, n, d, dtype):
    rng = np.random.default_rng(n * 99991 + d)
    x, xf = _rows(_values(rng, n, d), dtype, 2, 1)
    r, rf = _rows(4 * _values(rng, n, d), dtype, 0, 3)
    w = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    log("rmsnorm8 %d x %d %s" % (n, d, dtype))
    for res, weight, eps in ((True, True, 1e-5), (False, True, 0.0), (True, False, 1e-2)):
        want, s64, h = ref.rmsnorm8(xf, w if weight else None, eps, rf if res else None)
        buf = _code_buffer(n, d)
        flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
        hb = torch.full((n + 1, d + 1), 7.0, dtype=dtype, device=DEV)
        c, s, hs = q.rmsnorm8(x, wd if weight else None, eps=eps, residual=r if res else None, out=buf[:n, :d],
                              sum_out=hb[:n, :d], status=flag)
        _check_codes(buf, n, d, want)
        s = s.cpu().numpy().astype(np.float64)
        # one rounding, and fp64 sums of up to 32768 squares in another order
        assert np.all(np.abs(s - s64) <= s64 * (2.0 ** -24 + 2.0 ** -36)), np.abs(s / s64 - 1).max()
        _same(hb[:n, :d].float(), ref.to_bf16(h) if dtype == torch.bfloat16 else h)
        assert (hb[n] == 7).all() and (hb[:, d] == 7).all() and flag.item() == 0
    # in place over the residual, and over x
    for over in ("residual", "x"):
        x2, r2 = x.clone(), r.clone()
        c2, s2, h2 = q.rmsnorm8(x2, wd, residual=r2, sum_out=r2 if over == "residual" else x2)
        c1, s1, h1 = q.rmsnorm8(x, wd, residual=r)
        assert torch.equal(c1, c2) and torch.equal(s1, s2) and torch.equal(h1, h2)
        assert h2.data_ptr() == (r2 if over == "residual" else x2).data_ptr()
        assert torch.equal(x2 if over == "residual" else r2, x if over == "residual" else r)
    c1, s1, h1 = q.rmsnorm8(x, wd)
    assert h1 is x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", [(2000, 4936), (1500, 13000), (900, 5000), (1200, 20480), (4000, 700)])
def test_rmsnorm8_in_place_many_rows(q, n, d, dtype):
    """h over x, in rows that several wavefronts share and whose last chunks do not fill them: no wavefront
    sees what another one has already written."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n + d)
    x = torch.randn((n, d), generator=gen, device=DEV)
    x[:, -8:] *= 10   # the largest values last
    x = x.to(dtype)
    r = x.clone()
    w = torch.rand((d,), generator=gen, device=DEV) + 0.5
    log("in place %d x %d %s" % (n, d, dtype))
    c1, s1, h1 = q.rmsnorm8(x, w, residual=r)
    for over in (0, 1):
        for _ in range(3):
            x2, r2 = x.clone(), r.clone()
            c2, s2, h2 = q.rmsnorm8(x2, w, residual=r2, sum_out=r2 if over else x2)
            assert torch.equal(s1, s2) and torch.equal(c1, c2) and torch.equal(h1, h2)


# enough rows for the kernels that hold 2 to 8 chunks a thread, each with lanes that have none at their last chunk
MANY = [(6000, 520), (1500, 2056), (800, 4001), (620, 5120), (400, 8192), (230, 13824), (180, 17000), (150, 20480),
        (95, 32768)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,d", MANY)
def test_many_rows(q, n, d, dtype):
    rng = np.random.default_rng(n + d)
    x, xf = _rows(_values(rng, n, d), dtype, 0, 0)
    r, rf = _rows(_values(rng, n, d), dtype, 1, 1)
    w = np.exp(0.3 * rng.standard_normal(d)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    log("many rows %d x %d %s" % (n, d, dtype))
    for sc, st in ((None, None), (w, wd)):
        want, ws = ref.quant8(xf, sc)
        buf = _code_buffer(n, d)
        _, s = q.quant8(x, scale=st, out=buf[:n, :d])
        _check_codes(buf, n, d, want)
        _same(s, ws)
        want, s64, h = ref.rmsnorm8(xf, sc, 1e-5, rf)
        buf = _code_buffer(n, d)
        _, s, hs = q.rmsnorm8(x, st, residual=r, out=buf[:n, :d])
        _check_codes(buf, n, d, want)
        s = s.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(s - s64) <= s64 * (2.0 ** -24 + 2.0 ** -36))
        _same(hs.float(), ref.to_bf16(h) if dtype == torch.bfloat16 else h)
    # gated: silu(0) = 0 exactly, and silu(100) = 100 in fp32: codes and scales of the rows 100 x, where the gate
    # is 100, and zeros elsewhere
    gate = torch.full((n, d), 100.0, device=DEV)
    gate[::3] = 0
    c, s = q.quant8(x, gate=gate.to(dtype))
    want, ws = ref.quant8(np.where(np.arange(n)[:, None] % 3 == 0, np.float32(0), xf * np.float32(100)))
    assert np.array_equal(c.cpu().numpy(), want)
    _same(s, ws)


def test_rmsnorm8_special_rows(q):
    d = 520
    a = np.random.default_rng(6).standard_normal((8, d)).astype(np.float32)
    a[1] = 0
    a[2, 519] = np.nan
    a[3, 8] = np.inf
    a[4] *= np.float32(1e30)   # squares past fp32
    a[5] *= np.float32(1e-30)  # squares below fp32
    a[6] = np.float32(3e38)
    r = np.zeros_like(a)
    r[6] = np.float32(3e38)    # the sum overflows
    for eps in (1e-5, 0.0):
        want, s64, h = ref.rmsnorm8(a, None, eps, r)
        flag = torch.zeros((1,), dtype=torch.int32, device=DEV)
        c, s, hs = q.rmsnorm8(torch.from_numpy(a).to(DEV), eps=eps, residual=torch.from_numpy(r).to(DEV), status=flag)
        s = s.cpu().numpy()
        assert np.array_equal(c.cpu().numpy(), want) and flag.item() == q.FLAG_NONFINITE
        assert np.array_equal(np.isnan(s), np.isnan(s64)) and s[1] == 0
        ok = ~np.isnan(s64)
        assert np.all(np.abs(s[ok] - s64[ok]) <= s64[ok] * (2.0 ** -24 + 2.0 ** -36))
        _same(hs, h)


# ------------------------------------------------------------------------------------- the product

def _code_matrix(rng, n, k, extra=0, low=-128):
    """Random codes in a buffer with junk past every row; the view and its values."""
    pitch = (k + 15) // 16 * 16 + extra
    full = torch.from_numpy(rng.integers(low, 128, (n, pitch), dtype=np.int8)).to(DEV)
    return full[:, :k]


def _product(q, xq, xs, wq, ws, od, pad=0, workspace=None):
    M, N = xq.shape[0], wq.shape[0]
    out = torch.full((M + 1, N + pad), 7.0, dtype=od, device=DEV)
    q.gemm8(xq, xs, wq, ws, out=out[:M, :N], workspace=workspace)
    torch.cuda.synchronize()
    assert (out[M] == 7).all() and (out[:M, N:] == 7).all(), "wrote outside the output"
    return out[:M, :N]


def _want(xq, xs, wq, ws, od):
    """The plain form, with the exact sums formed on the GPU in fp64 (below 2^53)."""
    c = torch.mm(xq.double(), wq.double().t().contiguous())
    y = c.float() * xs[:, None]   # |c| < 2^31: the conversion from fp64 rounds the whole number once
    y = y * ws[None, :]
    return y.to(od)


def _check_product(q, M, N, K, od, extra=0, pad=0, seed=0):
    rng = np.random.default_rng(M * 1000003 + N * 1009 + K + seed)
    xq, wq = _code_matrix(rng, M, K, extra), _code_matrix(rng, N, K, 16 if extra else 0)
    xs = torch.from_numpy(np.exp(rng.standard_normal(M)).astype(np.float32)).to(DEV)
    ws = torch.from_numpy(np.exp(rng.standard_normal(N)).astype(np.float32)).to(DEV)
    log("gemm8 M=%d N=%d K=%d %s" % (M, N, K, od))
    got = _product(q, xq, xs, wq, ws, od, pad)
    want = _want(xq, xs, wq, ws, od)
    bad = got != want
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 64, 65, 77, 127, 128, 129, 200, 256, 257, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (17, 15), (100, 130), (64, 1003), (272, 257), (1000, 512)])
def test_gemm8_small(q, M, N, K):
    od = torch.bfloat16 if (M + N) % 2 else torch.float32
    _check_product(q, M, N, K, od, extra=(M % 3) * 32, pad=M % 2)


@pytest.mark.parametrize("K", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 640,
                               1000, 2049])
@pytest.mark.parametrize("M,N", [(3, 40), (40, 72), (130, 140), (600, 520)])
def test_gemm8_depths(q, M, N, K):
    _check_product(q, M, N, K, torch.float32)


@pytest.mark.parametrize("M,N,K", [
    (1, 5120, 5120), (16, 13824, 5120), (5, 5120, 13824), (33, 4096, 4096), (77, 4096, 11008), (128, 11008, 4096),
    (200, 5120, 13824), (512, 5120, 5120), (1500, 5120, 5120), (2048, 13824, 5120), (1000, 4100, 1111),
    (4097, 300, 2000), (300, 20000, 700), (3000, 3001, 999)])
def test_gemm8_large(q, M, N, K):
    for od in (torch.bfloat16, torch.float32):
        _check_product(q, M, N, K, od)


# Sizes at which each kind of tile is chosen, with k whole and in parts, most with a ragged end of k, and the
# kernel for few rows at each of its widths.
@pytest.mark.parametrize("M,N,K", [
    (1233, 7060, 756), (786, 9426, 17),                                       # 256 x 256
    (1275, 4960, 440), (273, 11373, 18), (200, 5833, 12948), (1502, 1393, 12032),     # 256 x 128
    (896, 4143, 346), (133, 11089, 17), (431, 1691, 11717), (87, 2768, 11524),        # 128 x 128
    (2336, 607, 820), (3285, 269, 21), (679, 350, 11734), (2401, 16, 11536),          # 128 x 64
    (433, 2830, 62), (200, 4153, 18), (47, 6050, 11362), (17, 13930, 13109),          # 64 x 128
    (131, 757, 53), (405, 85, 4879), (1, 19, 11132), (127, 213, 6194),                # 64 x 64
    (8, 5120, 1001), (9, 4568, 6656), (32, 13824, 640), (33, 1365, 2049), (63, 4102, 4090)])   # few rows
def test_gemm8_every_kernel(q, M, N, K):
    for od in (torch.bfloat16, torch.float32):
        _check_product(q, M, N, K, od, extra=16 * (M % 2), pad=N % 2)


def test_gemm8_deepest(q):
    """K at its limit, every product at its largest: sums of 131071 * 2^14 < 2^31."""
    K = q.w8.GEMM8_MAX_COLS
    for M, N in ((1, 20), (20, 300), (300, 300)):
        one = torch.ones
        for a, b in ((-128, -128), (-128, 127), (127, 127)):
            full = (M, K // 16 * 16 + 16)
            xq = torch.full(full, a, dtype=torch.int8, device=DEV)[:, :K]
            wq = torch.full((N, full[1]), b, dtype=torch.int8, device=DEV)[:, :K]
            y = _product(q, xq, one(M, device=DEV), wq, one(N, device=DEV), torch.float32)
            assert (y == float(np.float32(K * a * b))).all(), (M, N, a, b)


def test_gemm8_scales_propagate(q):
    """Zero scales give zeros, NaN scales (rows with a value that is not finite) NaN, and nothing else."""
    rng = np.random.default_rng(3)
    for M in (4, 40, 300):
        xq, wq = _code_matrix(rng, M, 256), _code_matrix(rng, 300, 256)
        xs, ws = torch.ones(M, device=DEV), torch.ones(300, device=DEV)
        xs[1], ws[7] = float("nan"), float("nan")
        xs[2], ws[8] = 0.0, 0.0
        y = _product(q, xq, xs, wq, ws, torch.float32)
        nan = torch.isnan(y)
        assert nan[1].all() and nan[:, 7].all() and int(nan.sum()) == 300 + M - 1
        assert (y[2][~nan[2]] == 0).all() and (y[:, 8][~nan[:, 8]] == 0).all()


def test_gemm8_far_offsets(q):
    """Matrices whose bytes pass 2^31 and 2^32 from their start: activations, weights and output."""
    K, ld = 96, 1 << 22
    rng = np.random.default_rng(4)
    for M, N in ((1030, 40), (40, 1030), (4, 1030)):
        big, small = max(M, N), min(M, N)
        buf = torch.zeros((big, ld), dtype=torch.int8, device=DEV)   # 4 GiB and more
        far, near = buf[:, :K], _code_matrix(rng, small, K)
        far.copy_(_code_matrix(rng, big, K))
        xq, wq = (far, near) if M == big else (near, far)
        xs, ws = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
        log("gemm8 far M=%d N=%d" % (M, N))
        assert torch.equal(_product(q, xq, xs, wq, ws, torch.float32), _want(xq, xs, wq, ws, torch.float32))
        del buf, far, xq, wq
    M, N, ldy = 1100, 33, 1 << 20   # 4.3 GiB of output
    xq, wq, xs, ws = _code_matrix(rng, M, K), _code_matrix(rng, N, K), torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    out = torch.zeros((M, ldy), dtype=torch.float32, device=DEV)
    q.gemm8(xq, xs, wq, ws, out=out[:, :N])
    assert torch.equal(out[:, :N], _want(xq, xs, wq, ws, torch.float32))
    assert int((out[:, N:] != 0).sum()) == 0


# --------------------------------------------------------------------------------- used together

def _mlp(q, x, h, norm, w_gu, w_down):
    """Norm, gate and up, gate, down: one MLP block of a W8A8 model, without its last addition."""
    c, s, h = q.rmsnorm8(x, norm, residual=h)
    gu = q.gemm8(c, s, *w_gu)
    f = gu.shape[1] // 2
    c2, s2 = q.quant8(gu[:, f:], gate=gu[:, :f])
    return q.gemm8(c2, s2, *w_down), h, (c, s, gu, c2, s2)


def _mlp_case(q, T, d, f, seed=0):
    rng = np.random.default_rng(seed)
    g = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)
    w_gu = q.quant8((0.05 * g(2 * f, d)).bfloat16())
    w_down = q.quant8((0.05 * g(d, f)).bfloat16())
    return g(T, d).bfloat16(), (2 * g(T, d)).bfloat16(), 1 + 0.1 * g(d), w_gu, w_down


@pytest.mark.parametrize("T", [1, 19, 150])
def test_mlp_block(q, T):
    """The block on the GPU against the block in fp64 on the same 8-bit weights.  Each stage adds its
    8-bit rounding: an error of at most half a step of 1/127 of a row's largest value, of uniform
    distribution: for Gaussian rows of 512 (largest about 3.2 sigma) 0.0073 sigma, for gated rows of 1000
    (heavier, largest at most 12 times their rms) 0.028 rms; gate and up also carry the bf16 rounding.
    The norm's part passes the gate with a factor below 2; all together below 5% of the result's rms."""
    d, f = 512, 1000
    x, h0, norm, w_gu, w_down = _mlp_case(q, T, d, f)
    y, h, (c, s, gu, c2, s2) = _mlp(q, x, h0, norm, w_gu, w_down)
    # every stage on the stage before it
    want, s64, h32 = ref.rmsnorm8(x.float().cpu().numpy(), norm.cpu().numpy(), 1e-5, h0.float().cpu().numpy())
    assert np.array_equal(c.cpu().numpy(), want)
    assert torch.equal(gu, _want(c, s, *w_gu, torch.bfloat16)) and torch.equal(y, _want(c2, s2, *w_down, torch.bfloat16))
    # and the whole
    hd = x.double() + h0.double()
    n = hd / torch.sqrt((hd ** 2).mean(1, keepdim=True) + 1e-5) * norm.double()
    w1, w2 = (q.dequant8(*w, out_dtype=torch.float32).double() for w in (w_gu, w_down))
    both = n @ w1.t().contiguous()
    act = both[:, f:] * both[:, :f] * torch.sigmoid(both[:, :f])
    yd = act @ w2.t().contiguous()
    rel = float((y.double() - yd).norm() / yd.norm())
    log("mlp T=%d relative error %.4f" % (T, rel))
    assert rel < 0.05


@pytest.mark.parametrize("T", [1, 24, 150])
def test_mlp_block_in_a_graph(q, T):
    """Captured once, replayed with other inputs and eager work between: every replay as the eager call."""
    x, h0, norm, w_gu, w_down = _mlp_case(q, T, 512, 1000, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _mlp(q, x, h0, norm, w_gu, w_down)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, _ = _mlp(q, x, h0, norm, w_gu, w_down)
    for i in range(4):
        x.copy_(torch.randn_like(x))
        h0.copy_(torch.randn_like(h0))
        want_y, want_h, _ = _mlp(q, x, h0, norm, w_gu, w_down)
        torch.cuda.synchronize()
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(h, want_h), i


def test_two_graphs_and_a_shared_workspace(q):
    """Two products captured into graphs of their own, with a workspace of the caller's that both use, one
    replayed after the other on one stream."""
    rng = np.random.default_rng(11)
    cases = []
    for M, N, K in ((77, 4096, 11008), (200, 1024, 4096)):
        assert q.gemm8_workspace(M, N, K) > 0
        cases.append((_code_matrix(rng, M, K), torch.rand(M, device=DEV), _code_matrix(rng, N, K),
                      torch.rand(N, device=DEV)))
    need = max(q.gemm8_workspace(c[0].shape[0], c[2].shape[0], c[0].shape[1]) for c in cases)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    want = [_want(*c, torch.bfloat16) for c in cases]
    graphs, outs = [], []
    for c in cases:
        outs.append(torch.zeros((c[0].shape[0], c[2].shape[0]), dtype=torch.bfloat16, device=DEV))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.gemm8(*c, out=outs[-1], workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_empty_matrices(q):
    e = lambda *s, **k: torch.empty(s, device=DEV, **k)
    c, s = q.quant8(e(0, 64, dtype=torch.bfloat16))
    assert c.shape == (0, 64) and s.shape == (0,)
    assert q.dequant8(c, s).shape == (0, 64)
    c, s, h = q.rmsnorm8(e(0, 64), residual=e(0, 64))
    assert c.shape == (0, 64) and h.shape == (0, 64)
    w = torch.zeros((5, 64), dtype=torch.int8, device=DEV)
    assert q.gemm8(c, s, w, torch.ones(5, device=DEV)).shape == (0, 5)
    assert q.gemm8(w, torch.ones(5, device=DEV), c, s).shape == (5, 0)


def _host_calls(q, rng):
    """Ordinary calls, and the same for the compiled module."""
    h = q.w8._host
    T = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV)
    x, wide, w = T(37, 1003), T(9, 640).bfloat16(), T(1003).abs() + 0.1
    c, s = q.quant8(T(37, 1003))
    big = torch.zeros((40, 1024), dtype=torch.int8, device=DEV)
    cw, sw = _code_matrix(rng, 50, 1003, 16), T(50).abs()
    return [
        (lambda: q.quant8(x), lambda: h.quant8(x, None, None)),
        (lambda: q.quant8(x, scale=w), lambda: h.quant8(x, w, None)),
        (lambda: q.quant8(wide[:, 320:], gate=wide[:, :320]), lambda: h.quant8(wide[:, 320:], None, wide[:, :320])),
        (lambda: q.dequant8(c, s), lambda: h.dequant8(c, s, None, True)),
        (lambda: q.dequant8(c, s, scale=w, out_dtype=torch.float32), lambda: h.dequant8(c, s, w, False)),
        (lambda: q.dequant8(big[:37, 16:1019], s), lambda: h.dequant8(big[:37, 16:1019], s, None, True)),
        (lambda: q.rmsnorm8(x, w, eps=1e-3), lambda: h.rmsnorm8(x, w, 1e-3, None)),
        (lambda: q.rmsnorm8(x, residual=x), lambda: h.rmsnorm8(x, None, 1e-5, x)),
        (lambda: q.gemm8(c, s, cw, sw), lambda: h.gemm8(c, s, cw, sw, True)),
        (lambda: q.gemm8(c, s, cw, sw, out_dtype=torch.float32), lambda: h.gemm8(c, s, cw, sw, False)),
    ]


def test_both_ways_through_the_binding(q, monkeypatch):
    """The compiled module takes the ordinary calls, and gives what the long way through w8.py gives."""
    flat = lambda r: [t.clone() for t in (r if isinstance(r, tuple) else (r,))]
    for call, direct in _host_calls(q, np.random.default_rng(13)):
        short, made = flat(call()), direct()
        assert made is not None
        made = flat(made)
        with monkeypatch.context() as m:
            m.setattr(q.w8, "_host", None)
            long = flat(call())
        for a, b, c in zip(short, long, made):
            assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
            assert torch.equal(a, b) and torch.equal(a, c)


def test_calls_keep_no_memory(q):
    calls = [c for c, _ in _host_calls(q, np.random.default_rng(14))]
    for c in calls:
        c()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(50):
        for c in calls:
            c()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before


def test_unusual_calls_are_left_to_the_long_way(q):
    h = q.w8._host
    f = lambda *s, **k: torch.zeros(s, device=DEV, **k)
    i8 = torch.int8
    for r in (h.quant8(f(4, 8).half(), None, None), h.quant8(f(4, 8).t(), None, None), h.quant8(f(8), None, None),
              h.quant8(f(0, 8), None, None), h.quant8(f(4, 8).cpu(), None, None), h.quant8(f(4, 8), f(7), None),
              h.quant8(f(4, 8), None, f(4, 7)), h.quant8(f(4, 8), None, f(4, 8).bfloat16()), h.quant8(3, None, None),
              h.quant8(f(4, 8)), h.quant8(f(2, 40000), None, None),
              h.dequant8(f(4, 8), f(4), None, True), h.dequant8(f(4, 24, dtype=i8)[:, :8], f(4), None, True),
              h.dequant8(f(4, 16, dtype=i8), f(3), None, True), h.dequant8(f(4, 16, dtype=i8), f(4).double(), None, True),
              h.rmsnorm8(f(4, 8), f(8), -1.0, None), h.rmsnorm8(f(4, 8), f(8), "a", None),
              h.rmsnorm8(f(4, 8), None, 1e-5, f(3, 8)), h.rmsnorm8(f(4, 8), None, 1e-5, f(4, 8).cpu()),
              h.gemm8(f(4, 16, dtype=i8), f(4), f(5, 32, dtype=i8), f(5), True),
              h.gemm8(f(4, 16, dtype=i8), f(4), f(5, 16, dtype=i8), f(4), True),
              h.gemm8(f(4, 16, dtype=i8), f(4), f(5, 16, dtype=i8), f(10)[::2], True)):
        assert r is None
    with pytest.raises(q.QamwError):
        q.quant8(f(2, 40000))
    with pytest.raises(q.QamwError):
        q.rmsnorm8(f(4, 8), eps=-1.0)
    with pytest.raises(ValueError, match="on cpu"):
        q.rmsnorm8(f(4, 8), residual=f(4, 8).cpu())


def test_two_streams(q):
    """Calls on two streams at once, each with its own buffers, give what they give alone."""
    cases = [_mlp_case(q, T, 512, 1000, seed=T) for T in (40, 200)]
    alone = [_mlp(q, *c)[0].clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        for st, c in zip(streams, cases):
            with torch.cuda.stream(st):
                got.append(_mlp(q, *c)[0])
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, alone[i % 2]), i


def test_channel_scale_path(q):
    """Weights with the activation-aware scale, activations with its inverse folded into the norm: the
    layer's output stays that of the unscaled layer up to the 8-bit rounding, and a weight matrix reads
    back within half a step of each row, divided by its channel's scale."""
    rng = np.random.default_rng(8)
    T, d, n = 64, 1024, 256
    x = torch.from_numpy(_values(rng, T, d)).to(DEV)
    w = torch.from_numpy((0.02 * rng.standard_normal((n, d))).astype(np.float32)).to(DEV)
    s = q.act_scale(x, 0.3)
    wq = q.quant8(w, scale=s)
    back = q.dequant8(*wq, scale=s, out_dtype=torch.float32)
    # half a step, and the roundings of the product, the scale and the read-back: a few 2^-24 of 127 steps
    assert bool(((back - w).abs() <= wq[1][:, None] / s * (0.5 + 2.0 ** -14)).all())
    norm = 1 + 0.1 * torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(DEV)
    c, xs, _ = q.rmsnorm8(x, norm / s)
    y = q.gemm8(c, xs, *wq, out_dtype=torch.float32)
    xd = x.double()
    ref_y = (xd / torch.sqrt((xd ** 2).mean(1, keepdim=True) + 1e-5) * norm.double()) @ w.double().t().contiguous()
    assert float((y.double() - ref_y).norm() / ref_y.norm()) < 0.05
