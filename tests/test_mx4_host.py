"""The 4-bit linear layers without a GPU: the library exports what include/qamw_mx4.h declares, the header is plain C,
and every bad argument is refused by host code before any HIP call, in the C ABI and in the binding.  The plain forms
that the GPU tests compare with are pinned here to closed forms."""
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mx4_reference as ref
import weight_quantization_codec_amd as q

ARG, UNSUP, WS = q.ERR_ARG, q.ERR_UNSUPPORTED, q.ERR_WORKSPACE
FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(q.LIB_PATH):
        from weight_quantization_codec_amd import _build
        _build.build()
    return q.load()


def test_exports_every_declared_symbol(lib):
    names = q.header_symbols(q.MX4_HEADER_PATH)
    assert set(names) == set(q.mx4.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", q.LIB_PATH], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert not [n for n in names if n not in exported]


def test_header_is_plain_c():
    text = re.sub(r"/\*.*?\*/", "", open(q.MX4_HEADER_PATH).read(), flags=re.S)
    for bad in ("hip_runtime", "torch", "hipStream_t", "namespace", "template"):
        assert bad not in text
    r = subprocess.run(["gcc", "-std=c99", "-fsyntax-only", "-x", "c", q.MX4_HEADER_PATH], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_stride_and_groups(lib):
    for d in (-3, 0, 1, 255, 256, 257, 1003, 5120, 2**31 - 1):
        want = (d + 255) // 256 if d > 0 else 0
        assert lib.qamw_mx4_groups(d) == want and q.mx4_groups(d) == want
        assert lib.qamw_mx4_stride(d) == 128 * want and q.mx4_stride(d) == 128 * want


def test_header_limits_match_binding():
    text = open(q.MX4_HEADER_PATH).read()
    for name in ("MX4_MAX_NORM_COLS", "MX4_MAX_COLS", "GEMM4_MAX_ROWS", "GEMM4_MAX_LD", "GEMM4_MAX_OUT",
                 "GEMM4_MAX_EXPERTS", "GEMM4_MAX_EXPERT_ROWS", "GEMM4_MAX_INDEXED"):
        m = re.search(r"#define QAMW_%s (.*)" % name, text)
        assert m and eval(m.group(1).replace("ll", "")) == getattr(q.mx4, name), name


def _quant(lib, **kw):
    a = dict(x=FAKE, dt=q.BF16, rows=4, d=64, ld=64, gate=None, ld_g=0, scale=None, out=FAKE, ld_q=128, e=FAKE, ld_e=32,
             st=None)
    a.update(kw)
    return lib.qamw_quant4(a["x"], a["dt"], a["rows"], a["d"], a["ld"], a["gate"], a["ld_g"], a["scale"], a["out"],
                           a["ld_q"], a["e"], a["ld_e"], a["st"], None)


# what the codes and scales of any row operator may not be, for 4 rows of 64 columns
BAD_CODES = [dict(out=None), dict(out=FAKE + 8), dict(ld_q=112), dict(ld_q=136), dict(e=None), dict(e=FAKE + 4),
             dict(ld_e=24), dict(ld_e=36)]
BIG = dict(d=(1 << 23) + 1, ld=1 << 24, ld_q=1 << 23)


@pytest.mark.parametrize("kw,code", [(k, ARG) for k in BAD_CODES] + [
    (dict(dt=7), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 30), UNSUP), (BIG, UNSUP), (dict(ld=63), ARG),
    (dict(gate=FAKE, ld_g=63), ARG), (dict(x=None), ARG), (dict(x=FAKE + 1), ARG), (dict(dt=q.F32, x=FAKE + 2), ARG),
    (dict(gate=FAKE + 1, ld_g=64), ARG), (dict(scale=FAKE + 2), ARG), (dict(st=FAKE + 1), ARG),
    (dict(d=257, ld=257), ARG),   # two groups, codes for one
])
def test_quant4_rejects(lib, kw, code):
    assert _quant(lib, **kw) == code


def _dequant(lib, **kw):
    a = dict(out=FAKE, rows=4, d=64, ld_q=128, e=FAKE, ld_e=32, scale=None, y=FAKE, dt=q.BF16, ld=64)
    a.update(kw)
    return lib.qamw_dequant4(a["out"], a["rows"], a["d"], a["ld_q"], a["e"], a["ld_e"], a["scale"], a["y"], a["dt"],
                             a["ld"], None)


@pytest.mark.parametrize("kw,code", [(k, ARG) for k in BAD_CODES] + [
    (dict(dt=2), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 30), UNSUP), (BIG, UNSUP), (dict(ld=63), ARG),
    (dict(y=None), ARG), (dict(y=FAKE + 1), ARG), (dict(dt=q.F32, y=FAKE + 2), ARG), (dict(scale=FAKE + 1), ARG),
])
def test_dequant4_rejects(lib, kw, code):
    assert _dequant(lib, **kw) == code


def _norm(lib, **kw):
    a = dict(x=FAKE, dt=q.BF16, rows=4, d=64, ld=64, res=None, ld_r=0, w=None, eps=1e-5, sum=None, ld_s=0, out=FAKE,
             ld_q=128, e=FAKE, ld_e=32, st=None)
    a.update(kw)
    return lib.qamw_rmsnorm4(a["x"], a["dt"], a["rows"], a["d"], a["ld"], a["res"], a["ld_r"], a["w"], a["eps"], a["sum"],
                             a["ld_s"], a["out"], a["ld_q"], a["e"], a["ld_e"], a["st"], None)


@pytest.mark.parametrize("kw,code", [(k, ARG) for k in BAD_CODES] + [
    (dict(dt=7), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 30), UNSUP),
    (dict(d=32769, ld=32769, ld_q=16512), UNSUP), (dict(ld=63), ARG), (dict(res=FAKE, ld_r=63), ARG),
    (dict(sum=FAKE * 2, ld_s=63), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.inf), ARG), (dict(eps=math.nan), ARG),
    (dict(x=None), ARG), (dict(x=FAKE + 1), ARG), (dict(res=FAKE + 1, ld_r=64), ARG), (dict(sum=FAKE + 1, ld_s=64), ARG),
    (dict(w=FAKE + 2), ARG), (dict(st=FAKE + 2), ARG),
    (dict(sum=FAKE, ld_s=128), ARG),                                # over x, with another pitch
    (dict(res=FAKE * 2, ld_r=64, sum=FAKE * 2, ld_s=128), ARG),     # over the residual, with another pitch
])
def test_rmsnorm4_rejects(lib, kw, code):
    assert _norm(lib, **kw) == code


def _gemm(lib, **kw):
    a = dict(x=FAKE, ld_x=256, xe=FAKE, ld_xe=32, M=4, w=FAKE, ld_w=256, we=FAKE, ld_we=256, N=32, g=2, y=FAKE, dt=q.BF16,
             ld_y=32, ws=None, wsb=0)
    a.update(kw)
    return lib.qamw_gemm4(a["x"], a["ld_x"], a["xe"], a["ld_xe"], a["M"], a["w"], a["ld_w"], a["we"], a["ld_we"], a["N"],
                          a["g"], a["y"], a["dt"], a["ld_y"], a["ws"], a["wsb"], None)


# what the operands of either product may not be
BAD_PRODUCT = [
    (dict(dt=7), ARG), (dict(N=-1), ARG), (dict(g=0), ARG), (dict(ld_y=31), ARG),
    (dict(N=(1 << 24) + 1, ld_y=1 << 25), UNSUP), (dict(g=(1 << 15) + 1), UNSUP),
    (dict(ld_x=(1 << 22) + 16), UNSUP), (dict(ld_w=(1 << 22) + 16), UNSUP),
    (dict(x=None), ARG), (dict(x=FAKE + 8), ARG), (dict(ld_x=240), ARG), (dict(ld_x=264), ARG),
    (dict(xe=None), ARG), (dict(xe=FAKE + 4), ARG), (dict(ld_xe=24), ARG), (dict(ld_xe=36), ARG),
    (dict(w=None), ARG), (dict(w=FAKE + 8), ARG), (dict(ld_w=240), ARG), (dict(ld_w=264), ARG),
    (dict(we=None), ARG), (dict(we=FAKE + 4), ARG), (dict(ld_we=248), ARG), (dict(ld_we=260), ARG),
    (dict(y=None), ARG), (dict(y=FAKE + 1), ARG), (dict(dt=q.F32, y=FAKE + 2), ARG),
]


@pytest.mark.parametrize("kw,code", BAD_PRODUCT + [
    (dict(M=-1), ARG), (dict(M=(1 << 24) + 1, ld_xe=1 << 28), UNSUP),
    (dict(M=1 << 20, N=1 << 19, ld_y=1 << 19, ld_xe=1 << 23, ld_we=1 << 22), UNSUP),
])
def test_gemm4_rejects(lib, kw, code):
    assert _gemm(lib, **kw) == code


def test_gemm4_noops_and_workspace(lib):
    assert _gemm(lib, M=0, x=None, xe=None, y=None) == q.OK
    assert _gemm(lib, N=0, ld_y=0, w=None, we=None) == q.OK
    for size in ((-1, 4, 1), (4, -1, 1), (4, 4, 0), ((1 << 24) + 1, 4, 1), (4, 4, (1 << 15) + 1), (0, 4, 1), (4, 0, 1)):
        assert lib.qamw_gemm4_workspace(*size) == 0
    assert q.gemm4_workspace(2**32 + 77, 4096, 43) == 0


def _grouped(lib, **kw):
    a = dict(x=FAKE, ld_x=256, xe=FAKE, ld_xe=32, x_rows=4, index=None, rows=4, w=FAKE, ld_w=256, by=256 * 32, we=FAKE,
             ld_we=256, eby=256, off=FAKE, E=3, N=32, g=2, y=FAKE, dt=q.BF16, ld_y=32)
    a.update(kw)
    return lib.qamw_gemm4_grouped(a["x"], a["ld_x"], a["xe"], a["ld_xe"], a["x_rows"], a["index"], a["rows"], a["w"],
                                  a["ld_w"], a["by"], a["we"], a["ld_we"], a["eby"], a["off"], a["E"], a["N"], a["g"],
                                  a["y"], a["dt"], a["ld_y"], None)


@pytest.mark.parametrize("kw,code", BAD_PRODUCT + [
    (dict(rows=-1), ARG), (dict(x_rows=-1), ARG), (dict(rows=5), ARG), (dict(E=0), ARG), (dict(E=1025), UNSUP),
    (dict(rows=(1 << 24) + 1, index=FAKE), UNSUP), (dict(x_rows=(1 << 24) + 1, ld_xe=1 << 28), UNSUP),
    (dict(by=-16), ARG), (dict(by=8), ARG), (dict(eby=-8), ARG), (dict(eby=4), ARG), (dict(off=None), ARG),
    (dict(off=FAKE + 2), ARG), (dict(index=FAKE + 2), ARG),
    (dict(E=1024, N=(1 << 20) + 1, ld_y=1 << 21, ld_we=1 << 24), UNSUP),   # 2^30 rows of weights and more
    (dict(index=FAKE, x_rows=1 << 24, ld_xe=1 << 27), UNSUP),   # 2^32 bytes of codes to choose rows from
])
def test_gemm4_grouped_rejects(lib, kw, code):
    assert _grouped(lib, **kw) == code


def test_gemm4_grouped_noops(lib):
    assert _grouped(lib, rows=0, x=None, xe=None, y=None, off=None) == q.OK
    assert _grouped(lib, N=0, ld_y=0, w=None, we=None) == q.OK


def test_row_operators_noops(lib):
    assert _quant(lib, rows=0, x=None, out=None, e=None) == q.OK
    assert _dequant(lib, rows=0, out=None, e=None, y=None) == q.OK
    assert _norm(lib, rows=0, x=None, out=None, e=None) == q.OK


# ---------------------------------------------------------------- the binding

def _mat(n, d, dtype=torch.bfloat16):
    return torch.zeros((n, d), dtype=dtype)


def _form(n, d):
    return torch.zeros((n, q.mx4_stride(d)), dtype=torch.uint8), torch.zeros((q.mx4_groups(d), n, 8), dtype=torch.uint8)


def test_binding_refuses_rows():
    x = _mat(4, 300)
    c, s = _form(4, 300)
    for bad in (x[0], x.half(), x.t(), x.to(torch.int8), None, _mat(4, 300).expand(4, 300)[:, ::2]):
        with pytest.raises(ValueError, match="^x "):
            q.quant4(bad)
        with pytest.raises(ValueError, match="^x "):
            q.rmsnorm4(bad)
    for kw, name in ((dict(gate=_mat(4, 299)), "gate"), (dict(gate=x.float()), "gate"), (dict(scale=torch.ones(299)), "scale"),
                     (dict(scale=torch.ones(300).double()), "scale"), (dict(status=torch.zeros(1)), "status"),
                     (dict(out=c), "together"), (dict(scales=s), "together"), (dict(out=c[:3], scales=s), "out"),
                     (dict(out=c[:, :128], scales=s), "out"), (dict(out=c.char(), scales=s), "out"),
                     (dict(out=c, scales=s[:1]), "scales"), (dict(out=c, scales=s[:, :3]), "scales"),
                     (dict(out=c, scales=s.transpose(0, 1).contiguous()), "scales"),
                     (dict(out=c, scales=s.transpose(0, 1).contiguous().transpose(0, 1)), "scales"),
                     (dict(out=torch.zeros((4, 264), dtype=torch.uint8)[:, 8:], scales=s), "out")):
        with pytest.raises(ValueError, match=name):
            q.quant4(x, **kw)
    for kw, name in ((dict(residual=_mat(3, 300)), "residual"), (dict(sum_out=x.float()), "sum_out"),
                     (dict(weight=torch.ones(299)), "weight"), (dict(out=c), "together")):
        with pytest.raises(ValueError, match=name):
            q.rmsnorm4(x, **kw)
    for call in (lambda: q.quant4(x), lambda: q.rmsnorm4(x), lambda: q.dequant4(c, s, 300)):
        with pytest.raises(ValueError, match="device"):
            call()
    for a, name in (((c[:, :256], s, 256), "codes"), ((c, s, 0), "d must"), ((c, s[:, :3], 300), "scales"),
                    ((c, s, 513), "codes"), ((c.t(), s, 300), "codes")):
        with pytest.raises(ValueError, match=name):
            q.dequant4(*a)
    with pytest.raises(ValueError, match="out_dtype"):
        q.dequant4(c, s, 300, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out must"):
        q.dequant4(c, s, 300, out=_mat(4, 299))


def test_binding_refuses_products():
    (xq, xs), (wq, ws) = _form(4, 300), _form(6, 300)
    other, oscales = _form(6, 600)
    for a, name in (((xq, xs, other, oscales), "groups"), ((xq, xs[:, :3], wq, ws), "x_scales"), ((xq, xs, wq, ws[:1]), "w_scales"),
                    ((xq[:, :192], xs, wq, ws), "xq"), ((xq, xs, wq.char(), ws), "wq"), ((xq, xs, wq, ws.int()), "w_scales")):
        with pytest.raises(ValueError, match=name):
            q.gemm4(*a)
    with pytest.raises(ValueError, match="out must"):
        q.gemm4(xq, xs, wq, ws, out=_mat(4, 7))
    with pytest.raises(ValueError, match="out_dtype"):
        q.gemm4(xq, xs, wq, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="device"):
        q.gemm4(xq, xs, wq, ws)
    wq, ws = wq.view(3, 2, -1), ws.view(-1, 3, 2, 8)
    off = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
    idx = torch.zeros(9, dtype=torch.int32)
    for a, kw, name in (((xq, xs, wq[0], ws, off), {}, "wq"), ((xq, xs, wq, ws[:, 0], off), {}, "w_scales"),
                        ((xq, xs, wq, ws[:, :2], off), {}, "w_scales"), ((xq, xs, wq, ws, off[:3]), {}, "offsets"),
                        ((xq, xs, wq, ws, off.long()), {}, "offsets"), ((xq, xs, wq, ws, off), dict(index=idx.long()), "index"),
                        ((xq, xs, wq, ws, off), dict(index=idx[::2]), "index"),
                        ((xq, xs, wq, ws, off), dict(out=_mat(5, 2)), "out must"),
                        ((xq, xs, wq, ws, off), dict(index=idx, out=_mat(4, 2)), "out must"),
                        ((xq, xs, wq[:0], ws[:, :0], off), {}, "experts"), ((xq, xs, other.view(3, 2, -1), ws, off), {}, "groups"),
                        ((xq, xs, wq.transpose(0, 1).contiguous().transpose(0, 1)[:, :, 8:], ws, off), {}, "wq"),
                        ((xq, xs, wq, ws, off), {}, "device")):
        with pytest.raises(ValueError, match=name):
            q.gemm4_grouped(*a, **kw)


def test_the_residual_stream_keeps_its_history():
    """h of rmsnorm4 would carry a residual stream on, without its history."""
    x, r = torch.zeros((4, 64)), torch.zeros((4, 64))
    with pytest.raises(ValueError, match="device"):
        q.rmsnorm4(x.clone().requires_grad_())   # h is x, with its history
    for kw in (dict(x=x, residual=r.clone().requires_grad_()), dict(x=x.clone().requires_grad_(), residual=r),
               dict(x=x.clone().requires_grad_(), sum_out=r)):
        with pytest.raises(ValueError, match="gradient"):
            q.rmsnorm4(**kw)
        with torch.no_grad(), pytest.raises(ValueError, match="device"):
            q.rmsnorm4(**kw)


# ---------------------------------------------------------------- the plain forms

def test_reference_codes_are_the_nearest_values():
    """Every fp32 value next to a border of two codes, and the borders themselves, in a block whose largest value is 6."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], dtype=np.float32)
    below, above = np.nextafter(borders, np.float32(0)), np.nextafter(borders, np.float32(9))
    ties = [0, 2, 2, 4, 4, 6, 6]
    for v, want in ((borders, ties), (below, range(7)), (above, range(1, 8))):
        for sign in (1, -1):
            a = np.zeros((1, 32), dtype=np.float32)
            a[0, :7], a[0, 7] = sign * v, 6
            c, s = ref.quantize(a)
            got = np.stack([c & 15, c >> 4], 2).reshape(-1)[:8]
            assert list(got) == [w + 8 * (sign < 0) for w in want] + [7] and s[0, 0, 0] == 127


def test_reference_scales():
    """top in (3.5 2^E, 7 2^E]: exponent E."""
    past7 = np.nextafter(np.float32(7), np.float32(8))
    for E in (-100, -3, 0, 5, 120):
        for top, exponent, value in ((7.0, E, 6), (past7, E + 1, 8), (3.5, E - 1, 3), (4.0, E, 4), (6.0, E, 6)):
            a = np.zeros((1, 40), dtype=np.float32)
            a[0, 3] = -np.float32(top) * np.float32(2.0 ** E)
            c, s = ref.quantize(a)
            assert s[0, 0, 0] == exponent + 127 and s[0, 0, 1:].max() == 0
            assert ref.read(c, s, 40)[0, 3] == -value * 2.0 ** E
    a = np.zeros((4, 64), dtype=np.float32)
    a[0, 5], a[1, 40], a[2, 0], a[3, 0] = np.nan, np.inf, 2.0 ** -119, np.nextafter(np.float32(2.0 ** -119), np.float32(0))
    c, s = ref.quantize(a)
    assert list(s[0, :, 0]) == [255, 0, 127 - 121, 0] and s[0, 1, 1] == 255
    v = ref.read(c, s, 64)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all() and v[2, 0] == 2.0 ** -119 and not c[3].any()


def test_reference_error():
    """A value's error is at most half a step of its binade: |a| / 6 from 1 on, a quarter of the power of two below,
    and one power of two for values up to 7."""
    rng = np.random.default_rng(3)
    a = (rng.standard_normal((50, 320)) * np.exp(3 * rng.standard_normal((50, 320)))).astype(np.float32)
    c, s = ref.quantize(a)
    unit = np.repeat(2.0 ** (s.transpose(1, 0, 2).reshape(50, -1) - 127.0), 32, 1)[:, :320]
    v = np.abs(a) / unit
    err = np.abs(ref.read(c, s, 320) - a) / unit
    assert v.max() <= 7 and (err <= np.where(v < 2, 0.25, np.where(v < 4, 0.5, 1.0))).all()


def test_reference_products():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((3, 300)).astype(np.float32), rng.standard_normal((5, 300)).astype(np.float32)
    xv, wv = ref.read(*ref.quantize(x)), ref.read(*ref.quantize(w))
    y, mag = ref.product(xv, wv)
    want = [[math.fsum(a * b for a, b in zip(xr, wr)) for wr in wv] for xr in xv]
    assert np.allclose(y, want, rtol=1e-14) and (mag >= np.abs(y)).all()
    assert xv.shape == (3, 512) and not xv[:, 300:].any()
