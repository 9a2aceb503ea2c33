"""The 8-bit linear layers without a GPU: the library exports what include/qamw_w8.h declares, the
header is plain C, and every bad argument is refused by host code before any HIP call, in the C ABI and
in the binding.  The plain forms that the GPU tests compare with are pinned here to closed forms."""
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import w8_reference as ref
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
    names = q.header_symbols(q.W8_HEADER_PATH)
    assert set(names) == set(q.w8.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", q.LIB_PATH], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert not [n for n in names if n not in exported]


def test_header_is_plain_c():
    text = re.sub(r"/\*.*?\*/", "", open(q.W8_HEADER_PATH).read(), flags=re.S)
    for bad in ("hip_runtime", "torch", "hipStream_t", "namespace", "template"):
        assert bad not in text
    r = subprocess.run(["gcc", "-std=c99", "-fsyntax-only", "-x", "c", q.W8_HEADER_PATH], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_stride(lib):
    for d in (-3, 0, 1, 15, 16, 17, 1003, 5120, 2**31 - 1):
        want = (d + 15) // 16 * 16 if d > 0 else 0
        assert lib.qamw_q8_stride(d) == want and q.q8_stride(d) == want


def test_header_limits_match_binding():
    text = open(q.W8_HEADER_PATH).read()
    for name in ("W8_MAX_COLS", "GEMM8_MAX_ROWS", "GEMM8_MAX_COLS", "GEMM8_MAX_LD", "GEMM8_MAX_OUT"):
        m = re.search(r"#define QAMW_%s (.*)" % name, text)
        assert m and eval(m.group(1).replace("ll", "")) == getattr(q.w8, name), name


def _quant(lib, **kw):
    a = dict(x=FAKE, dt=q.BF16, rows=4, d=64, ld=64, gate=None, ld_g=0, scale=None, out=FAKE, ld_q=64, s=FAKE, st=None)
    a.update(kw)
    return lib.qamw_quant8(a["x"], a["dt"], a["rows"], a["d"], a["ld"], a["gate"], a["ld_g"], a["scale"], a["out"],
                           a["ld_q"], a["s"], a["st"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 30), UNSUP),
    (dict(d=32769, ld=32769, ld_q=32784), UNSUP), (dict(ld=63), ARG), (dict(gate=FAKE, ld_g=63), ARG),
    (dict(x=None), ARG), (dict(s=None), ARG), (dict(out=None), ARG), (dict(out=FAKE + 8), ARG), (dict(ld_q=72), ARG),
    (dict(ld_q=48), ARG), (dict(x=FAKE + 1), ARG), (dict(dt=q.F32, x=FAKE + 2), ARG),
    (dict(gate=FAKE + 1, ld_g=64), ARG), (dict(scale=FAKE + 2), ARG), (dict(s=FAKE + 2), ARG), (dict(st=FAKE + 1), ARG),
])
def test_quant8_rejects(lib, kw, code):
    assert _quant(lib, **kw) == code


def _dequant(lib, **kw):
    a = dict(codes=FAKE, rows=4, d=64, ld_q=64, s=FAKE, scale=None, out=FAKE, dt=q.BF16, ld=64)
    a.update(kw)
    return lib.qamw_dequant8(a["codes"], a["rows"], a["d"], a["ld_q"], a["s"], a["scale"], a["out"], a["dt"], a["ld"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 30), UNSUP),
    (dict(d=1 << 30, ld_q=1 << 30, ld=1 << 30), UNSUP), (dict(ld=63), ARG), (dict(codes=None), ARG), (dict(codes=FAKE + 4), ARG), (dict(ld_q=65), ARG), (dict(ld_q=48), ARG), (dict(s=None), ARG),
    (dict(out=None), ARG), (dict(out=FAKE + 1), ARG), (dict(dt=q.F32, out=FAKE + 2), ARG), (dict(scale=FAKE + 1), ARG),
])
def test_dequant8_rejects(lib, kw, code):
    assert _dequant(lib, **kw) == code


def _norm(lib, **kw):
    a = dict(x=FAKE, dt=q.BF16, rows=4, d=64, ld=64, res=None, ld_r=0, w=None, eps=1e-5, sum=None, ld_s=0, out=FAKE,
             ld_q=64, s=FAKE, st=None)
    a.update(kw)
    return lib.qamw_rmsnorm8(a["x"], a["dt"], a["rows"], a["d"], a["ld"], a["res"], a["ld_r"], a["w"], a["eps"], a["sum"],
                             a["ld_s"], a["out"], a["ld_q"], a["s"], a["st"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(rows=1 << 30), UNSUP),
    (dict(d=32769, ld=32769, ld_q=32784), UNSUP), (dict(ld=63), ARG), (dict(res=FAKE, ld_r=63), ARG),
    (dict(sum=FAKE * 2, ld_s=63), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.inf), ARG), (dict(eps=math.nan), ARG),
    (dict(x=None), ARG), (dict(s=None), ARG), (dict(out=None), ARG), (dict(out=FAKE + 8), ARG), (dict(ld_q=72), ARG),
    (dict(x=FAKE + 1), ARG), (dict(res=FAKE + 1, ld_r=64), ARG), (dict(sum=FAKE + 1, ld_s=64), ARG),
    (dict(w=FAKE + 2), ARG), (dict(s=FAKE + 2), ARG), (dict(st=FAKE + 2), ARG),
    (dict(sum=FAKE, ld_s=128), ARG),                                # over x, with another pitch
    (dict(res=FAKE * 2, ld_r=64, sum=FAKE * 2, ld_s=128), ARG),     # over the residual, with another pitch
])
def test_rmsnorm8_rejects(lib, kw, code):
    assert _norm(lib, **kw) == code


def _gemm(lib, **kw):
    a = dict(x=FAKE, ld_x=64, xs=FAKE, M=4, w=FAKE, ld_w=64, wsc=FAKE, N=32, K=64, y=FAKE, dt=q.BF16, ld_y=32, ws=None,
             wsb=0)
    a.update(kw)
    return lib.qamw_gemm8(a["x"], a["ld_x"], a["xs"], a["M"], a["w"], a["ld_w"], a["wsc"], a["N"], a["K"], a["y"], a["dt"],
                          a["ld_y"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), ARG), (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=0), ARG), (dict(ld_y=31), ARG),
    (dict(M=(1 << 24) + 1), UNSUP), (dict(N=(1 << 24) + 1, ld_y=1 << 25), UNSUP),
    (dict(K=131072, ld_x=131072, ld_w=131072), UNSUP), (dict(ld_x=(1 << 22) + 16), UNSUP),
    (dict(ld_w=(1 << 22) + 16), UNSUP), (dict(x=None), ARG), (dict(w=None), ARG), (dict(xs=None), ARG),
    (dict(wsc=None), ARG), (dict(y=None), ARG), (dict(x=FAKE + 8), ARG), (dict(w=FAKE + 8), ARG), (dict(ld_x=72), ARG),
    (dict(ld_w=72), ARG), (dict(ld_x=48), ARG), (dict(xs=FAKE + 2), ARG), (dict(wsc=FAKE + 1), ARG), (dict(y=FAKE + 1), ARG),
    (dict(dt=q.F32, y=FAKE + 2), ARG),
])
def test_gemm8_rejects(lib, kw, code):
    assert _gemm(lib, **kw) == code


def test_gemm8_workspace(lib):
    """Workspace sizes are bounded, 0 for sizes that are refused, and a short one is refused."""
    for bad in ((-1, 4, 4), (4, -1, 4), (4, 4, 0), (4, 4, 131072), ((1 << 24) + 1, 4, 4), (1 << 20, 1 << 19, 64)):
        assert lib.qamw_gemm8_workspace(*bad) == 0
    for M in (1, 16, 17, 33, 64, 77, 128, 200, 256, 300, 512, 1500, 8192):
        for N, K in ((64, 13824), (4096, 11008), (5120, 5120), (13824, 5120)):
            need = lib.qamw_gemm8_workspace(M, N, K)
            assert need <= 256 << 20
            if need:
                ld = (K + 15) // 16 * 16
                base = dict(M=M, N=N, K=K, ld_x=ld, ld_w=ld, ld_y=N)
                assert _gemm(lib, **base) == WS
                assert _gemm(lib, ws=FAKE, wsb=need - 1, **base) == WS
                assert _gemm(lib, ws=FAKE + 64, wsb=need, **base) == WS


def test_empty_calls_are_noops(lib):
    assert _quant(lib, rows=0, x=None, out=None, s=None) == q.OK
    assert _dequant(lib, rows=0, codes=None, s=None, out=None) == q.OK
    assert _norm(lib, rows=0, x=None, out=None, s=None) == q.OK
    assert _gemm(lib, M=0, x=None, y=None) == q.OK
    assert _gemm(lib, N=0, w=None, y=None, ld_y=0) == q.OK


# ------------------------------------------------------------------ the binding, with host tensors

def _bad(fn, match, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_rejects_rows(lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for fn in (q.quant8, q.rmsnorm8):
        _bad(fn, "x", x[0])
        _bad(fn, "x", x.half())
        _bad(fn, "contiguous", torch.zeros((64, 4)).t())
        _bad(fn, "overlap", torch.zeros((64,)).as_strided((4, 16), (8, 1)))
        _bad(fn, "out", x, out=torch.zeros((4, 64), dtype=torch.uint8))
        _bad(fn, "out", x, out=torch.zeros((4, 80), dtype=torch.int8))
        _bad(fn, "16-byte", x, out=torch.zeros((4, 72), dtype=torch.int8)[:, :64])
        _bad(fn, "row_scale", x, row_scale=torch.zeros(3))
        _bad(fn, "row_scale", x, row_scale=torch.zeros(4, dtype=torch.float64))
        _bad(fn, "status", x, status=torch.zeros(1))
        _bad(fn, "device", x)   # everything fits: the device check
    _bad(q.quant8, "gate", x, gate=x[:3])
    _bad(q.quant8, "gate", x, gate=x.float())
    _bad(q.quant8, "scale", x, scale=torch.ones(63))
    _bad(q.quant8, "scale", x, scale=torch.ones(128)[::2])
    _bad(q.rmsnorm8, "residual", x, residual=x[:, :32])
    _bad(q.rmsnorm8, "sum_out", x, sum_out=x.float())
    _bad(q.rmsnorm8, "weight", x, torch.ones(64, dtype=torch.bfloat16))


def test_binding_rejects_codes(lib):
    c = torch.zeros((4, 64), dtype=torch.int8)
    s = torch.ones(4)
    _bad(q.dequant8, "codes", c.to(torch.uint8), s)
    _bad(q.dequant8, "row_scale", c, s[:3])
    _bad(q.dequant8, "out", c, s, out=torch.zeros((4, 63)))
    _bad(q.dequant8, "out_dtype", c, s, out_dtype=torch.float16)
    _bad(q.dequant8, "16-byte", torch.zeros((4, 60), dtype=torch.int8), s)
    # 4 x 60 codes with a pitch of 64 whose storage ends with the last code
    short = torch.zeros((3 * 64 + 60,), dtype=torch.int8).as_strided((4, 60), (64, 1))
    _bad(q.dequant8, "16-byte chunk", short, s)
    _bad(q.dequant8, "device", c, s)
    w, ws = torch.zeros((8, 64), dtype=torch.int8), torch.ones(8)
    _bad(q.gemm8, "columns", c, s, w[:, :48], ws)
    _bad(q.gemm8, "x_scale", c, s[:2], w, ws)
    _bad(q.gemm8, "w_scale", c, s, w, ws[:7])
    _bad(q.gemm8, "wq", c, s, w.float(), ws)
    _bad(q.gemm8, "out", c, s, w, ws, out=torch.zeros((4, 9)))
    _bad(q.gemm8, "out_dtype", c, s, w, ws, out_dtype=torch.int32)
    _bad(q.gemm8, "workspace", c, s, w, ws, workspace=torch.zeros(4))
    _bad(q.gemm8, "contiguous", c, s, torch.zeros((64, 8), dtype=torch.int8).t(), ws)
    _bad(q.gemm8, "device", c, s, w, ws)


# ------------------------------------------------------------------ the plain forms

def test_reference_rounding_to_bf16():
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.float32(1e3)
    assert np.array_equal(ref.to_bf16(x), torch.from_numpy(x).to(torch.bfloat16).float().numpy())


def test_reference_quantizer():
    # powers of two: 127 / top is exact up to its own rounding, ties go to even
    a = np.array([[127, 63.5, 0.5, 1.5, -2.5, 0], [0, 0, 0, 0, 0, 0], [1, np.nan, 0, 0, 0, 0], [1, 2, -np.inf, 0, 0, 0],
                  [1e-37, 0, 0, 0, 0, 0]], dtype=np.float32)
    qv, s = ref.quant8(a)
    assert qv[0].tolist() == [127, 64, 0, 2, -2, 0] and s[0] == 1.0
    assert not qv[1:].any() and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == 0
    # a code is off by at most half a step, and by what the roundings of 127 / top and of the product add:
    # two relative errors of 2^-24 on a value of at most 127, less than 2^-16; the row scale adds one more
    a = np.random.default_rng(1).standard_normal((50, 300)).astype(np.float32)
    qv, s = ref.quant8(a)
    s64 = np.abs(a.astype(np.float64)).max(1) / 127
    assert np.all(np.abs(qv * s64[:, None] - a) <= s64[:, None] * (0.5 + 2.0 ** -16))
    assert np.all(np.abs(s - s64) <= s64 * 2.0 ** -24)


def test_reference_norm_and_product():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((5, 40)).astype(np.float32), rng.standard_normal(40).astype(np.float32)
    qv, s, h = ref.rmsnorm8(x, w, 1e-3, 2 * x)
    y = (3.0 * x) * w / np.sqrt((9.0 * x.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-3)
    assert np.all(np.abs(qv * s[:, None] - y) <= s[:, None] * 0.51)
    a, b = rng.integers(-128, 128, (3, 70)), rng.integers(-128, 128, (4, 70))
    assert np.array_equal(ref.sums(a, b), a @ b.T)
