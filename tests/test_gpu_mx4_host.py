"""The compiled short way of the 4-bit binding: the same answers as the long way, what it does with failures and with the
interpreter's lock, products that need a workspace, and calls of several threads and graphs at once."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from helpers import DEV
from test_gpu_mx4 import KERNELS, _form

pytestmark = pytest.mark.gpu

PARTS = (77, 4096, 11008)   # k in parts: a workspace


def _bind(q, fn):
    """The compiled module with `fn` in place of every function of the library that launches."""
    address = ctypes.cast(fn, ctypes.c_void_p).value
    size = ctypes.cast(q.load().qamw_gemm4_workspace, ctypes.c_void_p).value
    q.mx4._host.bind4(address, address, address, size, address, address)


def _tensors():
    x = torch.ones((4, 256), device=DEV)
    c = torch.zeros((4, 128), dtype=torch.uint8, device=DEV)
    s = torch.zeros((1, 4, 8), dtype=torch.uint8, device=DEV)
    return x, c, s, torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)


def _calls(q):
    x, c, s, off = _tensors()
    w, ws = c.view(2, 2, 128), s.view(1, 2, 2, 8)
    return [lambda: q.quant4(x), lambda: q.dequant4(c, s, 256), lambda: q.rmsnorm4(x, residual=x),
            lambda: q.gemm4(c, s, c, s), lambda: q.gemm4_grouped(c, s, w, ws, off)]


NAMES = ["quant4", "dequant4", "rmsnorm4", "gemm4", "gemm4_grouped"]


@pytest.mark.parametrize("which", range(5), ids=NAMES)
def test_a_failed_launch_is_an_error(q, which):
    """An error of the runtime, which may come behind a kernel that is already queued, is raised: the call is not
    queued a second time."""
    call, seen = _calls(q)[which], []
    fake = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: seen.append(1) or q.ERR_HIP)
    try:
        _bind(q, fake)
        with pytest.raises(q.QamwError) as e:
            call()
        assert e.value.code == q.ERR_HIP and len(seen) == 1
    finally:
        q.mx4.bind(q.load())
    call()


def test_other_threads_run_during_a_launch(q):
    """The library is called without the interpreter lock: in place of its functions stands the interpreter's own check
    for the lock, which gives 0 (no error) only where it is not held."""
    try:
        _bind(q, ctypes.pythonapi.PyGILState_Check)
        for call in _calls(q):
            call()
    finally:
        q.mx4.bind(q.load())


def test_both_ways_agree(q, monkeypatch):
    """Views, column offsets, rows of experts, indexes: what the short way takes it answers as the long way does, and what
    it does not take the long way answers."""
    rng = np.random.default_rng(3)
    both = torch.randn((40, 1300), device=DEV).to(torch.bfloat16)
    scale = torch.rand(600, device=DEV) + 0.5
    xq, xs, _ = _form(q, rng, 50, 600, extra=32)
    wq, ws, _ = _form(q, rng, 5 * 70, 600)
    w3, ws4 = wq.view(5, 70, -1), ws.reshape(3, 5, 70, 8)
    off = torch.tensor([0, 9, 9, 30, 44, 50], dtype=torch.int32, device=DEV)
    index = torch.randint(-1, 51, (50,), dtype=torch.int32, device=DEV)
    calls = [lambda: q.quant4(both[:, 3:603], scale=scale, gate=both[:, 700:]), lambda: q.quant4(both[5:6, :600]),
             lambda: q.quant4(both[::2, :600]), lambda: q.rmsnorm4(both[:, :600], scale, residual=both[:, 600:1200]),
             lambda: q.rmsnorm4(both[:1, :600], None, eps=0.1)[:2], lambda: q.dequant4(xq, xs, 600, scale=scale),
             lambda: q.dequant4(xq[7:9], xs[:, 7:9], np.int64(513), out_dtype=torch.float32),
             lambda: q.gemm4(xq[3:30], xs[:, 3:30], wq[:99], ws[:, :99]), lambda: q.gemm4(xq[4:5], xs[:, 4:5], wq, ws, out_dtype=torch.float32),
             lambda: q.gemm4_grouped(xq, xs, w3, ws4, off), lambda: q.gemm4_grouped(xq, xs, w3, ws4, off, index=index),
             lambda: q.gemm4_grouped(xq[:30], xs[:, :30], w3[1:3], ws4[:, 1:3], off[1:4], index=index[:30].clamp(0, 29))]
    short = [c() for c in calls]
    monkeypatch.setattr(q.mx4, "_host", None)
    for i, (a, c) in enumerate(zip(short, calls)):
        b = c()
        for u, v in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
            v = v[:9] if i == 11 else v      # (rows 0 to 8 of that call have no group; its groups begin at row 9)
            u = u[:9] if i == 11 else u
            assert u.shape == v.shape and (i == 11 or torch.equal(u, v)), i
    a, b = calls[11](), calls[11]()
    assert torch.equal(a[9:], b[9:])


def test_empty_matrices(q):
    x = torch.empty((0, 600), device=DEV)
    c, s = q.quant4(x)
    assert tuple(c.shape) == (0, 384) and tuple(s.shape) == (3, 0, 8)
    assert tuple(q.dequant4(c, s, 600).shape) == (0, 600)
    assert [tuple(t.shape) for t in q.rmsnorm4(x)] == [(0, 384), (3, 0, 8), (0, 600)]
    w, ws, _ = _form(q, np.random.default_rng(1), 10, 600)
    assert tuple(q.gemm4(c, s, w, ws).shape) == (0, 10) and tuple(q.gemm4(w, ws, c, s).shape) == (10, 0)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert tuple(q.gemm4_grouped(c, s, w.view(2, 5, -1), ws.reshape(3, 2, 5, 8), off).shape) == (0, 5)
    out = torch.full((10, 5), 7.0, device=DEV)
    q.gemm4_grouped(w, ws, w.view(2, 5, -1), ws.reshape(3, 2, 5, 8), off, out=out)   # no group has a row
    assert (out == 7).all()


def test_workspaces(q):
    """A workspace that is given, one that the call makes, one that is too short."""
    M, N, K = PARTS
    rng = np.random.default_rng(5)
    xq, xs, _ = _form(q, rng, M, K)
    wq, ws, _ = _form(q, rng, N, K)
    need = q.gemm4_workspace(M, N, q.mx4_groups(K))
    assert need > 0
    y = q.gemm4(xq, xs, wq, ws, out_dtype=torch.float32)
    work = torch.full((need,), 255, dtype=torch.uint8, device=DEV)   # nothing in it has to start at zero
    assert torch.equal(q.gemm4(xq, xs, wq, ws, out_dtype=torch.float32, workspace=work), y)
    with pytest.raises(ValueError, match="workspace"):
        q.gemm4(xq, xs, wq, ws, workspace=work[:-1])


def test_threads_with_a_stream_each(q):
    """Products of several kernels from several threads at once, a stream each."""
    sizes = [PARTS, (9, 4096, 4000), (515, 5120, 4096), (2049, 4100, 1200)]
    assert set(sizes) <= set(KERNELS)
    rng = np.random.default_rng(6)
    inputs = [(_form(q, rng, M, K)[:2], _form(q, rng, N, K)[:2]) for M, N, K in sizes]
    want = [q.gemm4(*x, *w) for x, w in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [q.gemm4(*inputs[k][0], *inputs[k][1]) for _ in range(20)]
        stream.synchronize()
        wrong.extend(k for y in got if not torch.equal(y, want[k]))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_with_parts(q):
    """Two captured graphs, each with the workspace that its call has made, replayed at once on two streams."""
    M, N, K = PARTS
    rng = np.random.default_rng(7)
    wq, ws, _ = _form(q, rng, N, K)
    xs = [[_form(q, rng, M, K)[:2] for _ in range(4)] for _ in range(2)]
    want = [[q.gemm4(*x, wq, ws) for x in row] for row in xs]
    streams, graphs, held, made = [torch.cuda.Stream() for _ in range(2)], [], [], []
    for k in range(2):
        c, s = (t.clone() for t in xs[k][0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = q.gemm4(c, s, wq, ws)
        graphs.append(g), held.append((c, s)), made.append(y)
    for i in range(4):
        for k in range(2):
            held[k][0].copy_(xs[k][i][0]), held[k][1].copy_(xs[k][i][1])
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(made[k], want[k][i]) for k in range(2)), i


def test_outputs_carry_no_history(q):
    x = torch.randn((4, 600), device=DEV, requires_grad=True)
    c, s = q.quant4(x)
    assert not c.requires_grad and not q.dequant4(c, s, 600).requires_grad
    c, s, h = q.rmsnorm4(x)
    assert h is x and not c.requires_grad
    with pytest.raises(ValueError, match="gradient"):
        q.rmsnorm4(x, residual=x.detach())
    with torch.no_grad():
        q.rmsnorm4(x, residual=x)
