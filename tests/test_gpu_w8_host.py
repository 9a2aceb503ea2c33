"""The compiled short way of the 8-bit binding: what it does with failures, with the interpreter lock, and
with products that need a workspace."""
import ctypes
import gc
import threading

import numpy as np
import pytest
import torch

from helpers import DEV
from test_gpu_w8 import _code_matrix, _want

pytestmark = pytest.mark.gpu


def _bind(q, fn):
    """The compiled module with `fn` in place of every function of the library that launches."""
    address = ctypes.cast(fn, ctypes.c_void_p).value
    size = ctypes.cast(q.load().qamw_gemm8_workspace, ctypes.c_void_p).value
    q.w8._host.bind(address, address, address, size, address, q.w8._failed)


def _tensors():
    one = lambda *s, **k: torch.ones(s, device=DEV, **k)
    return one(4, 64), one(4, 64, dtype=torch.int8), one(4)


def _calls(q):
    x, c, s = _tensors()
    return [lambda: q.quant8(x), lambda: q.dequant8(c, s), lambda: q.rmsnorm8(x, residual=x),
            lambda: q.gemm8(c, s, c, s)]


@pytest.mark.parametrize("which", range(4), ids=["quant8", "dequant8", "rmsnorm8", "gemm8"])
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
        q.w8.bind(q.load())
    call()


def test_memory_that_is_not_there_is_asked_for_once(q):
    """Without room for the output the allocator's error comes out as it is, and the call ends there."""
    c = torch.ones((1 << 16, 16), dtype=torch.int8, device=DEV)
    s = torch.ones(1 << 16, device=DEV)
    ooms = lambda: torch.cuda.memory_stats()["num_ooms"]
    before = ooms()
    torch.cuda.empty_cache()   # no block that would do is kept from earlier
    torch.cuda.set_per_process_memory_fraction(0.02)   # of 288 GB; the output takes 17
    try:
        with pytest.raises(torch.OutOfMemoryError):
            q.gemm8(c, s, c, s, out_dtype=torch.float32)
        assert ooms() == before + 1
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)


def test_other_threads_run_during_a_launch(q):
    """The library is called without the interpreter lock, as through ctypes: in place of the library's functions
    stands the interpreter's own check for the lock, which gives 0 (no error) only where it is not held."""
    h, (x, c, s) = q.w8._host, _tensors()
    assert ctypes.pythonapi.PyGILState_Check() == 1   # held here
    try:
        _bind(q, ctypes.pythonapi.PyGILState_Check)
        assert h.quant8(x, None, None) is not None
        assert h.dequant8(c, s, None, True) is not None
        assert h.rmsnorm8(x, None, 1e-5, x) is not None
        assert h.gemm8(c, s, c, s, True) is not None
    finally:
        q.w8.bind(q.load())


def test_gradients_are_not_cut_off(q):
    """A residual stream that records gradients is refused by the compiled way too; without recording it is taken."""
    x = torch.ones((4, 64), device=DEV)
    for a, b in ((x.clone().requires_grad_(), x), (x, x.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            q.rmsnorm8(a, residual=b)
        with torch.no_grad():
            assert torch.equal(q.rmsnorm8(a, residual=b)[2], 2 * x)
    a = x.clone().requires_grad_()
    assert q.rmsnorm8(a)[2] is a
    assert not q.rmsnorm8(x, torch.ones(64, device=DEV, requires_grad=True), residual=x)[2].requires_grad


# products with k in parts, whose sums wait in a workspace that the call makes
PARTS = [(77, 4096, 11008), (200, 1024, 4096)]


def _parts(q, seed=0):
    rng = np.random.default_rng(seed)
    cases = []
    for M, N, K in PARTS:
        assert q.gemm8_workspace(M, N, K) > 0
        cases.append((_code_matrix(rng, M, K), torch.from_numpy(rng.random(M, dtype=np.float32)).to(DEV),
                      _code_matrix(rng, N, K), torch.from_numpy(rng.random(N, dtype=np.float32)).to(DEV)))
    return cases


@pytest.mark.parametrize("od", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_products_in_parts(q, od, monkeypatch):
    """By the compiled way, alone and through the package, and by the long way; nothing stays allocated."""
    for case in _parts(q):
        want = _want(*case, od)
        assert torch.equal(q.gemm8(*case, out_dtype=od), want)
        made = q.w8._host.gemm8(*case, od is torch.bfloat16)
        assert made is not None and torch.equal(made, want)
        with monkeypatch.context() as m:
            m.setattr(q.w8, "_host", None)
            assert torch.equal(q.gemm8(*case, out_dtype=od), want)
        del made
        gc.collect()   # tensors that errors of earlier calls still hold, or they go during the count
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        for _ in range(50):
            q.gemm8(*case, out_dtype=od)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == before


def test_products_in_parts_on_two_streams(q):
    """Calls that may overlap, on streams of their own: each has a workspace to itself."""
    cases = _parts(q, 1)
    want = [_want(*c, torch.bfloat16) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            got.append((q.gemm8(*cases[i // 2 % 2]), want[i // 2 % 2]))
    torch.cuda.synchronize()
    for i, (y, w) in enumerate(got):
        assert torch.equal(y, w), i


def test_products_in_parts_in_a_graph(q):
    """Captured without a workspace of the caller's; replays with other inputs and eager calls between."""
    cases = _parts(q, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in cases:
            q.gemm8(*c)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = [q.gemm8(*c) for c in cases]
    for i in range(4):
        for c in cases:
            c[0].copy_(torch.randint_like(c[0], -128, 128))
            c[1].uniform_()
        want = [_want(*c, torch.bfloat16) for c in cases]
        eager = [q.gemm8(*c) for c in cases]
        torch.cuda.synchronize()
        for y in made:
            y.fill_(float("nan"))
        graph.replay()
        more = [q.gemm8(*c) for c in cases]
        torch.cuda.synchronize()
        for y, e, m, w in zip(made, eager, more, want):
            assert torch.equal(y, w) and torch.equal(e, w) and torch.equal(m, w), i


def test_errors_of_others_are_not_ours(q):
    """A call answers for its own launches: an error that an earlier call of the runtime left is not its error, and
    stays for whoever asks for it."""
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
    hip = ctypes.CDLL(paths.pop())
    assert not paths
    calls = _calls(q) + [lambda c=c: q.gemm8(*c) for c in _parts(q)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    for call in calls:
        assert hip.hipSetDevice(1 << 20) != 0   # no such device: refused, and remembered
        call()
        assert hip.hipGetLastError() != 0
        assert hip.hipGetLastError() == 0
    torch.cuda.synchronize()


def test_calls_of_several_threads(q):
    """Threads with a stream each, whose calls overlap on the host and on the GPU."""
    cases = _parts(q, 3) + [_parts(q, 4)[1]]
    want = [_want(*c, torch.bfloat16) for c in cases]
    x = [torch.randn((50 + i, 1003), device=DEV) for i in range(len(cases))]
    rows = [q.quant8(v) for v in x]
    torch.cuda.synchronize()
    wrong, done = [], []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(40):
                y, (c, s) = q.gemm8(*cases[i]), q.quant8(x[i])
                if not (torch.equal(y, want[i]) and torch.equal(c, rows[i][0]) and torch.equal(s, rows[i][1])):
                    wrong.append(i)
        stream.synchronize()
        done.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and sorted(done) == [0, 1, 2]
