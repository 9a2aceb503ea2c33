"""The compiled short way of the 8-bit binding: what it does with failures, with the interpreter lock, and
with products that need a workspace."""
import ctypes

import pytest
import torch

from helpers import DEV

pytestmark = pytest.mark.gpu


def _bind(q, fn):
    """The compiled module with `fn` in place of every function of the library that launches."""
    address = ctypes.cast(fn, ctypes.c_void_p).value
    size = ctypes.cast(q.load().qamw_gemm8_workspace, ctypes.c_void_p).value
    q.w8._host.bind(address, address, address, size, address, q.w8._failed)


def _tensors():
    return torch.ones((4, 64), device=DEV), torch.ones((4, 64), dtype=torch.int8, device=DEV), torch.ones(4, device=DEV)


def _calls(q):
    x, c, s = _tensors()
    return [lambda: q.quant8(x), lambda: q.dequant8(c, s), lambda: q.rmsnorm8(x, residual=x), lambda: q.gemm8(c, s, c, s)]


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
