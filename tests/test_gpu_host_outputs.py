"""Outputs that the compiled short way makes (csrc/host_calls.hpp), where new tensors are watched or filled: as the long way
makes them."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from helpers import DEV

pytestmark = pytest.mark.gpu


def _calls(q):
    x = torch.randn((9, 300), device=DEV).to(torch.bfloat16)
    a8, b8 = q.quant8(x), q.quant8(torch.randn((40, 300), device=DEV))
    a4, b4 = q.quant4(x), q.quant4(torch.randn((40, 300), device=DEV))
    w, ws = b4[0].view(2, 20, -1), b4[1].view(-1, 2, 20, 8)
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device=DEV)
    return {"quant8": lambda: q.quant8(x), "dequant8": lambda: q.dequant8(*a8), "rmsnorm8": lambda: q.rmsnorm8(x, residual=x),
            "gemm8": lambda: q.gemm8(*a8, *b8), "quant4": lambda: q.quant4(x), "dequant4": lambda: q.dequant4(*a4, 300),
            "rmsnorm4": lambda: q.rmsnorm4(x, residual=x), "gemm4": lambda: q.gemm4(*a4, *b4),
            "gemm4_grouped": lambda: q.gemm4_grouped(*a4, w, ws, off)}


OUTPUTS = {"quant8": 2, "dequant8": 1, "rmsnorm8": 3, "gemm8": 1, "quant4": 2, "dequant4": 1, "rmsnorm4": 3, "gemm4": 1,
           "gemm4_grouped": 1}
EACH = pytest.mark.parametrize("name", list(OUTPUTS))


def _same(a, b):
    a, b = (t if isinstance(t, tuple) else (t,) for t in (a, b))
    assert len(a) == len(b) and all(torch.equal(u, v) for u, v in zip(a, b))


@EACH
def test_dispatch_modes_see_them(q, name):
    class Seen(TorchDispatchMode):
        made = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.made += "empty" in func.name()
            return func(*args, **(kwargs or {}))
    call = _calls(q)[name]
    want = call()
    with Seen() as seen:
        got = call()
    assert seen.made >= OUTPUTS[name]
    _same(got, want)


@EACH
def test_profilers_see_them(q, name):
    call = _calls(q)[name]
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        call()
    assert sum(e.count for e in prof.key_averages() if "empty" in e.key) >= OUTPUTS[name]


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.utils.deterministic.fill_uninitialized_memory = True
    torch.use_deterministic_algorithms(False)


@EACH
def test_under_deterministic_algorithms(q, name, deterministic):
    torch.use_deterministic_algorithms(False)
    call = _calls(q)[name]
    want = call()
    torch.use_deterministic_algorithms(True)
    _same(call(), want)


@pytest.mark.parametrize("short", [True, False], ids=["short way", "long way"])
def test_rows_without_a_group_are_filled(q, short, deterministic, monkeypatch):
    """What no group has is what torch.empty leaves: NaN under deterministic algorithms."""
    c, s = q.quant4(torch.randn((700, 300), device=DEV))
    w, ws = c[:40].view(2, 20, -1), s[:, :40].reshape(-1, 2, 20, 8)
    off = torch.tensor([3, 4, 9], dtype=torch.int32, device=DEV)
    for _ in range(4):   # memory that an output may get, without NaN
        torch.full((700, 20), 7.0, device=DEV, dtype=torch.bfloat16)
    if not short:
        monkeypatch.setattr(q.mx4, "_host", None)
    y = q.gemm4_grouped(c, s, w, ws, off)
    assert y[:3].isnan().all() and y[9:].isnan().all() and not y[3:9].isnan().any()
    torch.utils.deterministic.fill_uninitialized_memory = False
    del y
    torch.full((700, 20), 7.0, device=DEV, dtype=torch.bfloat16)   # freed at once: the next one's memory
    y = q.gemm4_grouped(c, s, w, ws, off)
    assert (y[9:] == 7).all()
