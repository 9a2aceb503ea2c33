"""The build entry point where the binding's optional host module does not compile."""
import os

import pytest

import __graft_entry__
import oracle
import synth_inputs
import weight_quantization_codec_amd as q
from weight_quantization_codec_amd import _build


@pytest.mark.parametrize("compiler", ["false", "/nowhere/c++"], ids=["fails", "missing"])
def test_build_without_the_host_module(monkeypatch, tmp_path, compiler):
    """The calls work without the module (w8.py), so the build goes on, says so, and leaves no older module behind,
    which might not fit the library."""
    done = []
    for mod, name in ((_build, "build"), (oracle, "build"), (synth_inputs, "build"), (synth_inputs, "build_gpu")):
        monkeypatch.setattr(mod, name, lambda *a, name=name, **k: done.append(name))
    monkeypatch.setattr(q, "load", lambda: done.append("load"))
    monkeypatch.setattr(_build, "HOST", str(tmp_path / "_w8_host.so"))
    monkeypatch.setenv("CXX", compiler)
    open(_build.HOST, "w").write("an older build")
    with pytest.warns(UserWarning, match="w8_host"):
        __graft_entry__.build()
    assert done == ["build", "build", "build", "build_gpu", "load"]
    assert not os.path.exists(_build.HOST)
