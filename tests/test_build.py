"""The build's decisions, with compilers that only pretend: what is compiled again, and what a
missing part of the toolchain costs."""
import os
import subprocess
import types

import pytest
import torch

from jagged_sequence_attention_gb300 import _build


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """Compilers that write what they are asked for, and a build folder of their own."""
    ran, broken = [], []

    def run(cmd, **kw):
        ran.append(" ".join(cmd))
        if any(b in ran[-1] for b in broken):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libjfa.so"))
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / os.path.basename(_build.CALLS)))
    monkeypatch.setattr(_build, "_nvcc", lambda: "nvcc")

    def build():
        ran.clear()
        assert _build.build() == _build.LIB
        return sorted(ran)

    return types.SimpleNamespace(build=build, broken=broken)


def test_nothing_is_compiled_twice(tools):
    assert len(tools.build()) == len(_build.SOURCES) + 2
    assert tools.build() == []


def test_another_torch_compiles_the_calls_again(tools, monkeypatch):
    tools.build()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")  # an upgrade in place: the same paths
    (cmd,) = tools.build()
    assert "cache_calls.cpp" in cmd
    assert tools.build() == []


def test_the_library_is_built_where_the_calls_cannot_be(tools):
    tools.broken.append("cache_calls.cpp")
    with pytest.warns(RuntimeWarning, match="no such header"):
        tools.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.CALLS)
    tools.broken.clear()
    (cmd,) = tools.build()  # and the calls once they can be
    assert "cache_calls.cpp" in cmd and os.path.exists(_build.CALLS)
    # one that can no longer be built from its sources does not stay as it was
    tools.broken.append("cache_calls.cpp")
    os.remove(os.path.join(_build.BUILD, "cache_calls.stamp"))
    with pytest.warns(RuntimeWarning):
        tools.build()
    assert not os.path.exists(_build.CALLS)


def test_without_torch_the_library_is_built(tools, monkeypatch):
    import builtins
    real = builtins.__import__

    def no_torch(name, *a, **k):
        if name == "torch":
            raise ImportError("no torch here")
        return real(name, *a, **k)

    monkeypatch.setattr(builtins, "__import__", no_torch)
    with pytest.warns(RuntimeWarning, match="no torch here"):
        tools.build()
    assert os.path.exists(_build.LIB)


def test_a_broken_library_is_an_error(tools):
    tools.broken.append("fwd.cu")
    with pytest.raises(RuntimeError, match="fwd.cu"):
        tools.build()


def test_calls_are_named_for_the_interpreter():
    import sysconfig
    assert os.path.basename(_build.CALLS) == "_cache_calls" + sysconfig.get_config_var("EXT_SUFFIX")


def test_missing_calls_fail_loudly(monkeypatch):
    _build.build()
    from jagged_sequence_attention_gb300 import jfa
    monkeypatch.setattr(jfa, "_calls", None)
    monkeypatch.setitem(__import__("sys").modules, "jagged_sequence_attention_gb300._cache_calls", None)
    monkeypatch.delattr("jagged_sequence_attention_gb300._cache_calls", raising=False)
    with pytest.raises(RuntimeError, match="not built"):
        jfa._cache_calls()
