"""What the build does again and what it does without, with the compilers replaced by a recorder."""
import os
import types

import pytest

from block_scaled_mlp_gb300 import _build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Commands that were run; `fails(cmd)` decides which ones fail.  Outputs go to a folder of the test's own."""
    c = types.SimpleNamespace(ran=[], fails=lambda cmd: False)

    def run(cmd, **kw):
        c.ran.append(cmd)
        if c.fails(cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libmxmlp.so"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    return c


def _binding(cmd):
    return any(str(a).endswith(("binding.cpp", "binding.o")) for a in cmd)


def test_builds_everything_once(compilers):
    assert _build.build() == _build.LIB
    assert len(compilers.ran) == len(_build.SOURCES) + 3       # objects, binding.o, two links
    assert os.path.exists(_build.LIB) and os.path.exists(_build.BINDING)
    compilers.ran.clear()
    _build.build()
    assert compilers.ran == []


def test_another_torch_rebuilds_the_binding_alone(compilers, monkeypatch):
    _build.build()
    compilers.ran.clear()
    monkeypatch.setattr("torch.__version__", "0.0.0+other")
    _build.build()
    assert len(compilers.ran) == 2 and all(_binding(c) for c in compilers.ran)
    compilers.ran.clear()
    _build.build()
    assert compilers.ran == []


def test_library_is_built_where_the_binding_does_not_compile(compilers, monkeypatch, capsys):
    _build.build()
    for f in (_build.LIB, os.path.join(_build.BUILD, "api.o")):
        os.remove(f)
    monkeypatch.setattr("torch.__version__", "0.0.0+other")
    compilers.fails = _binding
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB)
    assert not os.path.exists(_build.BINDING)                    # the other torch's is not left behind
    assert "no such header" in capsys.readouterr().err
    compilers.fails = lambda cmd: False
    _build.build()
    assert os.path.exists(_build.BINDING)


def test_a_source_that_does_not_compile_fails_the_build(compilers):
    compilers.fails = lambda cmd: any(str(a).endswith("norm.cu") for a in cmd)
    with pytest.raises(RuntimeError, match="norm.cu"):
        _build.build()
