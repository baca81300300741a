"""What the build compiles and links, with the compilers replaced by a recorder (no GPU, nothing compiled)."""
import os
import subprocess
import sys

import pytest

from quantised_gguf_weight_gb300 import build as qbuild


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Command lines of the build, in a folder of its own; each makes its output file."""
    ran = []
    monkeypatch.setattr(qbuild, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(qbuild, "LIB", str(tmp_path / "libqk.so"))
    monkeypatch.setattr(qbuild, "BINDING", str(tmp_path / "qk_torch.so"))
    monkeypatch.setattr(qbuild, "BINDING_FOR", str(tmp_path / "qk_torch.for"), raising=False)

    def run(cmd):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    class Popen:
        returncode = 0

        def __init__(self, cmd, **kw):
            run(cmd)

        def communicate(self):
            return b"", None

    monkeypatch.setattr(subprocess, "Popen", Popen)
    monkeypatch.setattr(subprocess, "check_call", run)
    return ran


def made(ran):
    return {os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in ran}


def test_library_and_binding(commands):
    qbuild.build()
    assert {"libqk.so", "qk_torch.so", "qk_torch.cpp.o", "qk_api.cu.o"} <= made(commands)
    assert qbuild.up_to_date()
    commands.clear()
    qbuild.build()
    assert not commands


def test_library_without_torch(commands, monkeypatch):
    """A C user needs no torch: the library is built and up to date, without the binding."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert qbuild.build() == qbuild.LIB and os.path.exists(qbuild.LIB)
    assert "libqk.so" in made(commands) and not any("torch" in m for m in made(commands))
    assert qbuild.up_to_date()


def test_binding_alone_where_the_library_is_there(commands, monkeypatch):
    """torch installed later: only the binding is compiled."""
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        qbuild.build()
    commands.clear()
    assert not qbuild.up_to_date()
    qbuild.build()
    assert made(commands) == {"qk_torch.cpp.o", "qk_torch.so"} and qbuild.up_to_date()


def test_binding_for_another_torch(commands, monkeypatch):
    """A torch of another version has another binary interface: the binding is made again, the library is not."""
    import torch
    qbuild.build()
    commands.clear()
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    assert not qbuild.up_to_date()
    qbuild.build()
    assert made(commands) == {"qk_torch.cpp.o", "qk_torch.so"} and qbuild.up_to_date()
