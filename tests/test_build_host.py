"""The build's steps on the host (no GPU and no nvcc needed: the compilers are stood in for)."""
import os
import subprocess
import types

import pytest

from fp8_quant_memory_gb300 import build


@pytest.fixture
def out(tmp_path, monkeypatch):
    """The build writes to tmp_path; compiling and linking only create their outputs."""
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfq.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_fq_binding.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src + ".o")

    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    return tmp_path


def test_the_library_does_not_need_the_binding(out, monkeypatch):
    """Without Python's or torch's headers the binding fails, loudly, and the C library is built all the same."""
    def fail():
        raise RuntimeError("g++ failed on fq_binding.cpp: Python.h: No such file or directory")

    monkeypatch.setattr(build, "_compile_binding", fail)
    (out / "_fq_binding.so").touch()  # an earlier build's, which may not fit the new library
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build(force=True)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert not build.up_to_date()


def test_library_and_binding(out, monkeypatch):
    monkeypatch.setattr(build, "_compile_binding", lambda: "fq_binding.o")
    monkeypatch.setattr(build, "_torch_paths", lambda: ([], "lib"))
    assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
