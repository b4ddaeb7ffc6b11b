"""The build of the library and of the row operators' Python module, with every compiler call recorded
instead of run: what is built where torch is missing, and when torch has changed."""
import os
import sys

import pytest
import torch

import dense_linear_solvers_gb300 as bs
from dense_linear_solvers_gb300 import _build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Products go to a folder of the test; the commands, each of which writes its output empty."""
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "objects"))
    for name in ("LIB", "PROBE_LIB", "ROWCALL"):
        monkeypatch.setattr(_build, name,
                            str(tmp_path / os.path.basename(getattr(_build, name))))
    seen = []

    def run(command, **_):
        seen.append(command)
        open(command[command.index("-o") + 1], "w").close()

    monkeypatch.setattr(_build.subprocess, "check_call", run)
    return seen


def outputs(commands):
    return {os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in commands}


def test_the_library_without_torch(commands, monkeypatch):
    """nvcc alone builds the C library."""
    monkeypatch.setitem(sys.modules, "torch", None)  # what importing it then raises: ImportError
    assert _build.build(force=True) == _build.LIB
    assert os.path.exists(_build.LIB) and os.path.exists(_build.PROBE_LIB)
    assert not os.path.exists(_build.ROWCALL)
    assert all(os.path.basename(c[0]) == "nvcc" for c in commands)
    commands.clear()
    _build.build()
    assert commands == []


def test_the_library_without_headers(commands, monkeypatch):
    paths = dict(_build.sysconfig.get_paths(), include=os.path.dirname(_build.BUILD))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: paths)
    _build.build(force=True)
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.ROWCALL)


def test_nothing_is_built_twice(commands):
    _build.build()
    assert {"libbsolve.so", "libbsolve_probe.so", "_rowcall.so"} <= outputs(commands)
    commands.clear()
    _build.build()
    assert commands == []


def test_another_torch(commands, monkeypatch):
    """The module is compiled again where torch's version or folder has changed, the library is not."""
    _build.build()
    folder, version = _build._torch()
    assert version == str(torch.__version__)
    for found in ((folder, "0.0.1"), (folder, version)):
        commands.clear()
        monkeypatch.setattr(_build, "_torch", lambda: found)
        _build.build()
        assert outputs(commands) == {"rowcall.o", "_rowcall.so"}, found
        assert any(_build.rowcall_target(found[1]) in a for a in commands[0])


def test_a_module_for_another_torch_is_refused(monkeypatch):
    """It would read tensors by another object layout."""
    _build.build()
    monkeypatch.setattr(bs, "_marshal", None)
    assert bs.bs_grec_tape_rows(1, 32) == 2
    monkeypatch.setattr(bs, "_marshal", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="compiled for torch"):
        bs.bs_grec_tape_rows(1, 32)
    monkeypatch.setattr(_build, "ROWCALL", "nowhere/_rowcall.so")
    with pytest.raises(RuntimeError, match="missing"):
        bs.bs_grec_tape_rows(1, 32)
