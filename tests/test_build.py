"""The build's own rules, with compilers replaced by a recorder."""
import os
import sys
import types

import pytest

from gguf_block_quantized_kind_amd import _build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Builds into tmp_path; every command is recorded and only leaves its output file."""
    ran = []

    def run(cmd, **kw):
        ran.append(list(cmd))
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "OBJDIR", str(tmp_path / "obj"))
    for name in ("LIBRARY", "PROBE_LIBRARY", "CALL_MODULE"):
        monkeypatch.setattr(_build, name, str(tmp_path / name))
    return ran


def test_the_library_builds_without_torch(commands, monkeypatch, tmp_path):
    for name in ("torch", "torch.utils", "torch.utils.cpp_extension"):
        monkeypatch.setitem(sys.modules, name, None)
    assert _build.build() == _build.LIBRARY
    assert os.path.exists(_build.LIBRARY) and os.path.exists(_build.PROBE_LIBRARY)
    assert not os.path.exists(_build.CALL_MODULE)
    assert all(cmd[0] == _build.hipcc() for cmd in commands)


def test_the_call_module_takes_the_compilers_rocm(commands, monkeypatch, tmp_path):
    pytest.importorskip("torch")
    cc = tmp_path / "rocm" / "bin" / "hipcc"
    cc.parent.mkdir(parents=True)
    cc.write_text("")
    monkeypatch.setenv("HIPCC", str(cc))
    _build.build()
    call = [cmd for cmd in commands if _build.CALL_SOURCE in cmd]
    assert len(call) == 1 and str(tmp_path / "rocm" / "include") in call[0]
    assert os.path.exists(_build.CALL_MODULE)
