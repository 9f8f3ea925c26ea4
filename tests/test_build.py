"""build(): what it makes again and when, with the compilers replaced by a recorder."""
import os
import subprocess
import sys

import pytest

from paged_kv_decode_table_gb300 import build as B


@pytest.fixture
def recorder(tmp_path, monkeypatch):
    """Targets below tmp_path, and compilers that only create their outputs.  Returns the outputs' names."""
    made = []
    for name in ("LIB", "CALLS"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "b"))
    if hasattr(B, "CALLS_TAG"):
        monkeypatch.setattr(B, "CALLS_TAG", str(tmp_path / "b" / "torch_calls.tag"))
    monkeypatch.setattr(B, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out).split(".tmp")[0])
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(B.subprocess, "run", run)
    return made


def test_both_are_made_once(recorder):
    B.build()
    assert {"libpkv.so", "_torch_calls.so"} <= set(recorder)
    recorder.clear()
    B.build()
    assert recorder == []


def test_the_library_is_made_without_torch(recorder, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.raises(ImportError):
        B.build()
    assert "libpkv.so" in recorder and os.path.exists(B.LIB)


def test_the_library_is_made_where_the_module_does_not_compile(recorder, monkeypatch):
    ok = B.subprocess.run

    def run(cmd, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        return ok(cmd, **kw)
    monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no such header"):
        B.build()
    assert "libpkv.so" in recorder and os.path.exists(B.LIB)


def test_a_module_of_another_torch_or_python_is_made_again(recorder, monkeypatch):
    import torch
    B.build()
    recorder.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    B.build()
    assert "_torch_calls.so" in recorder and "libpkv.so" not in recorder
    recorder.clear()
    monkeypatch.setattr(B.sys if hasattr(B, "sys") else sys, "version_info", (3, 99, 0, "final", 0))
    B.build()
    assert "_torch_calls.so" in recorder and "libpkv.so" not in recorder
