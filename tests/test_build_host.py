"""The build (CPU): libfa.so and its ctypes entry points need no compiled binding (g++, PyTorch headers), and the binding is
built for the Python and PyTorch that load it."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import attention_forward_05_gb300 as fa
from attention_forward_05_gb300 import _build


def test_library_loads_where_the_binding_cannot_be_built(tmp_path):
    """A fresh tree with a built libfa.so, no binding and a g++ that fails: lib() works, the compiled binding raises."""
    fa.lib()
    root = os.path.dirname(os.path.dirname(os.path.abspath(fa.__file__)))
    shutil.copytree(os.path.join(root, "include"), tmp_path / "include")
    shutil.copytree(os.path.join(root, "attention_forward_05_gb300"), tmp_path / "attention_forward_05_gb300",
                    ignore=shutil.ignore_patterns("_build", "__pycache__"))
    out = tmp_path / "attention_forward_05_gb300" / "_build"
    out.mkdir()
    shutil.copyfile(fa.lib_path(), out / "libfa.so")
    tools = tmp_path / "tools"
    tools.mkdir()
    for name in ("g++", "c++"):
        (tools / name).write_text("#!/bin/sh\nexit 1\n")
        (tools / name).chmod(0o755)
    code = ("import attention_forward_05_gb300 as fa\n"
            "assert fa.lib().fa_rope(*[None] * 5, 1, 4, 2, 8, 64, 1, None, 0, None, None, 1, 64, 0, 0, None) == 1\n"
            "assert fa.fa_bwd_workspace_bytes(1, 2, 64, 64) >= 0\n"
            "try:\n    fa._load_binding()\nexcept RuntimeError as e:\n    assert 'g++' in str(e)\nelse:\n    raise SystemExit('no error')\n"
            "print(fa.__file__)\n")
    env = dict(os.environ, PATH=f"{tools}:{os.environ['PATH']}", PYTHONPATH=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=tmp_path, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().startswith(str(tmp_path))


def test_binding_is_built_for_the_running_pytorch(monkeypatch):
    """Another PyTorch or Python has another file: one that is there for this version is not loaded by it."""
    fa._load_binding()
    path = _build.binding_path()
    assert os.path.exists(path) and not _build.binding_is_stale() and not _build.is_stale()
    monkeypatch.setattr(torch, "__version__", "99.1.0+cu999")
    assert _build.binding_path() != path and _build.binding_is_stale() and not _build.is_stale()
    monkeypatch.undo()
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: ".cpython-399-none.so")
    assert _build.binding_path() != path and _build.binding_is_stale()
    monkeypatch.undo()
    assert _build.binding_path() == path


@pytest.mark.parametrize("newer,library,binding", [("csrc/fa_rope.cu", True, False), ("csrc/fa_binding.cpp", False, True)])
def test_sources_rebuild_what_they_are_part_of(monkeypatch, newer, library, binding):
    fa._load_binding()
    real = os.path.getmtime
    monkeypatch.setattr(_build.os.path, "getmtime", lambda p: real(p) + (1e9 if str(p).endswith(newer) else 0))
    assert _build.is_stale() == library and _build.binding_is_stale() == binding
