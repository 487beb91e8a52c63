"""The C ABI is built with hipcc alone: neither PyTorch nor g++ has to be there."""

import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from gemv_tq2_g128_amd import build as B


@pytest.fixture
def compiled(monkeypatch):
    """What would be compiled."""
    done = []
    monkeypatch.setattr(B, "_compile", lambda sources, name, verbose: done.append(name) or name)
    monkeypatch.setattr(B, "_run", lambda cmd, verbose: done.append(cmd))
    monkeypatch.setattr(os, "replace", lambda a, b: None)
    return done


def test_without_torch(monkeypatch, compiled, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(sys.modules, "torch", None)               # importing it raises
    assert B.build() == B.LIB_NAME
    assert compiled == [B.PROBE_LIB_NAME, B.LIB_NAME]
    assert B.BINDING_NAME in capsys.readouterr().out


def test_with_torch(compiled):
    pytest.importorskip("torch")
    assert B.build() == B.LIB_NAME
    assert compiled[:2] == [B.PROBE_LIB_NAME, B.LIB_NAME] and B.BINDING_SOURCE in " ".join(compiled[2])


def test_without_gcc(monkeypatch, tmp_path):
    """The host compiler that ROCm brings builds the same module."""
    pytest.importorskip("torch")
    which = shutil.which
    monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    assert os.path.exists(B.host_compiler()) and "g++" not in B.host_compiler().replace("clang++", "")
    monkeypatch.setattr(B, "BINDING_NAME", os.path.join(str(tmp_path), "_binding.so"))
    B._compile_binding(False)
    res = subprocess.run([sys.executable, "-c", "import ctypes, sys; from gemv_tq2_g128_amd import attn; "
                          "import importlib.util as u; s = u.spec_from_file_location('_binding', sys.argv[1]); "
                          "m = u.module_from_spec(s); s.loader.exec_module(m); print(sorted(n for n in dir(m) if n[0] != '_'))",
                          str(tmp_path / "_binding.so")], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                         env={**os.environ, "LD_LIBRARY_PATH": B.PKG_DIR + ":" + os.environ.get("LD_LIBRARY_PATH", "")},
                         cwd=os.path.dirname(B.PKG_DIR))
    assert "['kv_append', 'paged_attention', 'q4_gemv']" in res.stdout, res.stdout
