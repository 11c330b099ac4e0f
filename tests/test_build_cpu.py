"""What ``build()`` decides and where it writes, with the compilers stood in for (CPU only)."""
import os
import subprocess
import sys

import pytest

from linear_attention_serving_chunkwise_gb300 import build as B


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Paths of a tree that has never been built, and compilers that write what they are asked for; the list of what that was."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name, at in (("OBJ", "_build"), ("LIB", "libkda_gb300.so"), ("BIND", "_bind.so")):
        monkeypatch.setattr(B, name, str(tmp_path / at))
    monkeypatch.setattr(subprocess, "run", run)
    return made


def test_the_binding_alone_is_built_without_the_folder_of_objects(compilers, monkeypatch):
    monkeypatch.setattr(B, "up_to_date", lambda lib=None: True)
    B.build()
    assert compilers == ["kda_bind.o", "_bind.so.tmp"] and os.path.exists(B.BIND)


WITHOUT_TORCH = """
import importlib.util, os, subprocess, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("build_alone", {path!r})
B = importlib.util.module_from_spec(spec)
spec.loader.exec_module(B)
for name in ("OBJ", "LIB", "BIND"):
    setattr(B, name, os.path.join({tmp!r}, name))
made = []

def run(cmd, **kw):
    out = cmd[cmd.index("-o") + 1]
    open(out, "w").close()
    made.append(os.path.basename(out))
    return subprocess.CompletedProcess(cmd, 0, "", "")

subprocess.run = run
B.build()
assert os.path.exists(B.LIB) and "kda_bind.o" not in made and not os.path.exists(B.BIND), made
B.build()                                                # and it is current
assert made.count("LIB.tmp") == 1, made
"""


def test_the_library_is_built_without_pytorch(tmp_path):
    """The C library needs nvcc alone; only its Python binding needs PyTorch."""
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH.format(path=B.__file__, tmp=str(tmp_path))], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "PyTorch" in r.stderr


@pytest.mark.parametrize("what", ["version", "folder", "interpreter"])
def test_a_binding_of_another_pytorch_or_python_is_built_anew(compilers, monkeypatch, what):
    """The stamp names all that the binding was compiled for; PyTorch's folder is in its search path."""
    import sysconfig
    import torch
    B.build()
    compilers.clear()
    B.build()
    assert compilers == []
    if what == "version":
        monkeypatch.setattr(torch, "__version__", "0.1")
    elif what == "folder":
        monkeypatch.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")
    else:
        of = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else of(name))
    B.build()
    assert "_bind.so.tmp" in compilers
    compilers.clear()
    B.build()
    assert compilers == []
