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

    for name, at in (("OBJ", "_build"), ("LIB", "libkda_gb300.so"), ("BIND", "_bind.so"), ("PKG", "")):
        monkeypatch.setattr(B, name, str(tmp_path / at))
    monkeypatch.setattr(subprocess, "run", run)
    return made


def test_the_binding_alone_is_built_without_the_folder_of_objects(compilers, monkeypatch):
    monkeypatch.setattr(B, "up_to_date", lambda lib=None: True)
    B.build()
    assert compilers == ["kda_bind.o", "_bind.so.tmp"] and os.path.exists(B.BIND)
