"""The build and the binding's parts, without a GPU: the library does not depend on the binding's native half, and parts of
another version are refused by name."""
import ctypes
import importlib.machinery
import importlib.util
import os
import subprocess

import pytest

from selective_state_space_causal_amd import _lib as L
from selective_state_space_causal_amd import attn as A
from selective_state_space_causal_amd import build as B


def test_the_library_is_built_where_the_native_half_is_not(monkeypatch, tmp_path):
    """A host compiler or torch headers that are missing cost the native half, which attn.py does without, and not the
    library; a native half of an earlier build does not stay beside it."""
    for name in ("LIB", "FAST"):
        monkeypatch.setattr(B, name, str(tmp_path / f"{name}.so"))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "sources", lambda: ["a.hip"])
    (tmp_path / "FAST.so").write_text("of an earlier build")
    done = []

    def run(cmd, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file")
        done.append("-shared" in cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.warns(UserWarning, match="Python.h"):
        assert B.build() == str(tmp_path / "LIB.so")
    assert done == [False, True] and (tmp_path / "LIB.so").read_text() == "made"
    assert not os.path.exists(tmp_path / "FAST.so")
