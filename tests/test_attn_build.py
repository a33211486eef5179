"""The build and the binding's parts, without a GPU: the library does not depend on the binding's native half, and parts of
another version are refused by name."""
import ctypes
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


def test_a_library_of_another_version_is_refused_by_version(monkeypatch, tmp_path):
    """Before any entry point is looked up that it may not have."""
    src, so = tmp_path / "old.c", tmp_path / "old.so"
    src.write_text(f"int ssm_abi_version(void) {{ return {L.ABI_VERSION - 1}; }}\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(L, "_lib", None)
    with pytest.raises(ImportError, match=f"ABI {L.ABI_VERSION - 1}"):
        L.load(str(so))


def test_the_attention_entry_points_have_a_version_of_their_own():
    """Version 2 is the library without them."""
    assert L.ABI_VERSION == 3
    with open(os.path.join(B.ROOT, "include", "ssm.h")) as f:
        assert "#define SSM_ABI_VERSION 3\n" in f.read()


def test_a_native_half_of_another_version_is_refused(monkeypatch):
    """It fills the library's structures by the layout it was compiled with."""
    from selective_state_space_causal_amd import _attn_fast
    lib = L.load()
    entries = [ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
        "ssm_rope", "ssm_kv_write", "ssm_kv_read", "ssm_attn_prefill", "ssm_attn_decode_step", "ssm_attn_decode_workspace_bytes")]
    with pytest.raises(ImportError, match="ABI"):
        _attn_fast.bind(L.ABI_VERSION + 1, *entries, A._fail)
    _attn_fast.bind(L.ABI_VERSION, *entries, A._fail)

    for error in (ImportError, TypeError):  # TypeError: of before versions were compared
        def refuses(*args):
            raise error("another ABI")
        monkeypatch.setattr(_attn_fast, "bind", refuses)
        monkeypatch.setattr(A, "_native", None)
        with pytest.warns(UserWarning, match="another ABI"):
            assert A._bound() is A._NoNative
