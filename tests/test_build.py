"""What the build makes where Python's headers, which only the binding's decode calls need, are missing
or do not compile: the library all the same.  (The compilers are stand-ins here.)"""
import os
import subprocess
import sysconfig
import types

import pytest

from block_scaled_fp8_gb300 import build as b


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """build() into tmp_path; nvcc always works, gcc if `state.gcc` and its include folders hold Python.h."""
    state = types.SimpleNamespace(gcc=True, include=tmp_path / "include", lib=str(tmp_path / "lib.so"),
                                  marshal=str(tmp_path / "marshal.so"))
    state.include.mkdir()

    def run(cmd, **kw):
        ok = "gcc" not in os.path.basename(cmd[0]) or (
            state.gcc and any(os.path.exists(os.path.join(d, "Python.h")) for d in cmd))
        if ok:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0 if ok else 1, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(state.include)})
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", state.lib)
    monkeypatch.setattr(b, "MARSHAL", state.marshal)
    monkeypatch.delenv("CC", raising=False)
    return state


@pytest.mark.filterwarnings("ignore:Python.h")
def test_without_python_headers_the_library_is_built(fake):
    open(fake.marshal, "w").close()       # of an earlier build
    assert b.build(force=True) == fake.lib
    assert os.path.exists(fake.lib) and not os.path.exists(fake.marshal)
    assert b.up_to_date()


def test_with_python_headers_both_are_built(fake):
    (fake.include / "Python.h").touch()
    b.build(force=True)
    assert os.path.exists(fake.lib) and os.path.exists(fake.marshal)
    os.remove(fake.marshal)
    assert not b.up_to_date()


def test_a_failed_extension_leaves_the_library(fake):
    (fake.include / "Python.h").touch()
    fake.gcc = False
    with pytest.raises(RuntimeError, match="gcc failed"):
        b.build(force=True)
    assert os.path.exists(fake.lib)
