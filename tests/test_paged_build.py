"""The build of the paged calls' marshalling module: a module that does not belong to the library is never left."""
import os
import shutil

import pytest

from local_linear_attention_flashlla_gb300 import build as lla_build


@pytest.fixture
def stale(tmp_path, monkeypatch):
    """A module of an earlier build, in a folder of its own."""
    path = tmp_path / "_paged_bind.so"
    path.write_bytes(b"of an earlier build")
    monkeypatch.setattr(lla_build, "BIND", str(path))
    return path


def test_without_a_compiler_none_is_left(stale, monkeypatch):
    monkeypatch.setattr(lla_build.shutil, "which", lambda name: None)
    assert lla_build.build_binding() is None
    assert not stale.exists()


def test_without_the_headers_none_is_left(stale, monkeypatch, tmp_path):
    monkeypatch.setattr(lla_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert lla_build.build_binding() is None
    assert not stale.exists()


def test_where_it_does_not_compile_the_build_goes_on(stale, monkeypatch, tmp_path):
    if not (shutil.which("gcc") or shutil.which("cc")):
        pytest.skip("no C compiler")
    if not os.path.exists(os.path.join(lla_build.sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers")
    (tmp_path / "paged_bind.c").write_text("this is not C\n")
    monkeypatch.setattr(lla_build, "CSRC", str(tmp_path))
    with pytest.warns(UserWarning, match="marshalled in Python"):
        assert lla_build.build_binding() is None
    assert not stale.exists()


def test_a_library_that_does_not_compile_leaves_both_as_they_were(stale, monkeypatch, tmp_path):
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "broken.cu").write_text("this is not C++\n")
    lib = tmp_path / "liblla.so"
    lib.write_bytes(b"library of an earlier build")
    monkeypatch.setattr(lla_build, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(lla_build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(lla_build, "LIB", str(lib))
    with pytest.raises(RuntimeError):
        lla_build.build()
    assert lib.read_bytes() == b"library of an earlier build" and stale.read_bytes() == b"of an earlier build"


def test_the_module_is_built_after_the_library(stale, monkeypatch, tmp_path):
    """The order of the steps, with commands that only write their output."""
    steps = []

    def fake(cmd):
        out = cmd[cmd.index("-o") + 1]
        steps.append((os.path.basename(out), stale.exists() and stale.read_bytes() == b"of an earlier build"))
        with open(out, "wb") as f:
            f.write(b"new")
        return ""

    monkeypatch.setattr(lla_build, "_run", fake)
    monkeypatch.setattr(lla_build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(lla_build, "LIB", str(tmp_path / "liblla.so"))
    lla_build.build()
    names = [n for n, _ in steps]
    assert "liblla.so.tmp" in names
    if "_paged_bind.so.tmp" in names:
        assert names[-1] == "_paged_bind.so.tmp" and names[-2] == "liblla.so.tmp"
        assert not steps[-1][1]                      # the module before was gone when the new library was there
        assert stale.read_bytes() == b"new"
    else:
        assert not stale.exists()
