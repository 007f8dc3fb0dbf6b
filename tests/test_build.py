"""What the build needs and when it builds again, on the host and without a compiler: the library
does not wait for torch or for the extension module, which follows the installed torch."""
import importlib.metadata
import os
import sys
import types

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    from paged_kv_cache_414_b200 import build
    made = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        if build.FAIL in out:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        made.append(os.path.basename(out))
        with open(out, "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "FAIL", "nothing fails", raising=False)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpa.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "made", made, raising=False)
    return build


def test_the_library_without_torch(build, monkeypatch):
    def version(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", version)
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.CALLS)


def test_the_library_when_the_module_does_not_compile(build, monkeypatch):
    monkeypatch.setattr(build, "FAIL", "_calls")
    with pytest.raises(RuntimeError):
        build.build()
    assert os.path.exists(build.LIB)


def test_the_module_follows_torch(build, monkeypatch):
    build.build()
    assert {"libpa.so.tmp", "_calls.so.tmp"} <= set(build.made)
    build.made.clear()
    build.build()
    assert build.made == []
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    build.build()
    assert build.made == ["_calls.so.tmp"]
    build.build()
    assert build.made == ["_calls.so.tmp"]
