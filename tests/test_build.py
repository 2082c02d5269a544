"""What the build needs: the C library nvcc and a C++ compiler, and nothing of
torch or Python (the compilers are stood in for)."""

import importlib.metadata
import os

import pytest

from paged_mla_decode_08_gb300 import build as M


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The build moved to an empty folder; its commands are recorded and their outputs made empty."""
    ran = []

    def run(cmd, log):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return ""

    monkeypatch.setattr(M, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(M, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(M, "LIB", str(tmp_path / "lib" / "libmladecode.so"))
    monkeypatch.setattr(M, "CALLS", str(tmp_path / "lib" / "_mla_calls.so"))
    monkeypatch.setattr(M, "_run", run)
    monkeypatch.setattr(M, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return ran


def without_torch(monkeypatch):
    find, version = M.importlib.util.find_spec, importlib.metadata.version

    def no_version(name):
        if name == "torch":
            raise importlib.metadata.PackageNotFoundError(name)
        return version(name)

    monkeypatch.setattr(M.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(M.importlib.metadata, "version", no_version)


def test_the_library_needs_no_torch(commands, monkeypatch):
    without_torch(monkeypatch)
    assert M.build() == M.LIB and os.path.exists(M.LIB) and not os.path.exists(M.CALLS)
    assert not any("torch" in part or "Python.h" in part for cmd in commands for part in cmd)
    made = len(commands)
    assert M.build() == M.LIB and len(commands) == made  # nothing changed


def test_the_library_needs_no_python_headers(commands, monkeypatch, tmp_path):
    paths = M.sysconfig.get_paths()
    monkeypatch.setattr(M.sysconfig, "get_paths", lambda: {**paths, "include": str(tmp_path)})
    assert M.build() == M.LIB and os.path.exists(M.LIB) and not os.path.exists(M.CALLS)


def test_the_module_follows_torch(commands, monkeypatch):
    """Built with torch, rebuilt alone for another torch, gone without."""
    if M._torch_dir() is None:
        pytest.skip("no CUDA torch with headers")
    M.build()
    assert os.path.exists(M.LIB) and os.path.exists(M.CALLS)
    made = len(commands)
    monkeypatch.setattr(M.importlib.metadata, "version", lambda name: "another")
    M.build()
    assert [cmd[cmd.index("-o") + 1] for cmd in commands[made:]] == [
        os.path.join(M.BUILD, M.CALLS_SOURCE + ".o"), M.CALLS + ".tmp"]
    without_torch(monkeypatch)
    M.build()
    assert os.path.exists(M.LIB) and not os.path.exists(M.CALLS)


def test_the_library_is_linked_though_the_module_fails(commands, monkeypatch):
    if M._torch_dir() is None:
        pytest.skip("no CUDA torch with headers")
    run = M._run

    def fails(cmd, log):
        if any(M.CALLS_SOURCE in part for part in cmd):
            raise RuntimeError("build step failed")
        return run(cmd, log)

    monkeypatch.setattr(M, "_run", fails)
    with pytest.raises(RuntimeError):
        M.build()
    assert os.path.exists(M.LIB) and not os.path.exists(M.CALLS)
