"""The build: libdsa.so without torch (a C program needs nothing else), _calls.so for the torch that is
installed."""
import os
import shutil
import subprocess
import sys

import pytest

from sparse_long_context_dsa_b200 import build as B

WITHOUT_TORCH = """
import sys
class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, NoTorch())
from importlib import metadata
def version(name, real=metadata.version):
    if name == "torch":
        raise metadata.PackageNotFoundError(name)
    return real(name)
metadata.version = version
"""


def test_the_library_builds_where_torch_is_missing(tmp_path):
    # a stand-in for nvcc writes the library; g++ is not reached
    root = tmp_path / "tree"
    pkg = root / "sparse_long_context_dsa_b200"
    shutil.copytree(B.CSRC, pkg / "csrc")
    shutil.copy(os.path.join(B.HERE, "build.py"), pkg / "build.py")
    shutil.copytree(os.path.join(B.ROOT, "include"), root / "include")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho built > "$2"\n')
    nvcc.chmod(0o755)
    run = WITHOUT_TORCH + f"sys.path.insert(0, {str(pkg)!r})\nimport build\nprint(build.build())\n"
    out = subprocess.run([sys.executable, "-c", run], env={**os.environ, "NVCC": str(nvcc)}, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.strip() == str(pkg / "libdsa.so") and (pkg / "libdsa.so").read_text() == "built\n"
    assert not (pkg / "_calls.so").exists()


@pytest.fixture
def calls(tmp_path, monkeypatch):
    so, stamp = tmp_path / "_calls.so", tmp_path / "_build" / "calls_torch.txt"
    monkeypatch.setattr(B, "CALLS", str(so))
    monkeypatch.setattr(B, "CALLS_TORCH", str(stamp))
    return so, stamp


def test_the_extension_is_stale_for_another_torch(calls, monkeypatch):
    so, stamp = calls
    assert B.calls_stale()
    so.write_text("x")
    assert B.calls_stale()                                         # nobody says which torch it is for
    stamp.parent.mkdir()
    stamp.write_text(B.torch_version())
    assert not B.calls_stale() and B.build_calls() == str(so)
    monkeypatch.setattr(B, "torch_version", lambda: "0.1")
    assert B.calls_stale()


def test_the_extension_is_stale_behind_its_sources(calls):
    so, stamp = calls
    so.write_text("x")
    stamp.parent.mkdir()
    stamp.write_text(B.torch_version())
    old = os.path.getmtime(os.path.join(B.CSRC, "calls.cpp")) - 10
    os.utime(so, (old, old))
    assert B.calls_stale()
