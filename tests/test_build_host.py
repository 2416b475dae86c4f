"""The build's order and names, with a compiler that only makes its output
files: the C library does not depend on torch or on the host compiler's way
with torch's headers."""
import os
import subprocess
import sysconfig

import pytest

from dense_fp32_gemm_gb300 import build as B


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """A build into tmp_path; `fail`: command names that fail."""
    fail = []

    def run(cmd, **kw):
        if os.path.basename(cmd[0]) in fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no such option")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "nvcc", lambda: "/nowhere/bin/nvcc")
    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B.subprocess, "check_call", lambda cmd, **kw: run(cmd).check_returncode())
    monkeypatch.delenv("CXX", raising=False)
    return fail


def test_builds_both(fake, tmp_path):
    assert os.path.exists(B.build()) and os.path.exists(B.marshal_path())


def test_library_without_torch(fake, tmp_path, monkeypatch):
    def missing(name):
        raise B.importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(B.importlib.metadata, "version", missing)
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: None)
    assert os.path.exists(B.build())
    assert not [f for f in os.listdir(tmp_path) if f.startswith("_marshal")]


def test_library_where_the_marshalling_module_fails(fake, tmp_path):
    fake.append("g++")
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        B.build()
    assert os.path.exists(tmp_path / B.LIB_NAME)


def test_module_name_carries_pythons_abi():
    assert sysconfig.get_config_var("SOABI") in os.path.basename(B.marshal_path())
