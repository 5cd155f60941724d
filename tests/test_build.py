"""The build's own logic (CPU, the compilers replaced by a fake): the library does
not depend on torch, and _host.so follows the torch that is installed."""

import os
import subprocess
import sys

import pytest

from mxfp8_moe_decode_gb300 import build as B


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """Compilers that write their output file; `fail` names one that does not."""
    calls, fail = [], []

    def run(cmd, **kw):
        name = os.path.basename(cmd[0])
        calls.append((name, cmd))
        if name in fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "HOST", str(tmp_path / "host.so"))
    monkeypatch.setattr(B, "HOST_KEY", str(tmp_path / "host.key"), raising=False)
    monkeypatch.setattr(B, "nvcc", lambda: "/opt/cuda/bin/nvcc")
    return calls, fail


def _count(calls, name):
    return sum(n == name for n, _ in calls)


def test_library_is_linked_when_the_host_module_fails(fake):
    calls, fail = fake
    fail.append("g++")
    with pytest.raises(RuntimeError, match="host.cpp"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.HOST)
    # what is missing is tried again, the library is not
    n = _count(calls, "nvcc")
    fail.clear()
    B.build()
    assert os.path.exists(B.HOST) and _count(calls, "nvcc") == n


def test_library_is_built_without_torch(fake, monkeypatch):
    calls, _ = fake
    monkeypatch.setitem(sys.modules, "torch", None)
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert _count(calls, "g++") == 0
    n = len(calls)
    B.build()
    assert len(calls) == n


def test_host_module_follows_torch(fake, monkeypatch):
    calls, _ = fake
    B.build()
    n = len(calls)
    B.build()
    assert len(calls) == n and _count(calls, "g++") == 1
    monkeypatch.setattr(B, "_host_key", lambda: "another torch")
    B.build()
    assert _count(calls, "g++") == 2 and len(calls) == n + 1
    B.build()
    assert _count(calls, "g++") == 2


def test_failed_link_leaves_the_old_library(fake):
    _, fail = fake
    B.build()
    with open(B.LIB, "w") as f:
        f.write("old")
    fail.append("nvcc")
    with pytest.raises(RuntimeError):
        B.build(force=True)
    with open(B.LIB) as f:
        assert f.read() == "old"
