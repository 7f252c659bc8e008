"""The library is built without torch and before the binding, and the binding for the
interpreter and the torch at hand (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from bit_quantized_kv_store_gb300 import build as B
from tests.conftest import ROOT
from tests.test_abi import K  # noqa: F401


def test_the_library_builds_without_torch(K, tmp_path):
    (tmp_path / "torch.py").write_text("raise ImportError('no torch here')\n")
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bit_quantized_kv_store_gb300", "build.py")], env=env,
                       cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == B.LIB, r.stdout + r.stderr


def test_a_binding_that_fails_leaves_the_library(K, monkeypatch):
    """The library is linked (here again: its time is set back) before the failure is raised."""
    def fail():
        raise RuntimeError("no compiler for the binding")
    monkeypatch.setattr(B, "_build_calls", fail)
    os.utime(B.LIB, (1, 1))
    with pytest.raises(RuntimeError, match="no compiler"):
        B.build()
    assert os.path.getmtime(B.LIB) > 1


def test_the_binding_is_rebuilt_for_another_interpreter(K, monkeypatch):
    commands = []

    class Failed:
        returncode, stdout, stderr = 1, "", "not run"

    def run(cmd, **kw):
        commands.append(cmd)
        return Failed()

    monkeypatch.setattr(B.subprocess, "run", run)
    B._build_calls()
    assert commands == []                                   # made for this one
    monkeypatch.setattr(sys, "version", "another interpreter")
    with pytest.raises(RuntimeError):
        B._build_calls()
    assert len(commands) == 1 and os.path.exists(B.CALLS)
