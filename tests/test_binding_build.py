"""The compiled binding module against the torch and Python that it was built for (no GPU, no compiler needed)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "compressed_sparse_long_v4a_b200"


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build script with its outputs in tmp_path and a compiler that only counts its calls."""
    import compressed_sparse_long_v4a_b200.build as b

    calls = []

    class Done:
        returncode, stderr = 0, ""

    def run(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "objects"))
    monkeypatch.setattr(b.subprocess, "run", run)
    return b, calls


def test_binding_is_built_once_for_a_torch(build):
    b, calls = build
    assert b.build_binding() == b.BINDING and len(calls) == 1
    b.build_binding()
    assert len(calls) == 1
    assert any(b.binding_tag() in x for x in calls[0])


def test_binding_is_built_again_for_another_torch(build, monkeypatch):
    import torch

    b, calls = build
    b.build_binding()
    monkeypatch.setattr(torch, "__version__", "9.9")
    b.build_binding()
    b.build_binding()
    assert len(calls) == 2 and any("torch 9.9 " in x for x in calls[1])


def test_binding_of_unknown_origin_is_built_again(build):
    b, calls = build
    open(b.BINDING, "w").close()  # newer than its sources
    b.build_binding()
    assert len(calls) == 1


def test_a_failed_build_is_tried_again(build, monkeypatch):
    b, calls = build
    b.build_binding()
    os.utime(b.BINDING, (0, 0))

    class Failed:
        returncode, stderr = 1, "no"

    with monkeypatch.context() as m:
        m.setattr(b.subprocess, "run", lambda cmd, **kw: Failed())
        with pytest.raises(RuntimeError, match="no"):
            b.build_binding()
    b.build_binding()
    assert len(calls) == 2


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_binding_built_for_another_torch_is_not_used():
    r = python(f"import torch; torch.__version__ = '9.9'; import {PACKAGE}")
    assert r.returncode != 0 and "built for torch" in r.stderr and "__graft_entry__.build()" in r.stderr
