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


def python(code, cwd=ROOT):
    r = subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


# every call that goes through the binding; nothing of them is reached
SERVING = f"""
import torch
{{before}}
import {PACKAGE} as v4a
assert v4a.v4a_version() > 0 and v4a.v4a_workspace_size("topk", batch=1, m=4, k=8, ctx_len=64, heads_i=1, d_i=8) > 0
assert v4a.v4a_shared_workspace_size(batch=1, heads=64, d=512, n_prefix=5, own_rows=0) > 0
x = torch.zeros((1, 1, 1, 64))
for call in (lambda: v4a.v4a_rope([(x, x)], rope_dims=64),
             lambda: v4a.v4a_hca_attend_shared(x, None, None, None, x, m=1, window=0, ctx_len=1),
             lambda: v4a.v4a_attend_weights(x, x[0], x, x, x, m=1, ctx_len=1),
             lambda: v4a.v4a_evict(x[0], x, x, x, x, x, budget=1)):
    try:
        call()
    except ImportError as e:
        print(e)
"""


def test_binding_built_for_another_torch_is_not_used():
    said = python(SERVING.format(before="torch.__version__ = '9.9'")).splitlines()
    assert len(said) == 4 and all("was built for torch" in x and "this is torch 9.9 " in x and "__graft_entry__.build()" in x for x in said)


def test_without_the_binding_only_the_serving_calls_fail(tmp_path):
    src, dst = os.path.join(ROOT, PACKAGE), tmp_path / PACKAGE
    dst.mkdir()
    for name in ("__init__.py", "build.py", "libv4a.so"):
        os.symlink(os.path.join(src, name), dst / name)
    said = python(SERVING.format(before=""), tmp_path).splitlines()
    assert len(said) == 4 and all("not built" in x and "__graft_entry__.build()" in x for x in said)
