"""The compiled part of the binding: the calls that do without it work without it, and one that was built for another
torch or Python is rebuilt, not loaded."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_230_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    build.build()
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout.split("\n")


def test_without_it_the_other_calls_work():
    out = run("""
from paged_kv_cache_230_gb300 import build
build.OPS = "/nonexistent/_pa_ops.so"
from paged_kv_cache_230_gb300 import pagedattn as pa
print(pa.status_string(0), pa.decode_split_workspace_size(1, 8, 128, 1000, 64) > 0)
try:
    pa.block_scores(None, None, None, None, None, 16)
except RuntimeError as e:
    print(e)
""")
    assert out[0].endswith("True") and "not built" in out[1]


def test_one_built_for_another_torch_is_not_loaded():
    out = run("""
from paged_kv_cache_230_gb300 import build
build.binding_target = lambda: "torch 0.0, .so"
from paged_kv_cache_230_gb300 import pagedattn as pa
print(pa.status_string(0))
try:
    pa.block_scores(None, None, None, None, None, 16)
except RuntimeError as e:
    print(e)
""")
    assert "not for torch 0.0" in out[1]


def test_it_is_loaded_once():
    out = run("""
from paged_kv_cache_230_gb300 import pagedattn as pa
for _ in range(2):
    try:
        pa.block_scores(None, None, None, None, None, 16)
    except ValueError as e:
        print(e, type(pa._ops).__name__)
""")
    assert out[0].endswith("module") and out[0] == out[1]


def test_one_built_for_another_torch_is_rebuilt(monkeypatch):
    build.build()
    assert build.binding_fresh()
    made = []
    monkeypatch.setattr(build, "_compile_binding", lambda: made.append("compiled") or "obj")
    monkeypatch.setattr(build, "_link_binding", lambda obj: made.append(obj))
    before = os.path.getmtime(build.LIB)
    build.build()
    assert made == []
    monkeypatch.setattr(build, "binding_target", lambda: "torch 0.0, .so")
    build.build()
    assert made == ["compiled", "obj"] and os.path.getmtime(build.LIB) == before


@pytest.mark.parametrize("missing", ["OPS", "OPS_FOR"])
def test_a_missing_one_is_rebuilt(monkeypatch, tmp_path, missing):
    build.build()
    made = []
    monkeypatch.setattr(build, "_compile_binding", lambda: "obj")
    monkeypatch.setattr(build, "_link_binding", made.append)
    monkeypatch.setattr(build, missing, str(tmp_path / "none"))
    build.build()
    assert made == ["obj"]
