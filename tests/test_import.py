"""CPU tests of the package without the binding's extension, and of what its
build holds to be up to date."""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build_module():
    spec = importlib.util.spec_from_file_location("_kvq_build_test", os.path.join(ROOT, "sm_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_contiguous_calls_need_no_extension(tmp_path):
    """Without _calls.so the package imports, and only the paged calls refuse."""
    pkg = tmp_path / "sm_b200"
    pkg.mkdir()
    for f in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(ROOT, "sm_b200", f), pkg / f)
    os.symlink(os.path.join(ROOT, "sm_b200", "libkvq.so"), pkg / "libkvq.so")
    code = """
import types, torch, sm_b200 as K
cache = types.SimpleNamespace(_address=0, _index=0)
assert K.cache_sizes(1, 1, 32, 64, 4, 32)[0] == 1024
assert K.lib.kvq_strerror(0)
for call in (lambda: K.qk_norm_rope(torch.zeros(2, 4, 64), None, None, None),
             lambda: K.paged_append(None, None, cache, None, None, None, 1)):
    try:
        call()
    except ImportError as e:
        assert "_calls.so" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("a paged call without its extension")
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr


def test_extension_of_another_torch_is_stale(tmp_path, monkeypatch):
    """File times do not tell: a torch installed anew brings other libraries."""
    b = build_module()
    so = tmp_path / "_calls.so"
    monkeypatch.setattr(b, "CALLS", str(so))
    monkeypatch.setattr(b, "CALLS_STAMP", str(tmp_path / "calls.stamp"))
    assert not b.calls_up_to_date()
    so.write_bytes(b"")
    assert not b.calls_up_to_date()                  # built by something that left no stamp
    b.stamp_calls()
    assert b.calls_up_to_date()
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert not b.calls_up_to_date()
    monkeypatch.undo()
    monkeypatch.setattr(b, "CALLS", str(so))
    monkeypatch.setattr(b, "CALLS_STAMP", str(tmp_path / "calls.stamp"))
    assert b.calls_up_to_date()
    os.utime(so, (0, 0))
    assert not b.calls_up_to_date()
