"""CPU test of the package without the binding's extension."""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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
