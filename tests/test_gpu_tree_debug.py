"""The drafted-token calls under the bounds-checked build (compiled with
CSA2_DEBUG): no index that a kernel forms, tensor-memory columns among them,
leaves its buffer (tests/_debug_tree_run.py, run in a child process so that
this process keeps the normal library)."""
import importlib.util
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_drafted_calls_stay_in_bounds():
    spec = importlib.util.spec_from_file_location(
        "csa2_build", os.path.join(ROOT, "fp4_kv_cache_index_gb300", "_build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert b.build(debug=True).endswith("libcsa2_debug.so")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_debug_tree_run.py")],
                       env=dict(os.environ, CSA2_DEBUG="1"), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "all cases clean" in r.stdout
