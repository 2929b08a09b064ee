"""The debug library on plans of expanded latent rows (tests/debug_expanded_cases.py, run in a
child process that loads libpa_gb300_debug.so)."""
import importlib.util
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_debug_library_cases():
    spec = importlib.util.spec_from_file_location(
        "pa_build_for_debug_expanded", os.path.join(ROOT, "paged_quantized_kv_gqa_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.build(debug=True).endswith("libpa_gb300_debug.so")
    env = dict(os.environ, PA_GB300_DEBUG="1")
    env.pop("PA_GB300_TRACE", None)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_expanded_cases.py")],
                       env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "all expanded cases passed" in r.stdout
