"""The multi-token calls and the page operations under the bounds-checked build:
their tests pass and no index check fires (a check that fires reports
DKV_E_INTERNAL, which every test reads)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = ["tests/test_extend_gpu.py", "tests/test_extend_routes_gpu.py", "tests/test_extend_contracts_gpu.py",
         "tests/test_extend_parts_gpu.py", "tests/test_extend_references_gpu.py", "tests/test_extend_range_gpu.py",
         "tests/test_page_ops_gpu.py"]


@pytest.mark.gpu
def test_operators_under_the_checked_build():
    from differentiated_kv_cache_dkv_gb300 import build

    build.build(checked=True)
    code = (
        "import sys, pytest\n"
        "from differentiated_kv_cache_dkv_gb300 import libdkv\n"
        "assert libdkv.load().dkv_build_flags() & 1 == 1\n"
        f"sys.exit(pytest.main({TESTS!r} + ['-q', '-x', '-m', 'gpu', '-p', 'no:cacheprovider']))\n"
    )
    env = dict(os.environ, DKV_LIBRARY="checked")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert "passed" in r.stdout
