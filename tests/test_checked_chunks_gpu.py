"""The chunk's attention, its significance and the eviction under the
bounds-checked build: their tests pass and no index check fires (a check that
fires reports DKV_E_INTERNAL, which every test reads)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "differentiated_kv_cache_dkv_gb300", "csrc")
TESTS = ["tests/test_chunk_gpu.py", "tests/test_chunk_segments_gpu.py", "tests/test_evict_gpu.py",
         "tests/test_evict_long_lists_gpu.py", "tests/test_chunk_weights_gpu.py"]


@pytest.mark.parametrize("name", ["chunk.cu", "chunk_sig.cu", "evict.cu"])
def test_the_kernels_check_their_indices(name):
    with open(os.path.join(CSRC, name)) as f:
        assert "in_range(" in f.read()


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
