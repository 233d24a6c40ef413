"""Host arithmetic of the multi-token and page-operation entry points: sizes
that no memory holds are refused instead of overflowing, and the entry points'
argument tests pass under AddressSanitizer and UndefinedBehaviorSanitizer."""
from __future__ import annotations

import ctypes
import os

import pytest

from differentiated_kv_cache_dkv_gb300 import build as libbuild
from differentiated_kv_cache_dkv_gb300 import libdkv
from tests.test_extend_abi import TAB, _ebatch, _pool
from tests.test_sanitizers import _asan_runtime, _run, _sanitized

BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return libdkv.load()


@pytest.mark.parametrize("kw", [dict(L=BIG, n_layers=BIG, R=1, Hkv=1, Hq=128, T=BIG, max_new=BIG, cap=BIG),
                                dict(L=BIG, n_layers=BIG, R=1, Hkv=1, Hq=1, T=BIG, max_new=4, cap=BIG),
                                dict(L=8, n_layers=8, R=1, Hkv=1, Hq=8, T=BIG, max_new=BIG, cap=BIG)])
def test_rows_that_no_memory_holds(lib, kw):
    n = ctypes.c_size_t(0)
    args = [ctypes.byref(x) for x in (_ebatch(**kw), _pool(), TAB)]
    assert lib.dkv_extend_workspace_size(*args, ctypes.byref(n)) == libdkv.DKV_E_INVAL
    assert lib.dkv_extend_attention(*args, 1 << 20, 1 << 62, None) == libdkv.DKV_E_INVAL
    assert lib.dkv_extend_significance(args[0], 256, 512, args[1], args[2], None) == libdkv.DKV_E_INVAL


@pytest.mark.parametrize("kw", [dict(), dict(L=64, n_layers=64, R=512, Hkv=8, Hq=64, T=1 << 22, max_new=1 << 13, cap=1 << 20),
                                dict(max_new=BIG, cap=BIG), dict(max_new=1, T=3, cap=BIG)])
def test_sizes_grow_with_the_tokens(lib, kw):
    n, last = ctypes.c_size_t(0), -1
    full = _ebatch(**kw).T
    for T in (1, full // 2 + 1, full):
        args = [ctypes.byref(x) for x in (_ebatch(**{**kw, "T": T}), _pool(), TAB)]
        assert lib.dkv_extend_workspace_size(*args, ctypes.byref(n)) == libdkv.DKV_OK
        assert n.value >= last
        last = n.value


@pytest.mark.skipif(os.environ.get("DKV_LIBRARY") == "sanitized", reason="this is the child")
def test_entry_points_under_sanitizers():
    _asan_runtime()
    assert _sanitized(libbuild.build(sanitize=True))
    assert "passed" in _run(["tests/test_extend_abi.py", "tests/test_extend_lists.py", "tests/test_extend_sizes.py"],
                            DKV_LIBRARY="sanitized")
