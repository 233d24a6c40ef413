"""Host arithmetic of the chunk and eviction entry points: sizes at the edge of
what is counted in 32 bits, and the entry points' argument tests under
AddressSanitizer and UndefinedBehaviorSanitizer."""
from __future__ import annotations

import ctypes
import os

import pytest

from differentiated_kv_cache_dkv_gb300 import build as libbuild
from differentiated_kv_cache_dkv_gb300 import libdkv
from tests.test_chunk_abi import _cbatch, _pages, _pool
from tests.test_sanitizers import _asan_runtime, _run, _sanitized

BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return libdkv.load()


@pytest.mark.parametrize("kw, pg", [(dict(L=65535, n_layers=65535, R=65535, Hkv=1, Hq=128, T=BIG, max_new=BIG, cap=BIG), {}),
                                    (dict(L=1, n_layers=1, R=1, Hkv=1, Hq=128, T=BIG, max_new=BIG, cap=BIG), {}),
                                    (dict(L=2, n_layers=2, R=1, Hkv=1, Hq=1, T=BIG, max_new=4, cap=64), {}),
                                    (dict(L=1, layer0=1, n_layers=BIG), {}), (dict(L=65535, layer0=BIG, n_layers=BIG), {}),
                                    (dict(R=65535, cap=BIG), dict(B=128, tmax=1 << 24)),
                                    # 2^15 / 256 items of up to 2^24 key tiles
                                    (dict(L=1, n_layers=1, R=1, Hq=1, Hkv=1, cap=BIG, max_new=BIG, T=1 << 15), dict(B=128, tmax=1 << 24)),
                                    (dict(), dict(F=BIG, B=128)), (dict(), dict(tmax=BIG, B=128, F=BIG))])
def test_sizes_that_are_refused(lib, kw, pg):
    n = ctypes.c_size_t(0)
    args = [ctypes.byref(x) for x in (_cbatch(**kw), _pages(**pg))]
    assert lib.dkv_chunk_workspace_size(*args, ctypes.byref(n)) == libdkv.DKV_E_INVAL
    pool = ctypes.byref(_pool())
    assert lib.dkv_chunk_attention(*args, pool, 1 << 20, 1 << 62, None) == libdkv.DKV_E_INVAL
    assert lib.dkv_chunk_significance(*args, 512, pool, None) == libdkv.DKV_E_INVAL


@pytest.mark.parametrize("kw", [dict(), dict(L=1, n_layers=1, R=1, Hq=1, Hkv=1, cap=BIG, max_new=BIG, T=1 << 14),
                                dict(L=64, n_layers=32, R=512, Hq=128, Hkv=8, cap=1 << 17, max_new=1 << 13, T=1 << 20)])
def test_sizes_grow_with_the_tokens(lib, kw):
    n, last = ctypes.c_size_t(0), -1
    full = _cbatch(**kw).T
    pages = _pages(F=1024, B=128, tmax=max(4, -(-_cbatch(**kw).cap // 128)))
    for T in (1, full // 2 + 1, full):
        assert lib.dkv_chunk_workspace_size(ctypes.byref(_cbatch(**{**kw, "T": T})), ctypes.byref(pages),
                                            ctypes.byref(n)) == libdkv.DKV_OK
        assert n.value >= last
        last = n.value


def test_eviction_sizes(lib):
    n = ctypes.c_size_t(0)
    tab = libdkv.dkv_tables(256, 6, 0, 512)

    def size(**kw):
        b = dict(L=2, R=3, Hq=8, Hkv=2, cap=64, sinks=0, window=0, reserved=0, unit_base=0, budgets=256, ctx_lens=512,
                 sig_sum=1024, sig_cnt=2048, classes=4096, slot_of=8192)
        b.update(kw)
        rc = lib.dkv_evict_workspace_size(ctypes.byref(libdkv.dkv_evict_batch(**b)), ctypes.byref(_pool()), ctypes.byref(tab),
                                          ctypes.byref(n))
        return rc, n.value

    # the most units, the most positions: more than 2^32 bytes of each list, counted in 64 bits
    rc, most = size(L=32767, R=65535, Hq=1, Hkv=1, cap=1 << 18)
    assert rc == libdkv.DKV_OK and most > 32767 * 65535 * (4 << 18)
    assert size(L=BIG, R=1, Hq=1, Hkv=1)[0] == libdkv.DKV_OK
    for kw in (dict(L=BIG, R=2, Hq=1, Hkv=1), dict(L=BIG, R=1, Hq=2, Hkv=2), dict(L=BIG, R=1, Hq=1, Hkv=1, unit_base=1),
               dict(cap=BIG), dict(sinks=-BIG - 1), dict(window=-BIG - 1)):
        assert size(**kw)[0] == libdkv.DKV_E_INVAL, kw
    assert size(sinks=BIG, window=BIG)[0] == libdkv.DKV_OK


@pytest.mark.skipif(os.environ.get("DKV_LIBRARY") == "sanitized", reason="this is the child")
def test_entry_points_under_sanitizers():
    _asan_runtime()
    assert _sanitized(libbuild.build(sanitize=True))
    assert "passed" in _run(["tests/test_chunk_abi.py", "tests/test_chunk_sizes.py", "tests/test_batches.py"],
                            DKV_LIBRARY="sanitized")
