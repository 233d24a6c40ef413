"""Calls of different sizes from two host threads at once, each on a pool and a
stream of its own: what one call asks of a kernel (its dynamic shared memory)
does not reach the other's launches.  The bindings release the interpreter's
lock while they are in the library, so the calls do overlap."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import make_decoder
from tests.test_evict_gpu import _check, _i32, _state

pytestmark = pytest.mark.gpu

CALLS = 1500


def at_once(calls):
    """Each of `calls` (of a stream) CALLS times in a thread and on a stream of its own."""
    streams = [torch.cuda.Stream() for _ in calls]
    errors, start = [], threading.Barrier(len(calls))
    torch.cuda.synchronize()

    def work(k):
        try:
            start.wait()
            for i in range(CALLS):
                calls[k](streams[k])
                if i % 100 == 99:
                    streams[k].synchronize()
        except Exception as e:  # reported below, on the main thread
            errors.append((k, i, e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


def test_evictions():
    sides = []
    for lens, cap in (([300], 512), ([9000], 40960)):
        w = W.small("threads", lens=lens, L=1, Hq=2, Hkv=1)
        sides.append((w, cap, *make_decoder(w, cap)))
    none = _i32([-1])
    before = [_state(s[2]) for s in sides]
    at_once([lambda st, s=s: s[2].evict(none, s[5], s[3], s[4], stream=st) for s in sides])
    for (w, cap, dec, sig, cnt, ctx), was in zip(sides, before):
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        now = _state(dec)
        assert all(np.array_equal(now[k], was[k]) for k in was)
        b = w.lens[0] // 3
        dec.evict(_i32([b]), ctx, sig, cnt, sinks=4)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        _check(dec, was, w, cap, [b], w.lens, sig, cnt, 4, 0, str(cap))
