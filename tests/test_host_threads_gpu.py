"""Calls of different sizes from two host threads at once, each on a pool and a
stream of its own: what one call asks of a kernel (its dynamic shared memory)
does not reach the other's launches.  The bindings release the interpreter's
lock while they are in the library, so the calls do overlap."""
from __future__ import annotations

import ctypes
import threading

import numpy as np
import pytest
import torch

import oracle
from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, make_decoder
from tests.gpu_helpers import assert_same_state, fetch, make_compactor, oracle_state, to_device
from tests.oracle_helpers import run_oracle
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


def _raw(fn, *args):
    """The library's function over these structures, of a stream: little time outside it, so that calls meet."""
    refs = [ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in args]

    def call(st):
        rc = fn(*refs, st.cuda_stream)
        if rc != libdkv.DKV_OK:
            raise libdkv.DkvError(rc, fn.__name__)

    return call


def test_evictions():
    sides, calls, none = [], [], _i32([-1])
    for lens, cap in (([300], 512), ([9000], 40960)) * 3:
        w = W.small("threads", lens=lens, L=1, Hq=2, Hkv=1)
        dec, sig, cnt, ctx = make_decoder(w, cap)
        batch = libdkv.make_evict_batch(1, 1, 2, 1, cap, none, ctx, sig, dec.classes, dec.slot_of, cnt)
        ws = torch.empty(libdkv.dkv_evict_workspace_size(batch, dec.pool, dec.tables), dtype=torch.uint8, device="cuda")
        calls.append(_raw(libdkv.load().dkv_evict, batch, dec.pool.c(), dec.tables.c(), ws.data_ptr(), ws.numel()))
        sides.append((w, cap, dec, sig, cnt, ctx, ws, _state(dec)))
    at_once(calls)
    for w, cap, dec, sig, cnt, ctx, _, was in sides:
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        now = _state(dec)
        assert all(np.array_equal(now[k], was[k]) for k in was)
        b = w.lens[0] // 3
        dec.evict(_i32([b]), ctx, sig, cnt, sinks=4)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        _check(dec, was, w, cap, [b], w.lens, sig, cnt, 4, 0, str(cap))


def _check_attention():
    w = W.small("threads", lens=[100], L=1, Hq=8, Hkv=2)
    q = torch.randn((1, 1, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    calls, outs = [], []
    for cap in (1024, 6144) * 3:  # about 77 and 86 KB a block
        dec, _, _, ctx = make_decoder(w, cap)
        out = torch.empty((1, 1, 8, 128), device="cuda")
        b = libdkv.dkv_attn_batch(1, 1, 8, 2, cap, 0, 1, q.data_ptr(), None, None, None, ctx.data_ptr(), SCALE,
                                  out.data_ptr(), None)
        calls.append(_raw(libdkv.load().dkv_decode_attention, b, dec.pool.c(), dec.tables.c()))
        outs.append((dec, ctx, out))
    at_once(calls)
    for dec, ctx, out in outs:
        now = out.clone()
        dec.attend(q, ctx, out, SCALE)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK and torch.equal(out, now)


def _check_compaction():
    sides, calls, lib = [], [], libdkv.load()
    for Hq in (128, 104) * 3:  # no per-token kernel for either: 67 and 54 KB a block
        w = W.small("threads", lens=[100, 300], L=1, Hq=Hq, Hkv=8)
        inp = W.make_inputs(w)
        comp, dev = make_compactor(w), to_device(inp)
        init = _raw(lib.dkv_init_pool, comp.pool.c())
        compact = _raw(lib.dkv_compact, comp.batch(dev), libdkv.dkv_params(w.alpha_h, w.alpha_l, -1, 0, None), comp.pool.c(),
                       comp.tables.c(), comp.workspace.data_ptr(), comp.workspace.numel())
        calls.append(lambda st, init=init, compact=compact: (init(st), compact(st)))
        sides.append((w, inp, dev, comp))
    at_once(calls)
    for w, inp, _, comp in sides:
        assert libdkv.dkv_get_status(comp.pool) == libdkv.DKV_OK
        so, pool, tab = run_oracle(w, W.to_numpy(inp), w.alpha_h, w.alpha_l, pool=oracle.Pool(comp.pool.F, w.P))
        assert so == oracle.OK
        assert_same_state(fetch(comp), oracle_state(pool, tab))


def _check_steps():
    sides, calls = [], []
    for cap in (8192, 16384) * 3:  # 51 and 92 KB a block
        w = W.small("threads", lens=[100], L=1, Hq=8, Hkv=8)
        dec, sig, cnt, ctx = make_decoder(w, cap)
        new = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
        d = {"k_new": new, "v_new": new, "sig_sum": sig, "sig_cnt": cnt, "ctx_lens": ctx, "new_lens": _i32([0])}
        # thresholds of 0 leave every class as it is
        calls.append(_raw(libdkv.load().dkv_decode_step, dec.batch(d), libdkv.dkv_params(0.0, 0.0, -1, 0, None), dec.pool.c(),
                          dec.tables.c(), dec.workspace.data_ptr(), dec.workspace.numel()))
        sides.append((dec, d, _state(dec)))
    at_once(calls)
    for dec, _, was in sides:
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        now = _state(dec)
        assert all(np.array_equal(now[k], was[k]) for k in was)


@pytest.mark.parametrize("check", [_check_attention, _check_compaction, _check_steps])
def test_other_calls_whose_shared_memory_depends_on_their_shape(check):
    check()
