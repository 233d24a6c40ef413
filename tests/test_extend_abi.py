"""CPU-side checks of the multi-token and page-operation entry points: invalid
arguments are refused synchronously (no kernel is launched), and the serial
restatement of the page operations keeps the invariants of a decode state."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from differentiated_kv_cache_dkv_gb300 import build as libbuild
from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.decode_helpers import HostDecode, check_state
from tests.page_ops_helpers import serial_defrag, serial_fork, serial_release

BAD = libdkv.DKV_E_INVAL


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return libdkv.load()


def _pool(**kw):
    p = dict(F=64, P=16, scheme=0, free_list=256, cursors=512, rev_unit=1024, rev_idx=2048, page_cls=4096,
             pages=8192, status=16384)
    p.update(kw)
    return libdkv.dkv_pool(**p)


TAB = libdkv.dkv_tables(256, 6, 0, 512)


def _ebatch(**kw):
    b = dict(L=2, R=3, Hq=8, Hkv=2, cap=64, layer0=0, n_layers=2, max_new=8, T=20, q=256, k_new=512, v_new=1024,
             new_lens=2048, ctx_lens=4096, scale=0.088, out=8192, lse=16384)
    b.update(kw)
    return libdkv.dkv_extend_batch(**b)


SHARED = [dict(Hq=7), dict(L=0), dict(R=-1), dict(R=70000), dict(Hq=256, Hkv=2), dict(layer0=1), dict(n_layers=-1),
          dict(cap=0), dict(max_new=-1), dict(T=-1), dict(T=1 << 31), dict(q=None), dict(q=264), dict(k_new=None),
          dict(v_new=None), dict(k_new=520), dict(v_new=1032), dict(new_lens=None), dict(ctx_lens=4098),
          dict(scale=float("nan")), dict(lse=16386)]


def test_extend_rejects_bad_arguments(lib):
    n = ctypes.c_size_t(0)
    size = lambda b, p, t: lib.dkv_extend_workspace_size(ctypes.byref(b), ctypes.byref(p), ctypes.byref(t),  # noqa: E731
                                                         ctypes.byref(n))
    assert size(_ebatch(), _pool(), TAB) == libdkv.DKV_OK
    need = n.value

    def attend(b=None, p=None, t=None, ws=1 << 20, wsb=1 << 40):
        return lib.dkv_extend_attention(ctypes.byref(b or _ebatch()), ctypes.byref(p or _pool()),
                                        ctypes.byref(t or TAB), ws, wsb, None)

    def sig(b=None, acc=256, s=512):
        return lib.dkv_extend_significance(ctypes.byref(b or _ebatch()), acc, s, ctypes.byref(_pool()),
                                           ctypes.byref(TAB), None)

    for bad in SHARED:
        assert attend(_ebatch(**bad)) == BAD, bad
        assert sig(_ebatch(**bad)) == BAD, bad
        assert size(_ebatch(**bad), _pool(), TAB) == BAD, bad
    for bad in (dict(out=None), dict(out=8200)):
        assert attend(_ebatch(**bad)) == BAD, bad
    assert attend(p=_pool(P=15)) == BAD and attend(t=libdkv.dkv_tables(256, 1, 0, 512)) == BAD
    assert attend(t=libdkv.dkv_tables(256, 6, 0, 520)) == BAD
    if need:
        assert attend(ws=None) == BAD and attend(ws=(1 << 20) + 16) == BAD and attend(wsb=need - 1) == BAD
    assert sig(_ebatch(lse=None)) == BAD and sig(acc=None) == BAD and sig(s=None) == BAD and sig(s=520) == BAD
    # nothing to do: accepted without a launch, whatever the pointers
    assert attend(_ebatch(T=0, q=None, out=None)) == libdkv.DKV_OK
    assert attend(_ebatch(n_layers=0)) == libdkv.DKV_OK
    assert sig(_ebatch(T=0, q=None, lse=None)) == libdkv.DKV_OK


def _fbatch(**kw):
    b = dict(L=2, R=3, Hq=8, Hkv=2, cap=64, n=1, unit_base=0, src=256, dst=512, ctx_lens=1024, classes=2048,
             slot_of=4096, sig_sum=8192, sig_cnt=16384)
    b.update(kw)
    return libdkv.dkv_fork_batch(**b)


def _rbatch(**kw):
    b = dict(L=2, R=3, Hkv=2, n=1, unit_base=0, reqs=256)
    b.update(kw)
    return libdkv.dkv_release_batch(**b)


def test_page_operations_reject_bad_arguments(lib):
    n = ctypes.c_size_t(0)
    assert lib.dkv_page_ops_workspace_size(ctypes.byref(_pool()), 12, ctypes.byref(n)) == libdkv.DKV_OK
    need = n.value
    assert need > 0
    for p, u in ((_pool(P=3), 12), (_pool(), 0), (_pool(), 1 << 31)):
        assert lib.dkv_page_ops_workspace_size(ctypes.byref(p), u, ctypes.byref(n)) == BAD

    def fork(b=None, p=None, t=None, ws=1 << 20, wsb=need):
        return lib.dkv_fork(ctypes.byref(b or _fbatch()), ctypes.byref(p or _pool()), ctypes.byref(t or TAB), ws, wsb,
                            None)

    def release(b=None, p=None, t=None, ws=1 << 20, wsb=need):
        return lib.dkv_release(ctypes.byref(b or _rbatch()), ctypes.byref(p or _pool()), ctypes.byref(t or TAB), ws,
                               wsb, None)

    def defrag(p=None, t=None, U=12, base=0, ws=1 << 20, wsb=need):
        return lib.dkv_defrag(ctypes.byref(p or _pool()), ctypes.byref(t or TAB), U, base, ws, wsb, None)

    for call in (fork, release, defrag):
        assert call(ws=None) == BAD and call(ws=(1 << 20) + 64) == BAD and call(wsb=need - 1) == BAD
        assert call(p=_pool(P=7)) == BAD and call(p=_pool(status=None)) == BAD
        assert call(t=libdkv.dkv_tables(None, 6, 0, 512)) == BAD and call(t=libdkv.dkv_tables(256, 6, 0, 516)) == BAD
    for bad in (dict(L=0), dict(R=0), dict(R=65536), dict(Hkv=0), dict(n=-1), dict(n=4), dict(unit_base=-1),
                dict(unit_base=2147483640)):
        assert fork(_fbatch(**bad)) == BAD and release(_rbatch(**bad)) == BAD, bad
    for bad in (dict(src=None), dict(dst=514), dict(ctx_lens=None), dict(cap=60), dict(cap=0), dict(classes=2049),
                dict(slot_of=4100), dict(sig_sum=8196), dict(sig_cnt=16388), dict(Hq=0),
                dict(classes=None, slot_of=None, sig_sum=None, sig_cnt=None)):
        assert fork(_fbatch(**bad)) == BAD, bad
    assert release(_rbatch(reqs=None)) == BAD and release(_rbatch(reqs=257)) == BAD
    assert defrag(U=0) == BAD and defrag(U=1 << 31) == BAD and defrag(base=-1) == BAD
    assert fork(_fbatch(n=0)) == libdkv.DKV_OK and release(_rbatch(n=0)) == libdkv.DKV_OK


def test_adopted_tensors_are_checked(lib):
    import torch
    F, P = 8, 4
    t = dict(free_list=torch.zeros(F, dtype=torch.int32), cursors=torch.zeros(2, dtype=torch.int64),
             rev_unit=torch.zeros(F, dtype=torch.int32), rev_idx=torch.zeros(F, dtype=torch.int32),
             page_cls=torch.zeros(F, dtype=torch.uint8),
             pages=torch.zeros((F, libdkv.dkv_page_bytes(0, P)), dtype=torch.uint8),
             status=torch.zeros(1, dtype=torch.int32))
    assert libdkv.DevicePool.from_tensors(P, 0, **t).F == F
    for name, x in (("pages", t["pages"][:, 8:]), ("cursors", t["cursors"].int()), ("rev_unit", t["rev_unit"][1:])):
        with pytest.raises(ValueError):
            libdkv.DevicePool.from_tensors(P, 0, **{**t, name: x})
    fwd, hdr = torch.zeros((6, 5), dtype=torch.int32), torch.zeros((6, 4), dtype=torch.int32)
    assert libdkv.DeviceTables.from_tensors(fwd, hdr).pmax == 5
    for a, b in ((fwd.long(), hdr), (fwd, hdr[1:]), (fwd[:, 1:], hdr)):
        with pytest.raises(ValueError):
            libdkv.DeviceTables.from_tensors(a, b)


def test_serial_page_operations_keep_a_decode_state_valid():
    """The tests' restatement on the oracle's own prefill: the invariants of
    every decode state hold after each operation."""
    w = W.small("ops_pin", lens=[100, 0, 61, 17], L=2, Hq=4, Hkv=2, P=8)
    cap = 112
    hd = HostDecode(w, cap, F=400, inp=W.make_inputs(w, 5))
    st = {"free_list": hd.pool.free_list.copy(), "cursors": hd.pool.cursors.astype(np.int64),
          "rev_unit": hd.pool.rev_unit.copy(), "rev_idx": hd.pool.rev_idx.copy(),
          "page_cls": hd.pool.page_cls.copy(), "pages": hd.pool.pages.copy(), "fwd": hd.tab.fwd.copy(),
          "unit_hdr": hd.tab.unit_hdr.copy()}
    cls = hd.classes.reshape(w.L, w.R * cap, w.Hkv).copy()
    lens = np.array(w.lens)

    def check():
        class Pool:
            pass
        p = Pool()
        p.P, p.F, p.scheme = w.P, 400, 0
        for k in ("free_list", "rev_unit", "rev_idx", "page_cls", "pages"):
            setattr(p, k, st[k])
        p.cursors = st["cursors"].astype(np.uint64)
        check_state(w, cap, p, st["fwd"], st["unit_hdr"], cls, lens)

    check()
    st = serial_fork(st, w.L, w.R, w.Hkv, [0], [1])
    cls[:, cap:2 * cap] = cls[:, :cap]
    lens[1] = lens[0]
    check()
    st = serial_release(st, w.L, w.R, w.Hkv, [0, 3])
    lens[[0, 3]] = 0
    check()
    st = serial_defrag(st)
    check()
    n = 400 - int(st["cursors"][1] - st["cursors"][0])
    assert (st["page_cls"][:n] != 0).all() and not st["page_cls"][n:].any()
