"""CPU-side checks of the chunk and eviction entry points: invalid arguments
are refused synchronously (no kernel is launched), and the serial restatement
of the eviction keeps the invariants of a decode state."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import build as libbuild
from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.chunk_helpers import serial_evict
from tests.decode_helpers import HostDecode, check_state

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


def _pages(**kw):
    p = dict(F=64, B=16, tmax=4, k=256, v=512, table=1024)
    p.update(kw)
    return libdkv.dkv_chunk_pages(**p)


def _cbatch(**kw):
    b = dict(L=2, R=3, Hq=8, Hkv=2, cap=64, layer0=0, n_layers=2, max_new=8, T=20, q_stride=0, kv_stride=0, q=256,
             k_new=512, v_new=1024, new_lens=2048, ctx_lens=4096, scale=0.088, out=8192, lse=16384)
    b.update(kw)
    return libdkv.dkv_chunk_batch(**b)


def test_chunk_calls_reject_bad_arguments(lib):
    n = ctypes.c_size_t(0)
    ref = ctypes.byref

    def size(b=None, g=None):
        return lib.dkv_chunk_workspace_size(ref(b or _cbatch()), ref(g or _pages()), ref(n))

    assert size() == libdkv.DKV_OK and n.value > 0
    need = n.value

    def attend(b=None, g=None, p=None, ws=1 << 20, wsb=1 << 40):
        return lib.dkv_chunk_attention(ref(b or _cbatch()), ref(g or _pages()), ref(p or _pool()), ws, wsb, None)

    def sig(b=None, g=None, s=512, p=None):
        return lib.dkv_chunk_significance(ref(b or _cbatch()), ref(g or _pages()), s, ref(p or _pool()), None)

    for bad in (dict(Hq=7), dict(L=0), dict(R=-1), dict(R=70000), dict(Hq=256, Hkv=2), dict(layer0=1),
                dict(n_layers=-1), dict(cap=0), dict(cap=65), dict(max_new=-1), dict(T=-1), dict(T=1 << 31),
                dict(q=None), dict(q=264), dict(k_new=None), dict(v_new=None), dict(k_new=520), dict(v_new=1032),
                dict(new_lens=None), dict(ctx_lens=4098), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(scale=0.0), dict(scale=-1.0), dict(lse=16386), dict(q_stride=1023), dict(q_stride=1016),
                dict(q_stride=-8), dict(kv_stride=248), dict(kv_stride=260), dict(kv_stride=1 << 40)):
        assert attend(_cbatch(**bad)) == BAD and sig(_cbatch(**bad)) == BAD and size(_cbatch(**bad)) == BAD, bad
    for bad in (dict(F=0), dict(F=1 << 31), dict(F=1 << 30), dict(B=4), dict(B=24), dict(B=256), dict(tmax=3),
                dict(k=None), dict(v=None), dict(table=None), dict(k=264), dict(v=520), dict(table=1026)):
        assert attend(g=_pages(**bad)) == BAD and sig(g=_pages(**bad)) == BAD and size(g=_pages(**bad)) == BAD, bad
    for bad in (dict(out=None), dict(out=8200)):
        assert attend(_cbatch(**bad)) == BAD, bad
    assert attend(ws=None) == BAD and attend(ws=(1 << 20) + 16) == BAD and attend(wsb=need - 1) == BAD
    assert attend(p=_pool(status=None)) == BAD and sig(p=_pool(status=None)) == BAD
    assert sig(_cbatch(lse=None)) == BAD and sig(s=None) == BAD and sig(s=520) == BAD
    # nothing to do: accepted without a launch, whatever the pointers
    assert attend(_cbatch(T=0, q=None, out=None), ws=None) == libdkv.DKV_OK
    assert attend(_cbatch(n_layers=0)) == libdkv.DKV_OK and attend(_cbatch(R=0)) == libdkv.DKV_OK
    assert sig(_cbatch(T=0, q=None, lse=None)) == libdkv.DKV_OK


def test_a_chunk_whose_work_does_not_fit_32_bits_is_refused(lib):
    n = ctypes.c_size_t(0)
    g = _pages(F=1 << 20, B=16, tmax=1 << 20)
    for max_new, T, want in ((1 << 24, 1 << 24, BAD), (1 << 24, 1 << 14, libdkv.DKV_OK), (1 << 14, 1 << 24, libdkv.DKV_OK),
                             (1 << 15, 1 << 15, BAD)):
        # groups of 128: 2 tokens an item, each of up to 2^17 key tiles
        b = _cbatch(R=1, Hq=128, Hkv=1, cap=1 << 24, max_new=max_new, T=T)
        assert lib.dkv_chunk_workspace_size(ctypes.byref(b), ctypes.byref(g), ctypes.byref(n)) == want, (max_new, T)


def test_evict_rejects_bad_arguments(lib):
    tab = libdkv.dkv_tables(256, 6, 0, 512)
    n = ctypes.c_size_t(0)
    ref = ctypes.byref

    def batch(**kw):
        b = dict(L=2, R=3, Hq=8, Hkv=2, cap=64, sinks=0, window=0, reserved=0, unit_base=0, budgets=256, ctx_lens=512,
                 sig_sum=1024, sig_cnt=2048, classes=4096, slot_of=8192)
        b.update(kw)
        return libdkv.dkv_evict_batch(**b)

    def size(b=None, p=None, t=tab):
        return lib.dkv_evict_workspace_size(ref(b or batch()), ref(p or _pool()), ref(t), ref(n))

    assert size() == libdkv.DKV_OK
    need = n.value

    def evict(b=None, p=None, t=tab, ws=1 << 20, wsb=1 << 40):
        return lib.dkv_evict(ref(b or batch()), ref(p or _pool()), ref(t), ws, wsb, None)

    for bad in (dict(L=0), dict(R=0), dict(R=70000), dict(Hq=7), dict(Hkv=0), dict(cap=0), dict(cap=72),
                dict(cap=(1 << 18) + 16), dict(sinks=-1), dict(window=-1), dict(reserved=1), dict(unit_base=-1),
                dict(unit_base=2 ** 31 - 5)):
        assert evict(batch(**bad)) == BAD and size(batch(**bad)) == BAD, bad
    for bad in (dict(budgets=None), dict(ctx_lens=None), dict(sig_sum=None), dict(sig_sum=1032), dict(sig_cnt=2050),
                dict(classes=None), dict(slot_of=None), dict(slot_of=8194), dict(budgets=258), dict(ctx_lens=514)):
        assert evict(batch(**bad)) == BAD, bad
    assert evict(p=_pool(P=15)) == BAD and evict(t=libdkv.dkv_tables(256, 0, 0, 512)) == BAD
    assert evict(t=libdkv.dkv_tables(256, 6, 0, 520)) == BAD and evict(t=libdkv.dkv_tables(None, 6, 0, 512)) == BAD
    assert evict(ws=None) == BAD and evict(ws=(1 << 20) + 16) == BAD and evict(wsb=need - 1) == BAD


def test_the_bindings_refuse_tensors_that_do_not_fit():
    q = torch.zeros((2, 5, 4, 128), dtype=torch.bfloat16)
    kv = torch.zeros((2, 5, 2, 128), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)

    def make(**kw):
        a = dict(q=q, new_lens=i, ctx_lens=i, k_new=kv, v_new=kv)
        a.update(kw)
        return libdkv.make_chunk_batch(2, 64, max_new=5, scale=0.1, **a)

    assert make().q_stride == 512 and make().kv_stride == 256
    rows = torch.zeros((2, 5, 8, 128), dtype=torch.bfloat16)
    b = make(q=rows[:, :, :4], k_new=rows[:, :, 4:6], v_new=rows[:, :, 6:])
    assert b.q_stride == b.kv_stride == 1024
    one = rows[:, :1]
    b = libdkv.make_chunk_batch(2, 64, one[:, :, :4].contiguous(), i, i, 1, 0.1)
    assert b.q_stride == 512
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :64]), dict(q=q.transpose(1, 2)), dict(k_new=None),
                dict(k_new=kv[:, :4]), dict(k_new=kv.half()), dict(v_new=rows[:, :, 6:]), dict(q=rows[:, :, ::2]),
                dict(new_lens=i.long()), dict(ctx_lens=i[:2]), dict(out=q.float()), dict(out=rows[:, :, :4]),
                dict(lse=torch.zeros((2, 5, 3))), dict(q=q[:1].expand(2, 5, 4, 128)), dict(q=one[:, :, :4])):
        with pytest.raises(ValueError):
            make(**bad)
    with pytest.raises(ValueError):
        libdkv.ChunkPages.from_tensors(torch.zeros((1, 4, 16, 2, 64), dtype=torch.bfloat16), kv, i)
    k = torch.zeros((1, 4, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        libdkv.ChunkPages.from_tensors(k, k[:, :3], i.view(3, 1))
    pages = libdkv.ChunkPages.from_tensors(k, k.clone(), i.view(3, 1))
    with pytest.raises(ValueError):  # two layers wanted, the pages have one
        libdkv.dkv_chunk_workspace_size(make(), pages)
    s = dict(budgets=i, ctx_lens=i, sig_sum=torch.zeros((1, 48, 4)), classes=torch.zeros(96, dtype=torch.uint8),
             slot_of=torch.zeros(96, dtype=torch.int32))
    libdkv.make_evict_batch(1, 3, 4, 2, 16, **s)
    for bad in (dict(budgets=i[:2]), dict(sig_sum=s["sig_sum"].double()), dict(classes=s["slot_of"]),
                dict(slot_of=s["slot_of"][:95]), dict(sig_cnt=i), dict(ctx_lens=i.long())):
        with pytest.raises(ValueError):
            libdkv.make_evict_batch(1, 3, 4, 2, 16, **{**s, **bad})


def test_the_serial_eviction_keeps_a_decode_state_valid():
    w = W.small("evict_cpu", lens=[200, 9, 64], L=2, Hq=4, Hkv=2)
    cap, budgets = 208, [50, 9, 0]
    hd = HostDecode(w, cap, inp=W.make_inputs(w))
    cls = hd.classes.reshape(w.L, w.R, cap, w.Hkv)
    slot = np.where(cls == 2, (cls == 2).cumsum(2) - 1, np.where(cls == 1, (cls == 1).cumsum(2) - 1, -1))
    st = {"free_list": hd.pool.free_list, "cursors": hd.pool.cursors.astype(np.int64), "rev_unit": hd.pool.rev_unit,
          "rev_idx": hd.pool.rev_idx, "page_cls": hd.pool.page_cls, "pages": hd.pool.pages, "fwd": hd.tab.fwd,
          "unit_hdr": hd.tab.unit_hdr, "classes": cls, "slot_of": slot.astype(np.int32)}
    sig = hd.ctx["sig_sum"].numpy()
    got = serial_evict(st, w.L, w.R, w.Hq, w.Hkv, cap, w.P, 8, 4, budgets, w.lens, sig, sinks=2)
    for u in range(w.U):
        l, r, h = u // (w.R * w.Hkv), u // w.Hkv % w.R, u % w.Hkv
        old, new = (int(x["unit_hdr"][u][:2].sum()) for x in (st, got))
        assert new == (old if old <= budgets[r] else max(budgets[r], int((cls[l, r, :2, h] != 0).sum())))

    class Pool:
        P, F, scheme = w.P, hd.pool.F, 0
    for k in ("free_list", "rev_unit", "rev_idx", "page_cls", "pages"):
        setattr(Pool, k, got[k])
    Pool.cursors = got["cursors"].astype(np.uint64)
    where = check_state(w, cap, Pool, got["fwd"], got["unit_hdr"], got["classes"].reshape(w.L, w.R * cap, w.Hkv),
                        np.array(w.lens))
    for (u, p), (_, _, s) in where.items():  # slot_of names the slot that holds the position
        assert got["slot_of"].reshape(cls.shape)[u // (w.R * w.Hkv), u // w.Hkv % w.R, p, u % w.Hkv] == s
