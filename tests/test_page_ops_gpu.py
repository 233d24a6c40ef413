"""Fork, release and defrag on the GPU against a serial restatement of the
definitions, their refusals (all-or-nothing), and a run of them together with
the calls around them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.decode_helpers import check_state
from tests.extend_helpers import SCALE, draw_new, make_decoder
from tests.page_ops_helpers import (assert_equal, assert_untouched, pool_state, serial_defrag, serial_fork,
                                    serial_release)

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _scatter(dec, seed):
    """Puts the pool into the middle of its life: a shuffled ring that is
    about to wrap, pages scattered over the pool."""
    p, t = dec.pool, dec.tables
    g = torch.Generator().manual_seed(seed)
    F = p.F
    to = torch.randperm(F, generator=g).to("cuda")
    head, tail = (int(x) for x in p.cursors)
    ring = (torch.arange(head, tail, device="cuda")) % F
    free = to[p.free_list[ring].long()].to(torch.int32)
    for name in ("rev_unit", "rev_idx", "page_cls", "pages"):
        x = getattr(p, name)
        x[to] = x.clone()
    live = t.fwd >= 0
    t.fwd[live] = to[t.fwd[live].long()].to(torch.int32)
    head2 = 3 * F - 7
    p.free_list[(torch.arange(head2, head2 + free.numel(), device="cuda")) % F] = \
        free[torch.randperm(free.numel(), generator=g).to("cuda")]
    p.cursors.copy_(torch.tensor([head2, head2 + free.numel()]))


def _decoder(lens, cap, F=None, **kw):
    w = W.small("pages", **dict(dict(lens=lens, L=2, Hq=6, Hkv=2), **kw))
    dec, sig, cnt, ctx = make_decoder(w, cap, F=F)
    _scatter(dec, 5)
    return w, dec, sig, cnt, ctx


FORKS = [
    dict(lens=[300, 0, 129], src=[0], dst=[1], P=16, scheme=0),
    dict(lens=[300, 0, 0, 40, 0], src=[0, 0, 3], dst=[4, 1, 2], P=6, scheme=1),
    dict(lens=[0, 0, 5, 0], src=[2, 3], dst=[0, 1], P=16, scheme=0),   # request 3 holds nothing
    dict(lens=[1000, 0, 900, 0], src=[2, 0], dst=[1, 3], P=64, scheme=2),
]


@pytest.mark.parametrize("c", FORKS, ids=lambda c: f"{c['src']}-{c['dst']}")
def test_fork(c):
    cap = -(-(max(c["lens"]) + 8) // 16) * 16
    w, dec, sig, cnt, ctx = _decoder(c["lens"], cap, P=c["P"], scheme=c["scheme"])
    before = pool_state(dec.pool, dec.tables)
    rows = {"classes": dec.classes.cpu().numpy().reshape(w.L, w.R, cap, w.Hkv),
            "slot_of": dec.slot_of.cpu().numpy().reshape(w.L, w.R, cap, w.Hkv),
            "sig": sig.cpu().numpy().reshape(w.L, w.R, cap, w.Hq), "cnt": cnt.cpu().numpy().reshape(1, w.R, cap, 1)}
    want = {k: v.copy() for k, v in rows.items()}
    for s, d in zip(c["src"], c["dst"]):
        for x in want.values():
            x[:, d, :c["lens"][s]] = x[:, s, :c["lens"][s]]
    dec.fork(_i32(c["src"]), _i32(c["dst"]), ctx, sig_sum=sig, sig_cnt=cnt)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    after = pool_state(dec.pool, dec.tables)
    assert_equal(after, serial_fork(before, w.L, w.R, w.Hkv, c["src"], c["dst"]), "fork")
    got = {"classes": dec.classes, "slot_of": dec.slot_of, "sig": sig, "cnt": cnt}
    for k, x in want.items():
        assert np.array_equal(got[k].cpu().numpy().reshape(x.shape), x), k
    lens = np.array(c["lens"])
    lens[c["dst"]] = lens[c["src"]]
    check_state(w, cap, _np_pool(dec, after), after["fwd"], after["unit_hdr"],
                dec.classes.cpu().numpy().reshape(w.L, w.R * cap, w.Hkv), lens)


def _np_pool(dec, st):
    class P:
        pass
    p = P()
    p.P, p.F, p.scheme = dec.pool.P, dec.pool.F, dec.pool.scheme
    for k in ("free_list", "rev_unit", "rev_idx", "page_cls", "pages"):
        setattr(p, k, st[k])
    p.cursors = st["cursors"].astype(np.uint64)
    return p


@pytest.mark.parametrize("reqs", [[0], [3, 0, 1], [2], [4, 3, 2, 1, 0]])
def test_release(reqs):
    lens = [300, 7, 0, 129, 64]
    w, dec, _, _, ctx = _decoder(lens, 320)
    before = pool_state(dec.pool, dec.tables)
    dec.release(_i32(reqs))
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    after = pool_state(dec.pool, dec.tables)
    assert_equal(after, serial_release(before, w.L, w.R, w.Hkv, reqs), "release")
    dec.release(_i32(reqs))  # they hold nothing now
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert_untouched(pool_state(dec.pool, dec.tables), after, "second release")


@pytest.mark.parametrize("F,P,scheme", [(None, 16, 0), (5000, 6, 1), (None, 32, 2)])
def test_defrag(F, P, scheme):
    lens = [300, 7, 0, 129, 64]
    w, dec, _, _, ctx = _decoder(lens, 320, P=P, scheme=scheme, **({} if F is None else {"F": F}))
    dec.release(_i32([3]))
    before = pool_state(dec.pool, dec.tables)
    q = W.decode_queries(w, w.L, 3).cuda()
    o = [torch.empty((w.L, w.R, w.Hq, 128), device="cuda") for _ in range(2)]
    ctx = ctx.clone()
    ctx[3] = 0
    dec.attend(q, ctx, o[0], SCALE)
    dec.defrag()
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    after = pool_state(dec.pool, dec.tables)
    assert_equal(after, serial_defrag(before), "defrag")
    n = dec.pool.F - int(after["cursors"][1] - after["cursors"][0])
    assert (after["page_cls"][:n] != 0).all() and not after["page_cls"][n:].any()
    dec.attend(q, ctx, o[1], SCALE)
    assert torch.equal(o[0], o[1])
    dec.defrag()  # a packed pool: nothing moves
    assert_equal(pool_state(dec.pool, dec.tables), serial_defrag(after), "second defrag")


def test_defrag_of_a_full_and_an_empty_pool():
    w = W.small("pages_edge", lens=[64, 64], L=1, Hq=2, Hkv=1, P=16, alpha_h=0.0, alpha_l=0.0)
    dec, _, _, _ = make_decoder(w, 64, F=8)  # every page owned
    before = pool_state(dec.pool, dec.tables)
    assert (before["page_cls"] != 0).all()
    dec.defrag()
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert_equal(pool_state(dec.pool, dec.tables), serial_defrag(before), "full")
    dec.release(_i32([0, 1]))
    st = pool_state(dec.pool, dec.tables)
    dec.defrag()
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert_equal(pool_state(dec.pool, dec.tables), serial_defrag(st), "empty")


def test_layer_by_layer_equals_one_call():
    lens = [300, 0, 129, 0]
    states = []
    for split in (False, True):
        w, dec, _, _, _ = _decoder(lens, 320)
        src, dst, reqs = _i32([0, 2]), _i32([3, 1]), _i32([2, 3])
        ws = torch.empty(libdkv.dkv_page_ops_workspace_size(dec.pool, dec.tables), dtype=torch.uint8, device="cuda")
        per = w.R * w.Hkv
        for l in range(w.L if split else 1):
            L = 1 if split else w.L
            t = libdkv.DeviceTables.from_tensors(dec.tables.fwd[l * per:(l + L) * per],
                                                 dec.tables.unit_hdr[l * per:(l + L) * per])
            libdkv.dkv_fork(libdkv.make_fork_batch(L, w.R, w.Hq, w.Hkv, 320, src, dst, unit_base=l * per), dec.pool, t,
                            ws)
        for l in range(w.L if split else 1):
            L = 1 if split else w.L
            t = libdkv.DeviceTables.from_tensors(dec.tables.fwd[l * per:(l + L) * per],
                                                 dec.tables.unit_hdr[l * per:(l + L) * per])
            libdkv.dkv_release(libdkv.make_release_batch(L, w.R, w.Hkv, reqs, unit_base=l * per), dec.pool, t, ws)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        states.append(pool_state(dec.pool, dec.tables))
    assert_equal(states[1], states[0], "layers")


def test_refusals_change_nothing():
    lens = [300, 0, 129, 0]
    w, dec, sig, cnt, ctx = _decoder(lens, 320)
    pool, tab = dec.pool, dec.tables

    def refused(code, call, what):
        before = pool_state(pool, tab)
        rows = [x.clone() for x in (dec.classes, dec.slot_of, sig, cnt)]
        call()
        assert libdkv.dkv_get_status(pool) == code, what
        assert_untouched(pool_state(pool, tab), before, what)
        assert all(torch.equal(a, b) for a, b in zip(rows, (dec.classes, dec.slot_of, sig, cnt))), what

    def fork(src, dst, c=ctx):
        return lambda: dec.fork(_i32(src), _i32(dst), c, sig_sum=sig, sig_cnt=cnt)

    E = libdkv.DKV_E_INTERNAL
    refused(E, fork([0], [2]), "the destination holds pages")
    refused(E, fork([0, 2], [1, 1]), "a destination twice")
    refused(E, fork([0, 1], [1, 3]), "a destination that is a source")
    refused(E, fork([0], [0]), "onto itself")
    refused(E, fork([4], [1]), "a source out of range")
    refused(E, fork([0], [-1]), "a destination out of range")
    refused(libdkv.DKV_E_LENS, fork([0], [1], _i32([321, 0, 0, 0])), "a context beyond cap")
    refused(E, lambda: dec.release(_i32([0, 0])), "released twice in one call")
    refused(E, lambda: dec.release(_i32([4])), "out of range")
    hdr, fwd = tab.unit_hdr.clone(), tab.fwd.clone()

    def with_bad(change, call, what):
        change()
        refused(E, call, what)
        tab.unit_hdr.copy_(hdr)
        tab.fwd.copy_(fwd)

    def set_hdr():
        tab.unit_hdr[0, 2] += 1

    def set_page():
        tab.fwd[1, 0] = pool.F

    def twice():
        tab.fwd[1, 0] = tab.fwd[1, 1]

    for change in (set_hdr, set_page, twice):
        with_bad(change, lambda: dec.release(_i32([0])), "release over bad tables")
        with_bad(change, fork([0], [1]), "fork over bad tables")
    with_bad(twice, lambda: dec.defrag(), "defrag over bad tables")
    cls = pool.page_cls.clone()
    pool.page_cls[int(fwd[0, 0])] = 0
    refused(E, lambda: dec.defrag(), "defrag over bad classes")
    pool.page_cls.copy_(cls)
    cur = pool.cursors.clone()
    pool.cursors[1] -= 1  # one page is neither free nor owned
    refused(E, lambda: dec.defrag(), "defrag over bad cursors")
    pool.cursors[1] = pool.cursors[0] + int(hdr[:, 2:].sum()) // 4
    refused(libdkv.DKV_E_NOMEM, fork([0], [1]), "too few pages")
    pool.cursors.copy_(cur)
    dec.fork(_i32([0]), _i32([1]), ctx, sig_sum=sig, sig_cnt=cnt)
    assert libdkv.dkv_get_status(pool) == libdkv.DKV_OK


def test_many_requests_and_layers():
    """More list units than one block takes, over a ring that wraps."""
    lens = [(37 * i) % 90 for i in range(20)]
    for i in (3, 11, 19):
        lens[i] = 0
    w, dec, sig, cnt, ctx = _decoder(lens, 96, L=3, Hq=4, Hkv=4, P=4)
    st = pool_state(dec.pool, dec.tables)
    src, dst = [1, 1, 7], [19, 3, 11]
    dec.fork(_i32(src), _i32(dst), ctx, sig_sum=sig, sig_cnt=cnt)
    st = serial_fork(st, w.L, w.R, w.Hkv, src, dst)
    assert_equal(pool_state(dec.pool, dec.tables), st, "fork")
    gone = [19, 0, 5, 6, 17, 2]
    dec.release(_i32(gone))
    st = serial_release(st, w.L, w.R, w.Hkv, gone)
    assert_equal(pool_state(dec.pool, dec.tables), st, "release")
    dec.defrag()
    assert_equal(pool_state(dec.pool, dec.tables), serial_defrag(st), "defrag")
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK


def test_a_speculative_loop():
    """As a server uses them: a prompt is forked, both branches score drafts
    over the pages, the accepted drafts' significance is added and they enter
    the cache one generation step each, one branch is released, the pool is
    packed.  The branch that lives on must match a decoder that never forked."""
    lens = [200, 0, 150]
    cap = 256
    w, dec, sig, cnt, ctx = _decoder(lens, cap, Hq=8, Hkv=2)
    w2, ref, sig2, cnt2, ctx2 = _decoder(lens, cap, Hq=8, Hkv=2)
    dec.fork(_i32([0]), _i32([1]), ctx, sig_sum=sig, sig_cnt=cnt)
    ctx[1] = ctx[0]
    new, acc = [4, 4, 3], [2, 3, 0]
    q, k, v = (x.cuda() for x in draw_new(w, new, w.L, 9))
    q[:, 4:8], k[:, 4:8], v[:, 4:8] = q[:, 0:4], k[:, 0:4], v[:, 0:4]  # both branches draft the same
    outs = []
    for d, s, c, cx, nw, ac in ((dec, sig, cnt, ctx, new, acc), (ref, sig2, cnt2, ctx2, [4, 0, 3], [2, 0, 0])):
        keep = torch.tensor([0, 1, 2, 3] + ([4, 5, 6, 7] if nw[1] else []) + [8, 9, 10], device="cuda")
        qq, kk, vv = (x[:, keep].contiguous() for x in (q, k, v))
        out = torch.empty_like(qq)
        lse = torch.empty(qq.shape[:3], device="cuda")
        d.extend(qq, _i32(nw), cx, 4, out, SCALE, k_new=kk, v_new=vv, lse=lse)
        d.extend_significance(qq, _i32(nw), _i32(ac), cx, 4, SCALE, lse, s, k_new=kk, v_new=vv)
        outs.append(out)
        starts = np.concatenate([[0], np.cumsum(nw)[:-1]])
        c2 = c.view(w.R, cap)
        for r in range(w.R):  # the caller's counts: the held tokens first, then the new ones
            c2[r, :int(cx[r])] += ac[r]
            for j in range(ac[r]):
                c2[r, int(cx[r]) + j] = ac[r] - j
        for step in range(max(ac)):
            one = [1 if step < a else 0 for a in ac]
            at = torch.tensor([int(starts[r]) + min(step, max(nw[r] - 1, 0)) if nw[r] else 0 for r in range(w.R)],
                              device="cuda")
            d.step({"k_new": kk[:, at].contiguous(), "v_new": vv[:, at].contiguous(), "sig_sum": s, "sig_cnt": c,
                    "ctx_lens": cx, "new_lens": _i32(one)}, w.alpha_h, w.alpha_l)
            assert libdkv.dkv_get_status(d.pool) == libdkv.DKV_OK
            cx += _i32(one)
    assert torch.equal(outs[0][:, :4], outs[1][:, :4]) and torch.equal(outs[0][:, 8:], outs[1][:, 4:])
    assert torch.equal(outs[0][:, :4], outs[0][:, 4:8])
    dec.release(_i32([1]))
    ctx[1] = 0
    dec.defrag()
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    st = pool_state(dec.pool, dec.tables)
    check_state(w, cap, _np_pool(dec, st), st["fwd"], st["unit_hdr"],
                dec.classes.cpu().numpy().reshape(w.L, w.R * cap, w.Hkv), ctx.cpu().numpy())
    qa = W.decode_queries(w, w.L, 3).cuda()
    a, b = (torch.empty((w.L, w.R, w.Hq, 128), device="cuda") for _ in range(2))
    dec.attend(qa, ctx, a, SCALE)
    ref.attend(qa, ctx2, b, SCALE)
    for r in (0, 2):
        torch.testing.assert_close(a[:, r], b[:, r], rtol=1e-5, atol=1e-6)
    assert torch.equal(dec.tables.unit_hdr.view(w.L, w.R, w.Hkv, 4)[:, [0, 2]],
                       ref.tables.unit_hdr.view(w.L, w.R, w.Hkv, 4)[:, [0, 2]])


def test_page_ops_in_a_graph_and_on_another_stream():
    lens = [300, 0, 129, 0]
    w, dec, sig, cnt, ctx = _decoder(lens, 320)
    src, dst, reqs = _i32([0]), _i32([1]), _i32([1])
    st0 = pool_state(dec.pool, dec.tables)
    dec.fork(src, dst, ctx)  # first use: the workspace is made
    dec.release(reqs)
    torch.cuda.synchronize()
    st = serial_release(serial_fork(st0, w.L, w.R, w.Hkv, [0], [1]), w.L, w.R, w.Hkv, [1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.fork(src, dst, ctx, sig_sum=sig, sig_cnt=cnt)
        dec.release(reqs)
        dec.defrag()
    assert_equal(pool_state(dec.pool, dec.tables), st, "capture runs nothing")
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        st = serial_defrag(serial_release(serial_fork(st, w.L, w.R, w.Hkv, [0], [1]), w.L, w.R, w.Hkv, [1]))
        assert_equal(pool_state(dec.pool, dec.tables), st, "replay")
    s = torch.cuda.Stream()
    dec.fork(src, dst, ctx, stream=s)
    s.synchronize()
    assert_equal(pool_state(dec.pool, dec.tables), serial_fork(st, w.L, w.R, w.Hkv, [0], [1]), "side stream")
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
