"""Attention of several new tokens a request over the pages, and the
significance of the accepted ones, against float64 from the raw page bytes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, check_attention, check_significance, draw_new, make_decoder, reference
from tests.page_ops_helpers import pool_state

pytestmark = pytest.mark.gpu

# request lengths, new tokens, heads, page tokens, scheme, layers
CASES = {
    "one token": dict(lens=[300], new=[1], Hq=8, Hkv=2, P=16, scheme=0),
    "drafts": dict(lens=[300, 7, 517, 0, 129], new=[4, 1, 8, 3, 0], Hq=8, Hkv=2, P=16, scheme=0),
    "odd group": dict(lens=[130, 257], new=[19, 37], Hq=14, Hkv=2, P=6, scheme=1),
    "4-bit keys": dict(lens=[129, 64, 1], new=[33, 2, 5], Hq=6, Hkv=2, P=8, scheme=2),
    "one head a group": dict(lens=[200, 33], new=[130, 129], Hq=3, Hkv=3, P=2, scheme=0),
    "chunk": dict(lens=[700], new=[300], Hq=8, Hkv=2, P=16, scheme=0),
    "whole tiles": dict(lens=[512], new=[128], Hq=4, Hkv=2, P=16, scheme=2),
    "wide group": dict(lens=[260], new=[17], Hq=16, Hkv=1, P=32, scheme=1),
    "long": dict(lens=[9000], new=[3], Hq=4, Hkv=1, P=64, scheme=0),
    "no context": dict(lens=[0, 0], new=[5, 140], Hq=8, Hkv=2, P=16, scheme=0),
}


def _workload(c, **kw):
    return W.small("extend", **dict(dict(L=1, lens=c["lens"], Hq=c["Hq"], Hkv=c["Hkv"], P=c["P"],
                                         scheme=c["scheme"]), **kw))


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _run(w, dec, ctx, new, q, k, v, layer0=0, acc=None, sig=None, max_new=None, lse=True, **kw):
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:3], float("nan"), device="cuda") if lse else None
    new_t, mx = _i32(new), max(new) if max_new is None else max_new
    qc = q.cuda()
    kc, vc = (None, None) if k is None else (k.cuda(), v.cuda())
    dec.extend(qc, new_t, ctx, mx, out, SCALE, k_new=kc, v_new=vc, lse=ls, layer0=layer0, **kw)
    if sig is not None:
        dec.extend_significance(qc, new_t, _i32(acc), ctx, mx, SCALE, ls, sig, k_new=kc, v_new=vc, layer0=layer0,
                                **kw)
    return out, ls


@pytest.mark.parametrize("name", list(CASES))
def test_attention_and_significance(name):
    c = CASES[name]
    w = _workload(c)
    cap = -(-(max(c["lens"]) + max(c["new"])) // 16) * 16
    dec, sig, _, ctx = make_decoder(w, cap)
    q, k, v = draw_new(w, c["new"], 1, 3)
    acc = [max(0, n - (r % 3)) for r, n in enumerate(c["new"])]
    before = sig.cpu().numpy()
    state = pool_state(dec.pool, dec.tables)
    out, lse = _run(w, dec, ctx, c["new"], q, k, v, acc=acc, sig=sig, max_new=max(c["new"]) + 3)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    ref = reference(state, w, q, k, v, c["new"], acc)
    check_attention(out, lse, ref, name)
    check_significance(sig.cpu().numpy(), before, ref, w, cap, c["lens"], acc, what=name)
    after = pool_state(dec.pool, dec.tables)
    assert all(np.array_equal(after[x], state[x]) for x in state)  # the pool is read only


def test_layers_in_one_call_and_one_by_one():
    w = W.small("extend_layers", lens=[140, 60], L=3, Hq=6, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 176)
    new = [9, 20]
    q, k, v = draw_new(w, new, 2, 5)
    s1, s2 = sig.clone(), sig.clone()
    out, lse = _run(w, dec, ctx, new, q, k, v, layer0=1, acc=new, sig=s1)
    ref = reference(pool_state(dec.pool, dec.tables), w, q, k, v, new, new, layer0=1)
    check_attention(out, lse, ref)
    check_significance(s1.cpu().numpy(), sig.cpu().numpy(), ref, w, 176, w.lens, new, layer0=1)
    for l in range(2):
        o, ls = _run(w, dec, ctx, new, q[l:l + 1].contiguous(), k[l:l + 1].contiguous(), v[l:l + 1].contiguous(),
                     layer0=1 + l, acc=new, sig=s2)
        check_attention(o, ls, tuple(x[l:l + 1] for x in ref[:4]) + ({},))
    torch.testing.assert_close(s1, s2, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("mix", ["all high", "all low", "nothing held"])
def test_lists_of_one_class(mix):
    ah, al = {"all high": (0.0, 0.0), "all low": (1e9, 0.0), "nothing held": (1e9, 1e9)}[mix]
    w = W.small("extend_mix", lens=[150, 128, 31], L=1, Hq=8, Hkv=2, alpha_h=ah, alpha_l=al)
    dec, sig, _, ctx = make_decoder(w, 192)
    new = [5, 40, 1]
    q, k, v = draw_new(w, new, 1, 11)
    before = sig.cpu().numpy()
    out, lse = _run(w, dec, ctx, new, q, k, v, acc=new, sig=sig)
    ref = reference(pool_state(dec.pool, dec.tables), w, q, k, v, new, new)
    check_attention(out, lse, ref, mix)
    check_significance(sig.cpu().numpy(), before, ref, w, 192, w.lens, new, what=mix)
    if mix == "nothing held":  # rows that attend nothing at all: zeros, -inf, nothing added
        sig2 = sig.clone()
        out, lse = _run(w, dec, ctx, new, q, None, None, acc=new, sig=sig2)
        assert not out.float().any() and bool((lse == float("-inf")).all()) and torch.equal(sig2, sig)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK


def test_held_tokens_alone():
    """Without k_new only the pages are attended; lse is optional."""
    w = W.small("extend_held", lens=[77, 300], L=1, Hq=8, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 320)
    new = [3, 6]
    q, k, v = draw_new(w, new, 1, 4)
    before = sig.cpu().numpy()
    out, lse = _run(w, dec, ctx, new, q, None, None, acc=[2, 6], sig=sig)
    st = pool_state(dec.pool, dec.tables)
    # the single-token attention gives the same answers row by row
    one = torch.empty((1, w.R, w.Hq, 128), device="cuda")
    rows = torch.tensor([0, 3])
    for i in range(3):
        dec.attend(q[:, rows + i].cuda().contiguous(), ctx, one, SCALE)
        got = out[:, rows + i].float()
        torch.testing.assert_close(got, one, rtol=2 ** -7, atol=2e-3)
    far = reference(st, w, q, k * 0, v * 0, new)  # bounds only
    assert np.isfinite(far[1]).all()
    changed = (sig.cpu().numpy() != before).reshape(w.R, 320, w.Hq)
    assert changed[0, :77].any() and not changed[0, 77:].any() and not changed[1, 300:].any()
    out2, _ = _run(w, dec, ctx, new, q, None, None, lse=False)
    assert torch.equal(out, out2)


def test_extreme_values_and_scales():
    """Queries and keys of very different sizes, a row whose largest logit
    comes last, large negative logits, zero queries."""
    w = W.small("extend_extreme", lens=[260, 40], L=1, Hq=4, Hkv=1, outlier_scale=300.0)
    dec, _, _, ctx = make_decoder(w, 400)
    new = [100, 9]
    q, k, v = draw_new(w, new, 1, 21, outlier=40.0)
    q[0, :, 0] *= 30.0
    q[0, :, 1] = 0.0
    q[0, :, 2] *= 2.0 ** -20
    k[0, 50:] *= 8.0
    v[0, 3] *= 1000.0
    v[0, 4] *= 2.0 ** -12
    out, lse = _run(w, dec, ctx, new, q, k, v)
    check_attention(out, lse, reference(pool_state(dec.pool, dec.tables), w, q, k, v, new), "extreme")
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK


def test_values_that_are_not_finite_are_reported():
    w = W.small("extend_nan", lens=[40, 50], L=1, Hq=4, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 64)
    new = [4, 6]
    q, k, v = draw_new(w, new, 1, 2)
    for t, x in ((k, float("nan")), (v, float("inf"))):
        bad = t.clone()
        bad[0, 2, 1, 9] = x
        kk, vv = (bad, v) if t is k else (k, bad)
        out, lse = _run(w, dec, ctx, new, q, kk, vv)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_RANGE
        zero = bad.clone()
        zero[0, 2, 1, 9] = 0.0
        kk, vv = (zero, v) if t is k else (k, zero)
        check_attention(out, lse, reference(pool_state(dec.pool, dec.tables), w, q, kk, vv, new), "taken as 0")
    # a query that is not finite spoils its own row alone
    qq = q.clone()
    qq[0, 5, 1, 3] = float("inf")
    out, _ = _run(w, dec, ctx, new, qq, k, v)
    good, _ = _run(w, dec, ctx, new, q, k, v)
    same = torch.ones(q.shape[:3], dtype=torch.bool)
    same[0, 5, 1] = False
    assert torch.equal(out.cpu()[same], good.cpu()[same])


def test_bad_lengths_write_nothing():
    w = W.small("extend_lens", lens=[40, 50], L=1, Hq=4, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 64)
    q, k, v = draw_new(w, [4, 6], 1, 2)
    for new, ctx_l, mx in (([4, 5], [40, 50], 8), ([5, 5], [40, 50], 4), ([-1, 11], [40, 50], 16),
                           ([4, 6], [40, 60], 8), ([4, 6], [-1, 50], 8)):
        before = sig.clone()
        lse0 = torch.zeros(q.shape[:3], device="cuda")
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        b = (q.cuda(), _i32(new), _i32(ctx_l), mx)
        dec.extend(*b, out, SCALE, k_new=k.cuda(), v_new=v.cuda(), lse=lse0)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_LENS
        assert bool((out == 7.0).all()) and not lse0.any()
    for acc in ([5, 6], [-1, 0]):
        dec.extend_significance(q.cuda(), _i32([4, 6]), _i32(acc), ctx, 8, SCALE, lse0, sig, k_new=k.cuda(),
                                v_new=v.cuda())
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_LENS
        assert torch.equal(sig, before)


def test_bad_tables_are_left_out():
    """A header that contradicts itself empties that unit's lists, a page id
    out of range leaves its tokens out; both are reported, the rest is right."""
    w = W.small("extend_bad", lens=[150, 90], L=1, Hq=4, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 176)
    new = [4, 3]
    q, k, v = draw_new(w, new, 1, 8)
    st = pool_state(dec.pool, dec.tables)
    ref = reference(st, w, q, k, v, new, new)
    hdr = dec.tables.unit_hdr.clone()
    dec.tables.unit_hdr[1, 0] = 1 << 30
    out, lse = _run(w, dec, ctx, new, q, k, v)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    st1 = {**st, "unit_hdr": st["unit_hdr"].copy()}
    st1["unit_hdr"][1] = 0
    check_attention(out, lse, reference(st1, w, q, k, v, new), "empty unit")
    dec.tables.unit_hdr.copy_(hdr)
    fwd = dec.tables.fwd.clone()
    p_hi = int(hdr[0, 2])
    last = p_hi - 1  # the high list's last page: dropping it leaves a shorter list
    dec.tables.fwd[0, last] = dec.pool.F
    s2 = sig.clone()
    out, lse = _run(w, dec, ctx, new, q, k, v, acc=new, sig=s2)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    st2 = {**st, "unit_hdr": st["unit_hdr"].copy(), "fwd": st["fwd"].copy()}
    st2["unit_hdr"][0, 0], st2["unit_hdr"][0, 2] = last * w.P, last
    st2["fwd"][0, last:-1] = st["fwd"][0, last + 1:]
    r2 = reference(st2, w, q, k, v, new, new)
    check_attention(out, lse, r2, "page left out")
    check_significance(s2.cpu().numpy(), sig.cpu().numpy(), r2, w, 176, w.lens, new, what="page left out")
    dec.tables.fwd.copy_(fwd)
    out, lse = _run(w, dec, ctx, new, q, k, v)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    check_attention(out, lse, ref)


def test_equal_inputs_give_equal_bits_on_another_stream_and_in_a_graph():
    w = W.small("extend_graph", lens=[1500, 900], L=1, Hq=8, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 1600)
    new = [8, 5]
    q, k, v = (x.cuda() for x in draw_new(w, new, 1, 6))
    new_t, out = _i32(new), [torch.zeros_like(q) for _ in range(3)]
    lse = [torch.zeros(q.shape[:3], device="cuda") for _ in range(3)]
    s = [sig.clone() for _ in range(3)]

    def both(i, stream=None):
        dec.extend(q, new_t, ctx, 8, out[i], SCALE, k_new=k, v_new=v, lse=lse[i], stream=stream)
        dec.extend_significance(q, new_t, new_t, ctx, 8, SCALE, lse[i], s[i], k_new=k, v_new=v, stream=stream)

    both(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    both(1, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(2)
    g.replay()
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(out[0], out[i]) and torch.equal(lse[0], lse[i]) and torch.equal(s[0], s[i])
    # new inputs in the same buffers: the replay answers for them
    q.copy_(torch.randn_like(q.float()).bfloat16())
    both(0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[2]) and torch.equal(lse[0], lse[2])


def test_no_tokens_at_all():
    w = W.small("extend_none", lens=[40], L=1, Hq=4, Hkv=2)
    dec, sig, _, ctx = make_decoder(w, 64)
    q = torch.zeros((1, 0, 4, 128), dtype=torch.bfloat16, device="cuda")
    before = sig.clone()
    dec.extend(q, _i32([0]), ctx, 0, torch.empty_like(q), SCALE)
    dec.extend_significance(q, _i32([0]), _i32([0]), ctx, 0, SCALE, torch.zeros((1, 0, 4), device="cuda"), sig)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK and torch.equal(sig, before)
