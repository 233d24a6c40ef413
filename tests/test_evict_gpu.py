"""Eviction by accumulated attention on the GPU, bit for bit against a serial
restatement."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.chunk_helpers import SCALE, serial_evict
from tests.extend_helpers import make_decoder
from tests.page_ops_helpers import assert_equal, assert_untouched, pool_state

pytestmark = pytest.mark.gpu

WIDTHS = ((8, 4), (8, 2), (4, 8))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(dec):
    st = pool_state(dec.pool, dec.tables)
    st["classes"], st["slot_of"] = dec.classes.cpu().numpy(), dec.slot_of.cpu().numpy()
    return st


def _check(dec, before, w, cap, budgets, ctx, sig, cnt, sinks, window, what):
    kh, vh = WIDTHS[w.scheme]
    want = serial_evict(before, w.L, w.R, w.Hq, w.Hkv, cap, w.P, kh, vh, budgets, ctx, sig.cpu().numpy(),
                        None if cnt is None else cnt.cpu().numpy(), sinks, window)
    got = _state(dec)
    assert_equal(got, want, what)
    for k in ("classes", "slot_of"):
        assert np.array_equal(got[k], want[k].reshape(-1)), f"{what}: {k}"
    return got


CASES = {
    "tiny": dict(w=dict(lens=[512], Hq=8, Hkv=2), budgets=[100], window=64, sinks=4),
    "ragged, one left alone": dict(w=dict(lens=[300, 7, 129, 0, 1], Hq=8, Hkv=2, L=2), budgets=[50, 3, -1, 5, 0]),
    "sums, group of 7": dict(w=dict(lens=[700, 90], Hq=28, Hkv=4, P=32), budgets=[350, 80], average=False, window=33),
    "group of 1, odd heads": dict(w=dict(lens=[250, 64], Hq=3, Hkv=3, L=2, P=6), budgets=[0, 31], sinks=1),
    "group of 5, scheme 1": dict(w=dict(lens=[333], Hq=15, Hkv=3, scheme=1, P=8), budgets=[200], window=1),
    "scheme 2": dict(w=dict(lens=[600, 200], Hq=8, Hkv=2, scheme=2, P=32), budgets=[10, 199]),
    "nothing protected stays": dict(w=dict(lens=[100, 100], Hq=4, Hkv=2), budgets=[0, 0]),
    "protected beyond the budget": dict(w=dict(lens=[100, 40], Hq=4, Hkv=2), budgets=[5, 5], sinks=10, window=20),
    "window over everything": dict(w=dict(lens=[100], Hq=4, Hkv=2), budgets=[5], window=2 ** 31 - 1),
    "pages of two": dict(w=dict(lens=[64, 33], Hq=4, Hkv=1, P=2), budgets=[20, 32]),
    "long": dict(w=dict(lens=[9000, 8500], Hq=8, Hkv=2), budgets=[3000, 7000], window=64, sinks=4),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_serial_form(name):
    c = CASES[name]
    w = W.small("evict", **{"L": 1, **c["w"]})
    cap = -(-(max(w.lens) + 16) // 16) * 16
    dec, sig, cnt, ctx = make_decoder(w, cap, seed=len(name))
    avg, sinks, window = c.get("average", True), c.get("sinks", 0), c.get("window", 0)
    budgets = c["budgets"]
    for step in range(3):  # the later ones on lists whose slots are out of order
        before = _state(dec)
        dec.evict(_i32(budgets), ctx, sig, cnt if avg else None, sinks=sinks, window=window)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        _check(dec, before, w, cap, budgets, w.lens, sig, cnt if avg else None, sinks, window, f"{name}, {step}")
        sig = sig[:, torch.randperm(sig.shape[1], device="cuda")].contiguous()
        budgets = [b * 2 // 3 for b in budgets]


@pytest.mark.parametrize("what", ["equal", "zero", "few values", "not finite", "negative"])
def test_equal_and_odd_weights(what):
    w = W.small("evict_odd", lens=[700, 333], L=1, Hq=8, Hkv=2)
    cap = 704
    dec, sig, cnt, ctx = make_decoder(w, cap)
    g = torch.Generator("cuda").manual_seed(1)
    if what == "equal":
        sig.fill_(0.25)
    elif what == "zero":
        sig.zero_()
        sig[:, ::3] = -0.0
    elif what == "few values":
        sig.copy_(torch.randint(0, 3, sig.shape, generator=g, device="cuda").float())
    elif what == "negative":
        sig.copy_(torch.randn(sig.shape, generator=g, device="cuda") * 1e-40)
    else:
        x = torch.rand((sig.shape[1],), generator=g, device="cuda")
        sig[:, x < 0.3] = float("inf")
        sig[:, x > 0.6] = float("nan")
        sig[:, x > 0.9] = float("-inf")
    budgets = [300, 100]
    before = _state(dec)
    dec.evict(_i32(budgets), ctx, sig, window=5)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    _check(dec, before, w, cap, budgets, w.lens, sig, None, 0, 5, what)


def test_keys_outside_shared_memory():
    """More positions a request than a block's shared memory holds keys for."""
    w = W.small("evict_long", lens=[45000], L=1, Hq=2, Hkv=1, P=64)
    cap = 45056
    dec, sig, cnt, ctx = make_decoder(w, cap)
    before = _state(dec)
    dec.evict(_i32([9000]), ctx, sig, cnt, sinks=4, window=64)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    _check(dec, before, w, cap, [9000], w.lens, sig, cnt, 4, 64, "long")


def test_a_wrapped_ring_and_the_units_of_two_calls():
    """Layer by layer with unit_base and table offsets gives what one call over the layers gives."""
    w = W.small("evict_layers", lens=[200, 150], L=3, Hq=4, Hkv=2)
    cap = 208
    a, sig, cnt, ctx = make_decoder(w, cap)
    b, *_ = make_decoder(w, cap)
    for d in (a, b):
        d.pool.cursors += 5 * d.pool.F  # the ring's slots stay, the counters have gone round
    budgets = _i32([60, 149])
    a.evict(budgets, ctx, sig, cnt)
    n, rows = w.R * w.Hkv, w.R * cap * w.Hkv
    for l in range(w.L):
        batch = libdkv.make_evict_batch(1, w.R, w.Hq, w.Hkv, cap, budgets, ctx, sig[l:l + 1], b.classes[l * rows:(l + 1) * rows],
                                        b.slot_of[l * rows:(l + 1) * rows], cnt, unit_base=l * n)
        view = libdkv._TableView(b.tables, l * n)
        ws = torch.empty(libdkv.dkv_evict_workspace_size(batch, b.pool, view), dtype=torch.uint8, device="cuda")
        libdkv.dkv_evict(batch, b.pool, view, ws)
    assert libdkv.dkv_get_status(a.pool) == libdkv.dkv_get_status(b.pool) == libdkv.DKV_OK
    x, y = _state(a), _state(b)
    assert_equal(x, y, "layers")
    assert np.array_equal(x["classes"], y["classes"]) and np.array_equal(x["slot_of"], y["slot_of"])


def test_errors_change_nothing():
    w = W.small("evict_err", lens=[200, 150], L=2, Hq=4, Hkv=2)
    cap = 208

    def harm(dec, ctx, what):
        u, row = 3, dec.tables.fwd.view(-1)
        if what == "lens":
            ctx[1] = cap + 1
        elif what == "negative":
            ctx[0] = -1
        elif what == "header":
            dec.tables.unit_hdr[u, 0] += 1
        elif what == "page id":
            row[u * dec.pmax] = dec.pool.F
        elif what == "reverse":
            dec.pool.rev_idx[int(row[u * dec.pmax])] += 1
        elif what == "class":
            dec.classes.view(w.L, w.R, cap, w.Hkv)[0, 1, 149, 1] ^= 3
        elif what == "class 3":
            dec.classes.view(w.L, w.R, cap, w.Hkv)[0, 1, 149, 1] = 3
        elif what == "slot":
            s = dec.slot_of.view(w.L, w.R, cap, w.Hkv)[0, 1, :, 1]
            held = (s >= 0).nonzero()[:, 0]
            s[held[0]] = 10 ** 6
        elif what == "slot twice":
            s = dec.slot_of.view(w.L, w.R, cap, w.Hkv)[0, 1, :, 1]
            c = dec.classes.view(w.L, w.R, cap, w.Hkv)[0, 1, :, 1]
            held = (c == 2).nonzero()[:, 0]
            s[held[0]] = s[held[1]]
        elif what == "cursors":
            dec.pool.cursors[1] += dec.pool.F

    for what, code in (("lens", libdkv.DKV_E_LENS), ("negative", libdkv.DKV_E_LENS), *(
            (x, libdkv.DKV_E_INTERNAL) for x in ("header", "page id", "reverse", "class", "class 3", "slot",
                                                 "slot twice", "cursors"))):
        dec, sig, cnt, ctx = make_decoder(w, cap)
        ctx = ctx.clone()
        harm(dec, ctx, what)
        before = _state(dec)
        dec.evict(_i32([60, 60]), ctx, sig, cnt)
        assert libdkv.dkv_get_status(dec.pool) == code, what
        assert_untouched(_state(dec), before, what)


@pytest.mark.parametrize("bad", [300, 304, -1, 2 ** 31 - 1])
def test_a_position_in_a_page_that_is_none(bad):
    """A token whose page slot names no position of its request: it is moved and reported, its own slot_of stays and
    everything else is right."""
    w = W.small("evict_pos", lens=[300], L=1, Hq=4, Hkv=2)
    cap, u, G = 304, 1, 2
    dec, sig, cnt, ctx = make_decoder(w, cap)
    kh, vh = WIDTHS[w.scheme]
    n_hi, n_lo, p_hi = (int(x) for x in dec.tables.unit_hdr[u, :3])
    first, n, code, per = (0, n_hi, 2, w.P) if n_hi > 1 else (p_hi, n_lo, 1, 2 * w.P)
    slot, cls = (x.view(cap, w.Hkv)[:, u] for x in (dec.slot_of, dec.classes))
    p = int(((cls == code) & (slot == n - 1)).nonzero()[0, 0])  # the token in the last slot is the one that stays
    sig.view(cap, w.Hq)[p, G * u:G * (u + 1)] = 1e6
    id_ = int(dec.tables.fwd.view(-1)[u * dec.pmax + first + (n - 1) // per])
    at = 16 * (kh + vh) * w.P + 16 * w.P + 4 * ((n - 1) % per)
    page = dec.pool.pages.view(torch.uint8).view(dec.pool.F, -1)[id_]
    assert page[at:at + 4].cpu().view(torch.int32).item() == p
    page[at:at + 4] = torch.tensor([bad], dtype=torch.int32).view(torch.uint8).cuda()
    before = _state(dec)
    dec.evict(_i32([1]), ctx, sig, cnt, window=0)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    want = serial_evict(before, w.L, w.R, w.Hq, w.Hkv, cap, w.P, kh, vh, [1], w.lens, sig.cpu().numpy(), cnt.cpu().numpy())
    want["slot_of"].reshape(cap, w.Hkv)[p, u] = n - 1
    got = _state(dec)
    assert_equal(got, want, str(bad))
    for k in ("classes", "slot_of"):
        assert np.array_equal(got[k], want[k].reshape(-1)), k


def test_a_captured_call():
    w = W.small("evict_graph", lens=[400, 150], L=1, Hq=4, Hkv=2)
    cap = 400
    dec, sig, cnt, ctx = make_decoder(w, cap)
    budgets = _i32([-1, -1])
    dec.evict(budgets, ctx, sig, cnt, window=16)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.evict(budgets, ctx, sig, cnt, window=16)
    for b in ([200, 149], [100, 40], [17, 16]):
        before = _state(dec)
        budgets.copy_(_i32(b))
        g.replay()
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        _check(dec, before, w, cap, b, w.lens, sig, cnt, 0, 16, str(b))


def test_chunks_compaction_decoding_and_eviction_together():
    """A prompt in chunks, its compaction from the pages as they lie, generation steps whose attention adds to the
    significance, drafts, an eviction to a budget, and the steps after it."""
    w = W.small("served", lens=[300], L=1, Hq=8, Hkv=2)
    Hq, Hkv, n, cap = w.Hq, w.Hkv, 300, 384
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((1, cap, h, 128), generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    pages = libdkv.ChunkPages(1, 1, Hkv, cap, 64, 8)
    pages.table[0] = torch.arange(1, 7, dtype=torch.int32)  # one run of pages: rows 64 .. of the pages' tokens
    dec = libdkv.Decoder(1, 1, Hq, Hkv, cap, w.P, 2 * cap, window=32)
    sig, cnt = torch.zeros((1, cap, Hq), device="cuda"), torch.zeros(cap, dtype=torch.int32, device="cuda")
    pos = torch.arange(cap, device="cuda")
    ctx = 0
    for m in (128, 100, 72):
        sl = slice(ctx, ctx + m)
        out, lse = torch.empty((1, m, Hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, m, Hq), device="cuda")
        b = libdkv.make_chunk_batch(Hkv, cap, q[:, sl], _i32([m]), _i32([ctx]), m, SCALE, k_new=k[:, sl],
                                    v_new=v[:, sl], out=out, lse=lse)
        ws = torch.empty(libdkv.dkv_chunk_workspace_size(b, pages), dtype=torch.uint8, device="cuda")
        libdkv.dkv_chunk_attention(b, pages, dec.pool, ws)
        libdkv.dkv_chunk_significance(b, pages, sig, dec.pool)
        ctx += m
        cnt += torch.where(pos < ctx - m, m, (ctx - pos).clamp(min=0)).to(torch.int32)
    assert torch.equal(cnt[:n], (n - pos[:n]).to(torch.int32))
    layer = {"L": 1, "R": 1, "Hq": Hq, "Hkv": Hkv, "T": n, "lens": _i32([n]), "sig_cnt": cnt, "sig_sum": sig,
             "k": pages.k[0, 1:].flatten(0, 1), "v": pages.v[0, 1:].flatten(0, 1)}
    assert torch.equal(layer["k"][:n], k[0, :n])
    dec.prefill_layer(layer, 0, n, 1.0, 0.2)
    dec.index(_i32([ctx]))
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK

    def steps(m, ctx):
        for _ in range(m):
            new = {"k_new": k[:, ctx:ctx + 1].contiguous(), "v_new": v[:, ctx:ctx + 1].contiguous()}
            out = torch.empty((1, 1, Hq, 128), device="cuda")
            dec.attend(q[:, ctx:ctx + 1].contiguous(), _i32([ctx]), out, SCALE, new_lens=_i32([1]), sig_sum=sig, **new)
            cnt[:ctx + 1] += 1
            dec.step({**new, "sig_sum": sig, "sig_cnt": cnt, "ctx_lens": _i32([ctx]), "new_lens": _i32([1])}, 1.0, 0.2)
            ctx += 1
        return ctx, out

    ctx, _ = steps(20, ctx)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    before = _state(dec)
    free = int(dec.pool.cursors[1] - dec.pool.cursors[0])
    dec.evict(_i32([120]), _i32([ctx]), sig, cnt, sinks=4)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    _check(dec, before, w, cap, [120], [ctx], sig, cnt, 4, 32, "served")
    hdr = dec.tables.unit_hdr.cpu()
    assert bool(((hdr[:, 0] + hdr[:, 1]) <= 120).all())
    assert int(dec.pool.cursors[1] - dec.pool.cursors[0]) > free
    ctx, out = steps(10, ctx)
    d = {n: torch.empty((1, 4, Hq, 128), dtype=torch.bfloat16, device="cuda") for n in ("out",)}
    dec.extend(q[:, ctx:ctx + 4].contiguous(), _i32([4]), _i32([ctx]), 4, d["out"], SCALE,
               k_new=k[:, ctx:ctx + 4].contiguous(), v_new=v[:, ctx:ctx + 4].contiguous())
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(d["out"].float()).all())
    # the index that the pages give is the one that was kept
    cls, slot = dec.classes.clone(), dec.slot_of.clone()
    dec.index(_i32([ctx]))
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert torch.equal(dec.classes, cls) and torch.equal(dec.slot_of, slot)
