"""The same operators where another kernel, another split or another layout of
the work answers: few rows a unit, page sizes around a tile, split contexts, the
widths of the significance's columns, more requests than are ordered, more list
units than a warp each."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, check_attention, check_significance, draw_new, make_decoder, reference
from tests.page_ops_helpers import assert_equal, pool_state, serial_fork, serial_release

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _check(w, new, max_new, acc=None, layer0=0, n_layers=None, held_only=False, seed=3):
    n_layers = w.L if n_layers is None else n_layers
    acc = list(new) if acc is None else acc
    cap = -(-(max(w.lens) + max_new) // 16) * 16
    dec, sig, _, ctx = make_decoder(w, cap)
    q, k, v = draw_new(w, new, n_layers, seed)
    if held_only:
        k = v = None
    before, state = sig.cpu().numpy(), pool_state(dec.pool, dec.tables)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    qc = q.cuda()
    kc, vc = (None, None) if k is None else (k.cuda(), v.cuda())
    dec.extend(qc, _i32(new), ctx, max_new, out, SCALE, k_new=kc, v_new=vc, lse=lse, layer0=layer0)
    dec.extend_significance(qc, _i32(new), _i32(acc), ctx, max_new, SCALE, lse, sig, k_new=kc, v_new=vc,
                            layer0=layer0)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    ref = reference(state, w, q, k, v, new, acc, layer0=layer0)
    check_attention(out, lse, ref)
    check_significance(sig.cpu().numpy(), before, ref, w, cap, w.lens, acc, layer0=layer0, new=k is not None)
    return out, lse


@pytest.mark.parametrize("P", [2, 6, 16, 64, 130])
@pytest.mark.parametrize("scheme", [0, 1, 2])
def test_few_rows_and_page_sizes(scheme, P):
    w = W.small("few", L=1, lens=[700, 129, 5, 0, 260, 128], Hq=8, Hkv=2, P=P, scheme=scheme)
    _check(w, [8, 3, 1, 2, 0, 5], 8)


@pytest.mark.parametrize("held_only", [False, True])
@pytest.mark.parametrize("scheme", [0, 1, 2])
def test_few_rows_of_a_split_context(scheme, held_only):
    """One long request makes the parts; the others have fewer tiles than parts, or none."""
    w = W.small("few_split", L=1, lens=[9000, 300, 0], Hq=4, Hkv=1, P=16, scheme=scheme)
    _check(w, [8, 2, 3], 8, acc=[5, 2, 0], held_only=held_only)


def test_few_rows_of_a_range_of_layers():
    w = W.small("few_layers", L=3, lens=[40, 300, 170], Hq=6, Hkv=2)
    _check(w, [4, 1, 7], 8, acc=[2, 0, 7], layer0=1, n_layers=2)


@pytest.mark.parametrize("max_new,G", [(8, 1), (8, 12), (9, 16), (16, 8), (17, 4), (32, 5), (33, 2), (64, 3), (65, 1),
                                       (70, 4), (129, 2), (300, 1), (1, 33), (2, 40), (1, 64)])
def test_columns_of_a_head(max_new, G):
    w = W.small("columns", L=1, lens=[300, 130], Hq=2 * G, Hkv=2)
    _check(w, [max_new, (max_new + 1) // 2], max_new, acc=[max_new - max_new // 3, (max_new + 1) // 2])


def test_several_groups_of_tiles_and_blocks_of_queries():
    """More token tiles than stay resident, more rows than one block holds."""
    w = W.small("groups", L=1, lens=[1500, 600], Hq=8, Hkv=2)
    _check(w, [200, 131], 200, acc=[190, 131])


def test_more_requests_than_are_ordered():
    lens = [(7 * i) % 40 for i in range(520)]
    w = W.small("requests", L=1, lens=lens, Hq=2, Hkv=1, P=2)
    new = [i % 3 for i in range(520)]
    _check(w, new, 2)


@pytest.mark.parametrize("P", [6, 16])
def test_few_rows_over_bad_tables(P):
    """A contradictory header empties its unit, a page id out of range leaves its page out."""
    w = W.small("few_bad", L=1, lens=[300, 300], Hq=4, Hkv=2, P=P)
    new = [4, 6]
    cap = 320
    dec, sig, _, ctx = make_decoder(w, cap)
    q, k, v = draw_new(w, new, 1, 5)
    dec.tables.unit_hdr[1, 2] += 1
    dec.tables.fwd[2, 1] = dec.pool.F
    dec.tables.fwd[3, 0] = -5
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    before = sig.cpu().numpy()
    dec.extend(q.cuda(), _i32(new), ctx, 6, out, SCALE, k_new=k.cuda(), v_new=v.cuda(), lse=lse)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    dec.extend_significance(q.cuda(), _i32(new), _i32(new), ctx, 6, SCALE, lse, sig, k_new=k.cuda(), v_new=v.cuda())
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    got = sig.cpu().numpy()
    assert np.isfinite(got).all()
    held = got[0, :300, 2:] - before[0, :300, 2:]  # the emptied unit (request 0, head 1): no held token gains
    assert not held.any()


@pytest.mark.parametrize("new", [[5, 8], [40, 30]])
def test_graphs_at_the_same_time(new):
    """Two captured calls with a workspace each, replayed side by side."""
    w = W.small("few_graph", L=1, lens=[2500, 700], Hq=8, Hkv=2)
    most = max(new)
    dec, sig, _, ctx = make_decoder(w, 2560)
    q, k, v = (x.cuda() for x in draw_new(w, new, 1, 9))
    n = _i32(new)

    batch = libdkv.make_extend_batch(1, 2, 2560, q, n, ctx, most, SCALE, k_new=k, v_new=v)
    need = libdkv.dkv_extend_workspace_size(batch, dec.pool, dec.tables)
    assert need > 0

    def call(out, lse, s, ws):
        dec.extend(q, n, ctx, most, out, SCALE, k_new=k, v_new=v, lse=lse, workspace=ws)
        dec.extend_significance(q, n, n, ctx, most, SCALE, lse, s, k_new=k, v_new=v)

    def buffers():
        return (torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"), sig.clone(),
                torch.empty(need, dtype=torch.uint8, device="cuda"))

    eager = buffers()
    call(*eager)
    runs = []
    for _ in range(2):
        side, b, g = torch.cuda.Stream(), buffers(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            call(*b)
        runs.append((side, g, b))
    torch.cuda.synchronize()
    for _ in range(3):
        for side, g, b in runs:
            with torch.cuda.stream(side):
                b[2].copy_(sig)
                g.replay()
    torch.cuda.synchronize()
    for _, _, b in runs:
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(b[:3], eager))
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK


def test_page_operations_on_more_units_than_a_warp_each():
    L, R, Hkv = 16, 300, 4
    lens = [(5 * i) % 23 for i in range(150)] + [0] * 150
    w = W.small("many_units", L=L, lens=lens, Hq=4, Hkv=Hkv, P=2)
    dec, _, _, ctx = make_decoder(w, 32)
    src, dst = list(range(150)), list(range(299, 149, -1))
    want = serial_fork(pool_state(dec.pool, dec.tables), L, R, Hkv, src, dst)
    dec.fork(_i32(src), _i32(dst), ctx)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert_equal(pool_state(dec.pool, dec.tables), want, "fork")
    want = serial_release(want, L, R, Hkv, src)
    dec.release(_i32(src))
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert_equal(pool_state(dec.pool, dec.tables), want, "release")


def test_a_last_wave_in_parts():
    """More row tiles than multiprocessors: the last, incomplete wave is split and merged."""
    w = W.small("waves", L=2, lens=[700, 150, 260], Hq=32, Hkv=8)
    _check(w, [250, 249, 0], 250, acc=[0, 249, 0])  # 48 units x 4 row tiles: a wave of 152 and 40 in halves


def test_many_parts():
    """One unit over a long context: more parts than a warp has lanes."""
    w = W.small("parts", L=1, lens=[30000], Hq=2, Hkv=1)
    _check(w, [7], 8, acc=[4])
    w = W.small("parts64", L=1, lens=[20000], Hq=8, Hkv=1)
    _check(w, [9], 9, acc=[9])
