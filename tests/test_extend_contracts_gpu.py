"""What the multi-token calls promise about wrong inputs, for every kernel (at
most 32 rows a unit, at most 128, more): lengths that contradict one another
write nothing, headers and page ids that contradict the tables leave their
tokens out and nothing else, new values that are not finite count as 0, a query
that is not finite spoils its own row."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, check_attention, check_significance, draw_new, make_decoder, reference
from tests.page_ops_helpers import pool_state

pytestmark = pytest.mark.gpu

# two query heads a group: 8, 80 and 400 rows a unit
NEW = {"few": [4, 3], "128 rows": [40, 30], "more": [200, 150]}


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _decoder(P, scheme=0, lens=(300, 310)):
    w = W.small("contracts", L=1, lens=list(lens), Hq=4, Hkv=2, P=P, scheme=scheme)
    return (w, *make_decoder(w, 528))


@pytest.mark.parametrize("rows", list(NEW))
def test_lengths_that_contradict_one_another_write_nothing(rows):
    a, b = NEW[rows]
    w, dec, sig, _, ctx = _decoder(16)
    q, k, v = (x.cuda() for x in draw_new(w, [a, b], 1, 2))
    most = max(a, b) + 2
    before = sig.clone()
    lse = torch.zeros(q.shape[:3], device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    for new, held, mx in (([a, b - 1], [300, 310], most), ([a, b], [300, 310], a - 1), ([-1, a + b + 1], [300, 310], a + b + 1),
                          ([a, b], [300, 529 - b], most), ([a, b], [-1, 310], most), ([a + 1, b], [300, 310], most)):
        dec.extend(q, _i32(new), _i32(held), mx, out, SCALE, k_new=k, v_new=v, lse=lse)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_LENS, (new, held, mx)
        assert bool((out == 7.0).all()) and not lse.any(), (new, held, mx)
        dec.extend_significance(q, _i32(new), _i32([0, 0]), _i32(held), mx, SCALE, lse, sig, k_new=k, v_new=v)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_LENS, (new, held, mx)
        assert torch.equal(sig, before)
    for acc in ([a + 1, b], [-1, 0]):
        dec.extend_significance(q, _i32([a, b]), _i32(acc), ctx, most, SCALE, lse, sig, k_new=k, v_new=v)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_LENS
        assert torch.equal(sig, before)


def _without_page(st, u, P, low, j):
    """The state whose unit u has lost page j of a list (not the list's last)."""
    st = {**st, "fwd": st["fwd"].copy(), "unit_hdr": st["unit_hdr"].copy()}
    h = st["unit_hdr"][u]
    at = j + (int(h[2]) if low else 0)
    st["fwd"][u, at:-1] = st["fwd"][u, at + 1:].copy()
    h[1 if low else 0] -= 2 * P if low else P
    h[3 if low else 2] -= 1
    return st


@pytest.mark.parametrize("scheme", [0, 1, 2])
@pytest.mark.parametrize("P", [6, 16])
@pytest.mark.parametrize("rows", list(NEW))
def test_tables_that_contradict_one_another(rows, P, scheme):
    new = NEW[rows]
    w, dec, sig, _, ctx = _decoder(P, scheme)
    q, k, v = draw_new(w, new, 1, 5)
    st = pool_state(dec.pool, dec.tables)
    hdr = st["unit_hdr"]
    assert (hdr[:, 2:] >= 3).all()  # pages enough to lose one in the middle of a list
    want = {**st, "unit_hdr": hdr.copy()}
    want["unit_hdr"][1] = 0
    want = _without_page(want, 0, P, False, 1)
    want = _without_page(want, 2, P, True, 0)
    want = _without_page(want, 3, P, True, 1)
    want = _without_page(want, 3, P, False, 0)
    dec.tables.unit_hdr[1, 2] += 1
    dec.tables.fwd[0, 1] = dec.pool.F
    dec.tables.fwd[2, int(hdr[2, 2])] = -5
    dec.tables.fwd[3, int(hdr[3, 2]) + 1] = 2 ** 31 - 1
    dec.tables.fwd[3, 0] = -2 ** 31
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    before = sig.cpu().numpy()
    qc, kc, vc = q.cuda(), k.cuda(), v.cuda()
    dec.extend(qc, _i32(new), ctx, max(new), out, SCALE, k_new=kc, v_new=vc, lse=lse)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    ref = reference(want, w, q, k, v, new, new)
    check_attention(out, lse, ref, rows)
    dec.extend_significance(qc, _i32(new), _i32(new), ctx, max(new), SCALE, lse, sig, k_new=kc, v_new=vc)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    check_significance(sig.cpu().numpy(), before, ref, w, 528, w.lens, new, what=rows)


@pytest.mark.parametrize("rows", list(NEW))
def test_values_that_are_not_finite(rows):
    new = NEW[rows]
    w, dec, sig, _, ctx = _decoder(16, lens=(60, 310))
    q, k, v = draw_new(w, new, 1, 2)
    st, tok = pool_state(dec.pool, dec.tables), new[0] - 1

    def run(q, k, v):
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        dec.extend(q.cuda(), _i32(new), ctx, max(new), out, SCALE, k_new=k.cuda(), v_new=v.cuda(), lse=lse)
        return out, lse

    for t in (k, v):
        for x in (float("nan"), float("inf"), float("-inf")):
            bad, zero = t.clone(), t.clone()
            bad[0, tok, 1, 9], zero[0, tok, 1, 9] = x, 0.0
            out, lse = run(q, *((bad, v) if t is k else (k, bad)))
            assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_RANGE
            check_attention(out, lse, reference(st, w, q, *((zero, v) if t is k else (k, zero)), new), "taken as 0")
    o, ob, ls, lb, _ = reference(st, w, q, k, v, new)
    rest = np.ones(o.shape[:3], bool)
    rest[0, tok, 1] = False
    for x in (float("nan"), float("inf"), float("-inf")):
        qq = q.clone()
        qq[0, tok, 1, 3] = x
        out, lse = run(qq, k, v)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
        assert np.all(np.abs(got[rest] - o[rest]) <= ob[rest]) and np.all(np.abs(gl[rest] - ls[rest]) <= lb[rest])
