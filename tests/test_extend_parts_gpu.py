"""Requests with equally many new tokens whose row tiles leave the last wave of
blocks incomplete: that wave's tiles are attended in parts and joined; the
widest group; equal bits every time."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, check_attention, check_significance, draw_new, make_decoder, reference
from tests.page_ops_helpers import pool_state

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _check(w, new, acc, held_only=False, parts=None):
    cap = -(-(max(w.lens) + max(new)) // 16) * 16
    dec, sig, _, ctx = make_decoder(w, cap)
    q, k, v = draw_new(w, new, w.L, 3)
    if held_only:
        k = v = None
    before, state = sig.cpu().numpy(), pool_state(dec.pool, dec.tables)
    qc, kc, vc = (None if x is None else x.cuda() for x in (q, k, v))
    if parts is not None:  # partial results need a workspace, whole rows none
        b = libdkv.make_extend_batch(w.L, w.Hkv, cap, qc, _i32(new), ctx, max(new), SCALE)
        assert (libdkv.dkv_extend_workspace_size(b, dec.pool, dec.tables) > 0) == parts
    outs = []
    for _ in range(3):
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        dec.extend(qc, _i32(new), ctx, max(new), out, SCALE, k_new=kc, v_new=vc, lse=lse)
        outs.append((out, lse))
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o, outs[0]))
    dec.extend_significance(qc, _i32(new), _i32(acc), ctx, max(new), SCALE, lse, sig, k_new=kc, v_new=vc)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    ref = reference(state, w, q, k, v, new, acc)
    check_attention(*outs[0], ref)
    check_significance(sig.cpu().numpy(), before, ref, w, cap, w.lens, acc, new=k is not None)


@pytest.mark.parametrize("held_only", [False, True])
@pytest.mark.parametrize("scheme", [0, 1, 2])
def test_equal_chunks_in_parts(scheme, held_only):
    # 2 layers x 3 requests x 8 heads of 4 row tiles: a wave of 152 and 40 in thirds
    w = W.small("parts", L=2, lens=[900, 150, 1], Hq=32, Hkv=8, scheme=scheme)
    _check(w, [250, 250, 250], [3, 250, 0], held_only, parts=True)


def test_an_equal_chunk_of_one_token_less_is_ragged():
    w = W.small("parts", L=2, lens=[900, 150, 1], Hq=32, Hkv=8)
    _check(w, [250, 249, 250], [3, 0, 250], parts=False)


@pytest.mark.parametrize("new", [[1, 1], [2, 1], [3, 3]])
def test_the_widest_group(new):
    w = W.small("widest", L=1, lens=[300, 40], Hq=128, Hkv=1)
    _check(w, new, [n - 1 for n in new])
