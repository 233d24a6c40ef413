"""The running reference of a row's softmax in the multi-token attention: where
it starts and where it has to move, for every kernel (at most 32 rows a unit, at
most 128, more)."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, check_attention, check_significance, reference
from tests.extend_logits import decoder_of, keys_of, queries_of
from tests.page_ops_helpers import pool_state

pytestmark = pytest.mark.gpu

LENS = [300, 170]
# new tokens with four query heads a group: 32, 128 and 320 rows a unit and a
# second request whose rows fill whole warps as well
NEW = {"few": [8, 8], "128 rows": [32, 16], "more": [80, 64]}
LISTS = {"high": (0.0, 0.0), "low": (1e9, 0.0)}


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _check(new, held, fresh, scheme=0, lists="high", what=""):
    """Levels of the held tokens and of the new ones (None: none are given) by
    their index; the attention and its significance against float64."""
    ah, al = LISTS[lists]
    w = W.small("levels", L=1, lens=LENS, Hq=8, Hkv=2, P=16, scheme=scheme, alpha_h=ah, alpha_l=al, n_outlier=0)
    cap = 400
    dec, sig, ctx = decoder_of(w, cap, keys_of([held(t) for n in LENS for t in range(n)], w.Hkv, 1, 3))
    T = sum(new)
    q = queries_of(T, w.Hq, 1, 4)
    k = v = None
    if fresh is not None:
        k = keys_of([fresh(t) for n in new for t in range(n)], w.Hkv, 1, 5)
        v = torch.randn((1, T, w.Hkv, 128), generator=torch.Generator().manual_seed(6)).bfloat16()
    state, before = pool_state(dec.pool, dec.tables), sig.cpu().numpy()
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    qc, kc, vc = (None if x is None else x.cuda() for x in (q, k, v))
    dec.extend(qc, _i32(new), ctx, max(new), out, SCALE, k_new=kc, v_new=vc, lse=lse)
    dec.extend_significance(qc, _i32(new), _i32(new), ctx, max(new), SCALE, lse, sig, k_new=kc, v_new=vc)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    ref = reference(state, w, q, k, v, new, new)
    check_attention(out, lse, ref, what)
    check_significance(sig.cpu().numpy(), before, ref, w, cap, LENS, new, new=k is not None, what=what)


@pytest.mark.parametrize("lists", list(LISTS))
@pytest.mark.parametrize("scheme", [0, 1, 2])
@pytest.mark.parametrize("rows", list(NEW))
def test_logits_that_grow_from_one_piece_of_a_tile_to_the_next(rows, scheme, lists):
    """6.5 more every 32 tokens: the references move several times in a tile,
    over weights and outputs that are already there."""
    _check(NEW[rows], lambda t: 6.5 * (t // 32), lambda t: 6.5 * (t // 32 + 4), scheme, lists, f"{rows} {lists}")


@pytest.mark.parametrize("with_new", [False, True])
@pytest.mark.parametrize("lists", list(LISTS))
@pytest.mark.parametrize("level", [-100.0, -1000.0])
@pytest.mark.parametrize("rows", list(NEW))
def test_logits_that_are_all_far_below_zero(rows, level, lists, with_new):
    """Keys with a common part against queries: every logit of every row lies
    below the smallest weight against 0, and the softmax is an ordinary one."""
    _check(NEW[rows], lambda t: level, (lambda t: level) if with_new else None, 0, lists, f"{rows} {level}")


@pytest.mark.parametrize("rows", list(NEW))
def test_first_tokens_below_the_smallest_weight_and_the_rest_above(rows):
    """Three quarters of the context at -92, the rest at -84: log2 units -132.7
    and -121.2 around the -126 below which a weight against 0 is none."""
    _check(NEW[rows], lambda t: -92.0 if t < 225 else -84.0, None, what=rows)
    _check(NEW[rows], lambda t: -87.6 if t < 225 else -87.0, None, what=rows)


@pytest.mark.parametrize("with_new", [False, True])
@pytest.mark.parametrize("rows", list(NEW))
def test_first_piece_below_and_the_first_tile_below(rows, with_new):
    for edge in (32, 128):
        _check(NEW[rows], lambda t: -120.0 if t < edge else -88.0, (lambda t: -110.0 + t % 7) if with_new else None,
               what=f"{rows} {edge}")
