"""Rows of the multi-token attention are independent: a query of any finite size
leaves the rows beside it (of other heads, tokens and requests of its block) as
they are, for every kernel."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, check_significance, draw_new, make_decoder, reference, unit_arrays
from tests.page_ops_helpers import pool_state

pytestmark = pytest.mark.gpu

NEW = {"few": [8, 3], "128 rows": [32, 20], "more": [80, 64]}
HUGE = (1, 1)  # token (of request 0) and query head of the row


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("scheme", [0, 1, 2])
@pytest.mark.parametrize("size", [1e6, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("rows", list(NEW))
def test_one_large_query(rows, size, scheme):
    new, (tok, head) = NEW[rows], HUGE
    w = W.small("range", L=1, lens=[300, 170], Hq=8, Hkv=2, P=16, scheme=scheme, alpha_h=0.3, alpha_l=0.0)
    dec, sig, _, ctx = make_decoder(w, 400)
    q, k, v = draw_new(w, new, 1, 9)
    big = q.clone()
    big[0, tok, head] = (big[0, tok, head].float() * size).bfloat16()
    st, before = pool_state(dec.pool, dec.tables), sig.cpu().numpy()
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    qc, kc, vc = big.cuda(), k.cuda(), v.cuda()
    dec.extend(qc, _i32(new), ctx, max(new), out, SCALE, k_new=kc, v_new=vc, lse=lse)
    dec.extend_significance(qc, _i32(new), _i32(new), ctx, max(new), SCALE, lse, sig, k_new=kc, v_new=vc)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    got, gl, gs = out.float().cpu().numpy(), lse.cpu().numpy(), sig.cpu().numpy()
    # the other rows: those of the call without the large query
    o, ob, ls, lb, sums = reference(st, w, q, k, v, new, new)
    rest = np.ones(o.shape[:3], bool)
    rest[0, tok, head] = False
    assert np.all(np.abs(got[rest] - o[rest]) <= ob[rest])
    assert np.all(np.abs(gl[rest] - ls[rest]) <= lb[rest])
    # its own: the value of its largest logit's token (logits this far apart leave the others nothing)
    kk, vv, _, pos = unit_arrays(st, 0, w.P, w.scheme)
    n = tok + 1
    kk = np.concatenate([kk, k[0, :n, 0].float().numpy().astype(np.float64)])
    vv = np.concatenate([vv, v[0, :n, 0].float().numpy().astype(np.float64)])
    x = SCALE * (kk @ big[0, tok, head].float().numpy().astype(np.float64))
    first, second = np.sort(x)[::-1][:2]
    mine = got[0, tok, head]
    assert first - second > 1e-4 * abs(first)  # a margin that the rounding of such logits does not reach
    assert np.all(np.abs(mine - vv[x.argmax()]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(vv[x.argmax()]))
    assert abs(gl[0, tok, head] - first) <= 1e-4 * abs(first)
    # significance: heads without it as ever; at its own each token has 0 to 1 more than from the other rows
    keep = {x: y for x, y in sums.items() if x[2] != head}
    seen = gs.copy()
    seen[..., head] = before[..., head]
    check_significance(seen, before, (None, None, None, None, keep), w, 400, [300, 170], new)
    assert np.isfinite(gs).all()
    pos, p, b = reference(st, w, q, k, v, new, [tok, 0])[4][0, 0, head]
    own, d = before[0, pos, head] + p[:len(pos)], gs[0, pos, head]
    after = reference(st, w, q, k, v, new, new)[4][0, 0, head][1][:len(pos)]
    slack = 1e-3 * (1 + after)
    assert np.all(d >= own - slack) and np.all(d <= before[0, pos, head] + after + 1 + slack)


@pytest.mark.parametrize("size", [1e6, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("rows", list(NEW))
def test_one_large_new_key_and_one_large_new_value(rows, size):
    """Rows before the key do not see it; a row after it takes its value alone or
    not at all, by the sign of the logit.  Values are linear."""
    new = NEW[rows]
    w = W.small("range", L=1, lens=[300, 170], Hq=8, Hkv=2, P=16, alpha_h=0.3, alpha_l=0.0)
    dec, _, _, ctx = make_decoder(w, 400)
    q, k, v = draw_new(w, new, 1, 9)
    tok = 2
    k[0, tok, 1] = (k[0, tok, 1].float() * size).bfloat16()
    v[0, tok, 1, 3] = size
    st = pool_state(dec.pool, dec.tables)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    dec.extend(q.cuda(), _i32(new), ctx, max(new), out, SCALE, k_new=k.cuda(), v_new=v.cuda(), lse=lse)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    got, gl = out[0, :new[0]].float().cpu().numpy(), lse[0, :new[0]].cpu().numpy()
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    qd, kd, vd = (x[0, :new[0]].float().numpy().astype(np.float64) for x in (q, k, v))
    for h in range(8):
        kk, vv, _, _ = unit_arrays(st, h // 4, w.P, 0)
        kk, vv = np.concatenate([kk, kd[:, h // 4]]), np.concatenate([vv, vd[:, h // 4]])
        x = SCALE * (qd[:, h] @ kk.T)
        x[:, -new[0]:] = np.where(np.tril(np.ones((new[0], new[0]), bool)), x[:, -new[0]:], -np.inf)
        mx = x.max(1, keepdims=True)
        p = np.exp(x - mx)
        s = p.sum(1, keepdims=True)
        p /= s
        # half a step of bf16 of the result; fp16 weights and values, and logits of
        # up to 60 that 300 additions leave 2^-10 uncertain: 2^-8 of the terms
        assert np.all(np.abs(got[:, h] - p @ vv) <= 2.0 ** -8 * np.abs(p @ vv) + 2.0 ** -8 * (p @ np.abs(vv))), h
        ls = (mx + np.log(s))[:, 0]
        assert np.all(np.abs(gl[:, h] - ls) <= 2.0 ** -10 + 1e-4 * np.abs(ls)), h
