"""Where an item has one row tile (128 / G tokens or fewer are left) the weights
enter the second product as the sum of two bf16 values.  The values here cancel
in one channel of every row, so that neither the output's own rounding nor its
size hides what the weights lost."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from tests.chunk_helpers import SCALE, Chunk, U

CASES = {
    # up to 16 rows: four times in the row tile
    "one row": dict(Hq=3, Hkv=3, ctx=40, new=1),
    "one row over several tiles": dict(Hq=2, Hkv=2, ctx=300, new=1),
    "twelve rows": dict(Hq=8, Hkv=2, ctx=30, new=3),
    "sixteen rows": dict(Hq=8, Hkv=1, ctx=130, new=2),
    "one row, a late maximum": dict(Hq=2, Hkv=2, ctx=128, new=1, high=(99, 120)),
    # more: one row tile
    "a hundred rows": dict(Hq=1, Hkv=1, ctx=20, new=100),
    "groups of 4": dict(Hq=8, Hkv=2, ctx=45, new=20),
    "groups of 7": dict(Hq=14, Hkv=2, ctx=9, new=18),
    "groups of 128": dict(Hq=128, Hkv=1, ctx=50, new=1),
    "several tiles": dict(Hq=4, Hkv=2, ctx=600, new=30),
    "a late maximum": dict(Hq=4, Hkv=1, ctx=128, new=9, high=(99, 120)),
    "a late maximum in the second tile": dict(Hq=4, Hkv=1, ctx=256, new=9, high=(201, 250)),
    # the last item of a chunk of several
    "what two row tiles leave": dict(Hq=8, Hkv=2, ctx=5, new=64 + 20),
}


def _setup(Hq, Hkv, ctx, new, high=()):
    """The inputs and, per row, outputs in float64 and the bound, both [new][Hq][128], with P [new][Hq][ctx + new].

    The weight of a position is rounded to bf16, half a step of which is 2^-8, and so is what that left of it, 2^-8 of
    2^-8; else as in Chunk.reference.  The products are added 16 at a time: 17 terms that lose at most 2 u each of the
    largest, for both halves 5 u a term.  Rows of items with two row tiles are bounded by 2^-8 alone."""
    G, tpt = Hq // Hkv, 128 // (Hq // Hkv)
    c = Chunk(Hq, Hkv, 16, [ctx], [new], seed=ctx + new, outlier=1.0)
    c.q = (c.q.float() * 0.1).bfloat16()
    c.q[..., 0] = 8.0 if high else 0.1
    place = lambda p: (0, int(c.table[0, p // 16]), p % 16)  # noqa: E731
    c.kn[..., 0] = 0
    for p in range(ctx):
        c.k[place(p)][:, 0] = 20.0 if p in high else 0.0  # 14 above the others: 20 octaves
    k, _ = c.appended()
    anchor = high[-1] if high else 3  # its value cancels the others'
    P = np.zeros((new, Hq, ctx + new))
    eta = np.zeros_like(P)
    kr = c.rows(k, 0, 0)
    seen = np.arange(ctx + new) <= ctx + np.arange(new)[:, None]
    for h in range(Hq):
        q = c.q[0, :, h].double().numpy()
        x = np.where(seen, SCALE * (q @ kr[:, h // G].T), -np.inf)
        mx = x.max(1, keepdims=True)
        e = np.exp(x - mx)
        P[:, h] = e / e.sum(1, keepdims=True)
        dx = 300 * U * SCALE * (np.abs(q) @ np.abs(kr[:, h // G]).T)
        eta[:, h] = np.where(seen, dx + 2 * U * np.minimum(mx + np.log(e.sum(1, keepdims=True)) - x, 200.0) + 2.0 ** -19, 0.0)
    first = new // (2 * tpt) * 2 * tpt  # of the last item
    rows = range(first, new) if new - first <= tpt else range(0)
    for h in range(Hkv):  # row j of the item cancels in channel j
        v = torch.cat([torch.stack([c.v[place(p)][h] for p in range(ctx)]), c.vn[0, :, h]]).double().numpy()
        at = c.v[place(anchor)][h]
        for j, (i, g) in enumerate((i, g) for i in rows for g in range(G)):
            p = P[i, h * G + g]
            at[j] = float(v[anchor, j] - p @ v[:, j] / p[anchor])
    _, v = c.appended()
    vr = c.rows(v, 0, 0)
    out, bound = np.zeros((new, Hq, 128)), np.zeros((new, Hq, 128))
    for h in range(Hq):
        both = np.expm1((P[:, h] * eta[:, h]).sum(1, keepdims=True))
        rho = np.where(seen, np.expm1(eta[:, h]) + both + 5 * (ctx + new + 32) * U, 0.0)
        lost = np.full((new, 1), 2.0 ** -8)
        lost[list(rows)] = 2.0 ** -16
        out[:, h] = P[:, h] @ vr[:, h // G]
        raw = (P[:, h] * (1.02 * rho + 1.02 * lost) + seen * 2.0 ** -120) @ np.abs(vr[:, h // G])
        bound[:, h] = raw * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(out[:, h])
    return c, list(rows), P, vr, out, bound


def _bf16(x):
    return torch.tensor(x, dtype=torch.float64).float().bfloat16().double().numpy()


def _outside(name, weights):
    """Of the entries that cancel, how many are outside the bound under these weights (of the exact ones, their largest
    1), and how many there are."""
    c, rows, P, vr, out, bound = _setup(**CASES[name])
    assert rows
    G, bad, n = c.Hq // c.Hkv, 0, 0
    for h in range(c.Hq):
        for j, i in enumerate(rows):
            ch, w = j * G + h % G, P[i, h] / P[i, h].max()
            bad += abs(weights(w) @ vr[:, h // G, ch] / w.sum() - out[i, h, ch]) > bound[i, h, ch]
            n += 1
    return bad, n


@pytest.mark.parametrize("name", CASES)
def test_two_bf16_values_stay_within_the_bound(name):
    assert _outside(name, lambda w: _bf16(w) + _bf16(w - _bf16(w)))[0] == 0


@pytest.mark.parametrize("name", [n for n, c in CASES.items() if c["ctx"] <= 50])
def test_one_bf16_value_leaves_the_bound(name):
    bad, n = _outside(name, _bf16)
    assert bad > 0.5 * n


def test_what_is_left_of_earlier_weights_follows_the_reference():
    """Position 99 moves the reference of its tile by 20 octaves; the second halves of the 96 weights before stay."""
    def stale(w):
        rest = _bf16(w - _bf16(w))
        rest[:96] *= 2.0 ** 20
        return _bf16(w) + rest

    bad, n = _outside("a late maximum", stale)
    assert bad > 0.5 * n


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_weights_of_one_row_tile_are_two_bf16_values(name):
    c, rows, _, _, out, bound = _setup(**CASES[name])
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    err = np.abs(d["out"][0].double().cpu().numpy() - out)
    assert np.all(err <= bound), f"off by {(err / bound).max():.3g} of the bound"
