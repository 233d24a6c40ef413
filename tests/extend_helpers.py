"""Test-side reference of the multi-token attention and its significance, in
float64 from raw page bytes, with the error bounds the library's results are
held to."""
from __future__ import annotations

import numpy as np
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.attention_helpers import U, unit_tokens

SCALE = 0.08838834764831845


def make_decoder(w: W.Workload, cap: int, seed: int = 7, F: int | None = None, device="cuda"):
    """A device Decoder holding the workload's prefill, its significance sums
    [L][R * cap][Hq] and counts [R * cap], and ctx_lens."""
    inp = W.make_inputs(w, seed)
    dec = libdkv.Decoder(w.L, w.R, w.Hq, w.Hkv, cap, w.P, F or 3 * w.pool_pages + 8, device=device, scheme=w.scheme)
    lens = torch.tensor(w.lens, dtype=torch.int32)
    sig = torch.zeros((w.L, w.R * cap, w.Hq))
    cnt = torch.zeros(w.R * cap, dtype=torch.int32)
    t = 0
    for r, n in enumerate(w.lens):
        sig[:, r * cap:r * cap + n] = inp["sig_sum"][:, t:t + n]
        cnt[r * cap:r * cap + n] = inp["sig_cnt"][t:t + n]
        t += n
    if w.T == 0:  # nothing to compact: empty units
        dec.tables.fwd.fill_(-1)
        dec.tables.unit_hdr.zero_()
    for l in range(w.L if w.T else 0):
        layer = {"L": 1, "R": w.R, "Hq": w.Hq, "Hkv": w.Hkv, "T": w.T, "lens": lens.to(device),
                 "sig_cnt": inp["sig_cnt"].to(device)}
        for k in ("k", "v", "sig_sum"):
            layer[k] = inp[k][l:l + 1].contiguous().to(device)
        dec.prefill_layer(layer, l, max(w.lens + [0]), w.alpha_h, w.alpha_l)
    ctx = lens.to(device)
    dec.index(ctx)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    return dec, sig.to(device), cnt.to(device), ctx


def draw_new(w: W.Workload, new_lens, n_layers: int, seed: int, outlier=10.0):
    """q, k_new, v_new bf16 (CPU) of packed new tokens."""
    g = torch.Generator().manual_seed(seed)
    T = int(sum(new_lens))
    q = torch.randn((n_layers, T, w.Hq, 128), generator=g)
    k = torch.randn((n_layers, T, w.Hkv, 128), generator=g)
    v = torch.randn((n_layers, T, w.Hkv, 128), generator=g)
    k[..., 5] *= outlier
    v[..., 77] *= outlier
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


def unit_arrays(st: dict, u: int, P: int, scheme: int):
    """fp64 K, V [n][128], |c| s + |z| of K and positions of a unit's tokens."""
    kq, vq, ks, kz, vs, vz, pos = unit_tokens(st["pages"], st["fwd"][u], st["unit_hdr"][u], P, scheme)
    k = kq * ks[:, None] + kz[:, None]
    v = vq * vs[:, None] + vz[:, None]
    return k, v, kq * ks[:, None] + np.abs(kz)[:, None], pos


def reference(st: dict, w: W.Workload, q, k_new, v_new, new_lens, acc_lens=None, layer0=0, scale=SCALE):
    """out, lse, their bounds, and per (layer, request, head q) the token
    positions' probability sums over the first acc rows with bounds.

    Bounds (u = 2^-24).  A logit is a sum of 128 products of exact factors (a
    code and a bf16 query value), added in fp32 in an order of the hardware's
    choosing with at most 2 u lost per addition, then s (q . c) + z (sum q)
    and the scale: |dx| <= 300 u scale sum_d |q_d| (|c_d| s + |z|), with the
    code taken from its middle (|c| <= 128 <= the form used here).  eta = |dx|
    + u |x - lse| + 2^-19 for the exponential (2^-22 relative) and the
    running rescales.  lse errs by sum_t p eta plus 2^-22 + u |lse|.
    Probabilities enter the value product rounded to fp16 (half a step is
    2^-11 of the value, 2^-32 of the row's largest weight where it is below
    fp16's normal range) against held values rounded to fp16 (2^-11), and as
    the sum of two bf16 values (2^-8 of 2^-8 at most) against the exact bf16
    new values; fp32 sums of n terms add n u.  The result is rounded to bf16: 2^-8."""
    has = k_new is not None  # else the held tokens alone are attended
    q, kn, vn = (x.float().numpy().astype(np.float64) for x in (q, k_new if has else q[:, :0], v_new if has else q[:, :0]))
    nl, T = q.shape[:2]
    G = w.Hq // w.Hkv
    out = np.zeros((nl, T, w.Hq, 128))
    ob = np.zeros_like(out)
    lse = np.full((nl, T, w.Hq), -np.inf)
    lb = np.zeros_like(lse)
    sig = {}
    for li in range(nl):
        t0 = 0
        for r, n in enumerate(new_lens):
            n = int(n)
            acc = 0 if acc_lens is None else int(acc_lens[r])
            for h in range(w.Hkv):
                u = ((layer0 + li) * w.R + r) * w.Hkv + h
                k, v, ka, pos = unit_arrays(st, u, w.P, w.scheme)
                m = len(pos)
                f = n if has else 0
                if has:
                    k = np.concatenate([k, kn[li, t0:t0 + n, h]])
                    v = np.concatenate([v, vn[li, t0:t0 + n, h]])
                    ka = np.concatenate([ka, np.abs(kn[li, t0:t0 + n, h])])
                seen = np.concatenate([np.ones((n, m), bool), np.tril(np.ones((n, n), bool))[:, :f]], 1)
                half = np.concatenate([np.full(m, 2.0 ** -10), np.full(f, 2.0 ** -16)])
                for g in range(G):
                    qh = q[li, t0:t0 + n, h * G + g]
                    if n == 0:
                        continue
                    if m + f == 0:  # nothing attended: 0 and -inf
                        if acc_lens is not None:
                            sig[li, r, h * G + g] = (pos, np.zeros(0), np.zeros(0))
                        continue
                    x = np.where(seen, scale * (qh @ k.T), -np.inf)
                    mx = x.max(1, keepdims=True)
                    e = np.exp(x - mx)
                    s = e.sum(1, keepdims=True)
                    p = e / s
                    ls = mx + np.log(s)
                    eta = np.where(seen, 300 * U * scale * (np.abs(qh) @ ka.T) + U * np.minimum(ls - x, 200.0)
                                   + 2.0 ** -19, 0.0)
                    both = np.expm1((p * eta).sum(1, keepdims=True))
                    rho = np.where(seen, np.expm1(eta) + both + (m + n + 32) * U, 0.0)
                    o = p @ v
                    out[li, t0:t0 + n, h * G + g] = o
                    lse[li, t0:t0 + n, h * G + g] = ls[:, 0]
                    raw = (p * (rho * 1.02 + half * 1.02) + seen * (2.0 ** -31 * p.max(1, keepdims=True))) @ np.abs(v)
                    ob[li, t0:t0 + n, h * G + g] = raw * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o)
                    lb[li, t0:t0 + n, h * G + g] = (1.01 * both + 2.0 ** -21 + 2 * U * np.abs(ls) +
                                                    (m + n + 32) * U)[:, 0]
                    if acc_lens is not None:
                        # the recomputed p uses the library's lse: its error counts too
                        pa, ra = p[:acc], rho[:acc] + 1.01 * lb[li, t0:t0 + acc, h * G + g][:, None]
                        sig[li, r, h * G + g] = (pos, pa.sum(0), (pa * ra).sum(0) + (acc + 4) * U * pa.sum(0))
            t0 += n
    return out, ob, lse, lb, sig


def check_attention(out, lse, ref, what=""):
    o, ob, ls, lb, _ = ref
    got = out.float().cpu().numpy().astype(np.float64)
    err = np.abs(got - o)
    assert np.all(np.isfinite(got)), f"{what}: outputs that are not finite"
    assert np.all(err <= ob), f"{what}: out off by {(err / np.maximum(ob, 1e-300)).max():.3g} of its bound"
    if lse is not None:
        gl = lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isfinite(gl), np.isfinite(ls)), f"{what}: which rows attend nothing"
        fin = np.isfinite(ls)
        el = np.abs(gl[fin] - ls[fin])
        assert np.all(el <= lb[fin]), f"{what}: lse off by {(el / lb[fin]).max():.3g} of its bound"


def check_significance(got: np.ndarray, before: np.ndarray, ref, w, cap, ctx, acc_lens, layer0=0, new=True, what=""):
    """sig_sum rows after the call against before + the reference's sums; rows
    of nothing attended are bit-equal."""
    sig = ref[4]
    seen = np.zeros(got.shape, bool)
    for (li, r, q), (pos, p, b) in sig.items():
        acc, m = int(acc_lens[r]), len(pos)
        l, base = layer0 + li, r * cap
        if acc == 0:
            continue
        rows = base + pos
        seen[l, rows, q] = True
        want = before[l, rows, q].astype(np.float64) + p[:m]
        err = np.abs(got[l, rows, q] - want)
        assert np.all(err <= b[:m] + 2 * U * np.abs(want)), f"{what}: held rows of ({li}, {r}, {q})"
        if new:
            rows = base + int(ctx[r]) + np.arange(acc)
            seen[l, rows, q] = True
            err = np.abs(got[l, rows, q] - p[m:m + acc])
            assert np.all(err <= b[m:m + acc] + 2 * U * p[m:m + acc]), f"{what}: new rows of ({li}, {r}, {q})"
    assert np.array_equal(got[~seen], before[~seen]), f"{what}: rows that nothing attends changed"
