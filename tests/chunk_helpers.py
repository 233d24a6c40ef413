"""Test-side reference of the attention of a chunk over bf16 pages and of its
significance, in float64, with the error bounds the library's results are held
to; and a serial restatement of the eviction over numpy copies of a state."""
from __future__ import annotations

import numpy as np
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from tests.page_ops_helpers import copy_state

U = 2.0 ** -24
SCALE = 0.08838834764831845


class Chunk:
    """Inputs of one call: pages that hold ctx tokens of each request, scattered, with NaN in every slot that holds
    none and table entries that name no page behind the last token."""

    def __init__(self, Hq, Hkv, B, ctx, new, seed=0, L=1, layer0=0, n_layers=1, fused=False, outlier=8.0, room=3):
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hkv, self.B, self.L, self.layer0, self.n_layers = Hq, Hkv, B, L, layer0, n_layers
        self.ctx, self.new, self.R, self.T = list(ctx), list(new), len(ctx), int(sum(new))
        self.cap = -(-max([c + n for c, n in zip(ctx, new)] + [1]) // 16) * 16
        tmax = -(-self.cap // B)
        used = [-(-(c + n) // B) for c, n in zip(ctx, new)]
        F = sum(used) + room
        order = torch.randperm(F, generator=g)
        self.table = torch.full((self.R, tmax), 2 ** 31 - 1, dtype=torch.int32)
        t = 0
        for r, n in enumerate(used):
            self.table[r, :n] = order[t:t + n].to(torch.int32)
            t += n
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.k = torch.full((L, F, B, Hkv, 128), float("nan"), dtype=torch.bfloat16)
        self.v = self.k.clone()
        for r, c in enumerate(self.ctx):
            for p in range(0, c, B):
                m = min(B, c - p)
                id_ = int(self.table[r, p // B])
                for x, ch in ((self.k, 5), (self.v, 77)):
                    y = rand(L, m, Hkv, 128)
                    y[..., ch] *= outlier
                    x[:, id_, :m] = y.bfloat16()
        rows = rand(n_layers, self.T, Hq + 2 * Hkv, 128)
        rows[:, :, Hq:Hq + Hkv, 5] *= outlier
        rows[:, :, Hq + Hkv:, 77] *= outlier
        rows = rows.bfloat16()
        self.q, self.kn, self.vn = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
        self.fused = fused
        if not fused:
            self.q, self.kn, self.vn = self.q.contiguous(), self.kn.contiguous(), self.vn.contiguous()
        self.max_new = max(self.new + [0])

    def device(self, **over):
        """Device tensors, the pages object, the pool and the batch (entries of `over` replace the batch's)."""
        d = {n: getattr(self, n).cuda() for n in ("k", "v", "table")}
        if self.fused:
            rows = torch.cat([self.q, self.kn, self.vn], 2).cuda()
            d["q"], d["kn"], d["vn"] = rows.split([self.Hq, self.Hkv, self.Hkv], 2)
        else:
            d.update({n: getattr(self, n).cuda() for n in ("q", "kn", "vn")})
        d["new"], d["ctx"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.new, self.ctx))
        d["out"] = torch.full((self.n_layers, self.T, self.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        d["lse"] = torch.full((self.n_layers, self.T, self.Hq), 7.0, device="cuda")
        d.update(over)
        d["pool"] = libdkv.DevicePool(1, 2)
        d["pages"] = libdkv.ChunkPages.from_tensors(d["k"], d["v"], d["table"])
        d["batch"] = libdkv.make_chunk_batch(self.Hkv, self.cap, d["q"], d["new"], d["ctx"],
                                             d.get("max_new", self.max_new), d.get("scale", SCALE), k_new=d["kn"],
                                             v_new=d["vn"], out=d["out"], lse=d["lse"], layer0=self.layer0, L=self.L)
        n = libdkv.dkv_chunk_workspace_size(d["batch"], d["pages"])
        d["ws"] = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
        return d

    def attend(self, d, stream=None):
        libdkv.dkv_chunk_attention(d["batch"], d["pages"], d["pool"], d["ws"], stream=stream)
        return libdkv.dkv_get_status(d["pool"], stream=stream)

    def appended(self):
        """The pages after the call."""
        k, v = self.k.clone(), self.v.clone()
        t = 0
        for r, (c, n) in enumerate(zip(self.ctx, self.new)):
            for i in range(n):
                id_, s = int(self.table[r, (c + i) // self.B]), (c + i) % self.B
                k[self.layer0:self.layer0 + self.n_layers, id_, s] = self.kn[:, t + i]
                v[self.layer0:self.layer0 + self.n_layers, id_, s] = self.vn[:, t + i]
            t += n
        return k, v

    def rows(self, x, r, li):
        """fp64 rows [ctx + new][Hkv][128] of request r in layer layer0 + li of the appended pages x."""
        n = self.ctx[r] + self.new[r]
        ids = self.table[r, :-(-n // self.B)].long()
        return x[self.layer0 + li, ids].flatten(0, 1)[:n].double().numpy()

    def reference(self, scale=SCALE, lse_in=None):
        """out, its bound, lse, its bound; with lse_in (the library's lse) also {(li, r): (sums [N][Hq], bound)}.

        Bounds (u = 2^-24).  A logit is a sum of 128 exact products, added in fp32 in an order of the hardware's
        choosing with at most 2 u lost per addition, then times the scale: |dx| <= 300 u scale sum_d |q_d| |k_d|.
        eta = |dx| + 2 u |x - lse| + 2^-19 for the exponential (2^-22 relative) and the rescales.  lse errs by
        sum_t p eta + 2^-21 + 2 u |lse|.  The weights enter the value product as bf16, half a step of which is 2^-8
        of the value; fp32 sums of n terms add n u; the result is rounded to bf16, 2^-8.  A recomputed
        p = exp(x - lse) errs by eta + 3 u |lse| and a sum of n of them by n u more."""
        k, v = self.appended()
        out = np.zeros((self.n_layers, self.T, self.Hq, 128))
        ob, lse = np.zeros_like(out), np.zeros((self.n_layers, self.T, self.Hq))
        lb, sig = np.zeros_like(lse), {}
        G = self.Hq // self.Hkv
        q = self.q.double().numpy()
        for li in range(self.n_layers):
            t0 = 0
            for r, (c, n) in enumerate(zip(self.ctx, self.new)):
                if n == 0:
                    continue
                kr, vr = self.rows(k, r, li), self.rows(v, r, li)
                seen = np.arange(c + n) <= c + np.arange(n)[:, None]
                sums = np.zeros((c + n, self.Hq))
                sb = np.zeros_like(sums)
                for h in range(self.Hq):
                    qh, kh, vh = q[li, t0:t0 + n, h], kr[:, h // G], vr[:, h // G]
                    x = np.where(seen, scale * (qh @ kh.T), -np.inf)
                    mx = x.max(1, keepdims=True)
                    e = np.exp(x - mx)
                    s = e.sum(1, keepdims=True)
                    p, ls = e / s, mx + np.log(s)
                    dx = 300 * U * scale * (np.abs(qh) @ np.abs(kh).T)
                    eta = np.where(seen, dx + 2 * U * np.minimum(ls - x, 200.0) + 2.0 ** -19, 0.0)
                    both = np.expm1((p * eta).sum(1, keepdims=True))
                    rho = np.where(seen, np.expm1(eta) + both + (c + n + 32) * U, 0.0)
                    o = p @ vh
                    out[li, t0:t0 + n, h], lse[li, t0:t0 + n, h] = o, ls[:, 0]
                    raw = (p * (1.02 * rho + 1.02 * 2.0 ** -8) + seen * 2.0 ** -120) @ np.abs(vh)
                    ob[li, t0:t0 + n, h] = raw * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o)
                    lb[li, t0:t0 + n, h] = (1.01 * both + 2.0 ** -21 + 2 * U * np.abs(ls) + (c + n + 32) * U)[:, 0]
                    if lse_in is not None:
                        given = lse_in[li, t0:t0 + n, h].astype(np.float64)[:, None]
                        p = np.where(seen, np.exp(x - given), 0.0)
                        sums[:, h] = p.sum(0)
                        sb[:, h] = (p * (np.expm1(eta + 3 * U * np.abs(given)) + (n + 8) * U)).sum(0) + n * 2.0 ** -126
                sig[li, r] = (sums, sb)
                t0 += n
        return out, ob, lse, lb, sig

    def check(self, d, ref, what=""):
        out, ob, lse, lb, _ = ref
        got = d["out"].float().cpu().numpy().astype(np.float64)
        assert np.all(np.isfinite(got)), f"{what}: outputs that are not finite"
        err = np.abs(got - out)
        assert np.all(err <= ob), f"{what}: out off by {(err / np.maximum(ob, 1e-300)).max():.3g} of its bound"
        if d["lse"] is not None:
            el = np.abs(d["lse"].cpu().numpy().astype(np.float64) - lse)
            assert np.all(el <= lb), f"{what}: lse off by {(el / lb).max():.3g} of its bound"
        k, v = self.appended()
        bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
        assert torch.equal(bits(d["k"]), bits(k)) and torch.equal(bits(d["v"]), bits(v)), f"{what}: pages"

    def check_significance(self, got, before, sig, what=""):
        seen = np.zeros(got.shape, bool)
        for (li, r), (sums, b) in sig.items():
            c, n = self.ctx[r], self.new[r]
            l, rows = self.layer0 + li, r * self.cap + np.arange(c + n)
            seen[l, rows] = True
            want = sums.copy()
            want[:c] += before[l, rows[:c]]
            err, bound = np.abs(got[l, rows] - want), b + 2 * U * np.abs(want)
            assert np.all(err <= bound), f"{what}: ({li}, {r}) off by {(err / bound).max():.3g} of its bound"
        assert np.array_equal(got[~seen], before[~seen]), f"{what}: rows of nothing attended changed"


def serial_evict(st: dict, L, R, Hq, Hkv, cap, P, kh, vh, budgets, ctx, sig, cnt=None, sinks=0, window=0, unit_base=0):
    """dkv_evict, one token after the other; st also has classes and slot_of [L * R * cap * Hkv]."""
    st = copy_state(st)
    F, G = st["free_list"].size, Hq // Hkv
    cls, slot = (st[k].reshape(L, R, cap, Hkv) for k in ("classes", "slot_of"))
    tail = int(st["cursors"][1])
    for u in range(L * R * Hkv):
        l, r, h = u // (R * Hkv), u // Hkv % R, u % Hkv
        c, b = int(ctx[r]), int(budgets[r])
        held = [p for p in range(c) if cls[l, r, p, h]]
        if b < 0 or len(held) <= b:
            continue
        w = sig[l, r * cap:(r + 1) * cap, h * G:(h + 1) * G].max(1)  # a NaN among them is the maximum here
        if cnt is not None:
            with np.errstate(divide="ignore", invalid="ignore"):
                w = w / cnt[r * cap:(r + 1) * cap].astype(np.float32)
        safe = [p for p in held if p < sinks or p >= c - window]
        rest = sorted((p for p in held if p not in set(safe)), key=lambda p: (-np.inf if np.isnan(w[p]) else w[p],
                                                                            not np.isnan(w[p]), -p), reverse=True)
        keep = set(safe) | set(rest[:max(0, b - len(safe))])
        row, hdr = st["fwd"][u].copy(), st["unit_hdr"][u].copy()
        new_hdr, kept, freed = [0, 0, 0, 0], [], []
        for i, (code, per, ku, vu) in enumerate(((2, P, kh, vh), (1, 2 * P, kh // 2, vh // 2))):
            n, first = int(hdr[i]), 0 if i == 0 else int(hdr[2])
            at = {int(slot[l, r, p, h]): p for p in held if cls[l, r, p, h] == code}
            assert sorted(at) == list(range(n))

            def pieces(s):
                pg, s = st["pages"][int(row[first + s // per])], s % per
                C = 16 * (kh + vh) * P
                return (pg[16 * ku * s:16 * ku * (s + 1)], pg[16 * kh * P + 16 * vu * s:16 * kh * P + 16 * vu * (s + 1)],
                        pg[C + 8 * s:C + 8 * s + 8], pg[C + 16 * P + 4 * s:C + 16 * P + 4 * s + 4])

            k = sum(p in keep for p in at.values())
            holes = [s for s in range(k) if at[s] not in keep]
            movers = [s for s in range(k, n) if at[s] in keep]
            for t, f in zip(holes, movers):
                for x, y in zip(pieces(t), pieces(f)):
                    x[:] = y
                slot[l, r, at[f], h] = t
            need = -(-k // per)
            for s in range(k, min(n, need * per)):
                for x, fill in zip(pieces(s), (0, 0, 0, 255)):
                    x[:] = fill
            have = int(hdr[2 + i])
            kept += [int(x) for x in row[first:first + need]]
            freed += [int(x) for x in row[first + need:first + have]]
            new_hdr[i], new_hdr[2 + i] = k, need
        for p in held:
            if p not in keep:
                cls[l, r, p, h], slot[l, r, p, h] = 0, -1
        st["fwd"][u] = -1
        st["fwd"][u][:len(kept)] = kept
        for j, p in enumerate(kept):
            st["rev_idx"][p] = j
        for p in freed:
            st["free_list"][tail % F] = p
            tail += 1
            st["rev_unit"][p] = st["rev_idx"][p] = -1
            st["page_cls"][p] = 0
        st["unit_hdr"][u] = new_hdr
    st["cursors"][1] = tail
    return st
