"""Decode states and new tokens whose logits are chosen: channel 0 of the keys
carries each token's level, channel 0 of the queries is the same for all rows,
the other channels are noise."""
from __future__ import annotations

import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE

Q0 = 8.0


def keys_of(levels, Hkv: int, L: int, seed: int, noise: float = 1.0) -> torch.Tensor:
    """bf16 [L][n][Hkv][128]: token t's logits are levels[t] + noise N(0, 1)."""
    g = torch.Generator().manual_seed(seed)
    k = noise * torch.randn((L, len(levels), Hkv, 128), generator=g)
    k[..., 0] = (torch.tensor(levels, dtype=torch.float32) / (SCALE * Q0)).view(1, -1, 1)
    return k.bfloat16()


def queries_of(n: int, Hq: int, L: int, seed: int) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((L, n, Hq, 128), generator=g)
    q[..., 0] = Q0
    return q.bfloat16()


def decoder_of(w: W.Workload, cap: int, keys: torch.Tensor, device="cuda"):
    """A device Decoder that holds the workload's tokens with the given keys,
    its significance sums [L][R * cap][Hq], and ctx_lens."""
    inp = W.make_inputs(w, 7)
    dec = libdkv.Decoder(w.L, w.R, w.Hq, w.Hkv, cap, w.P, 3 * w.pool_pages + 8, device=device, scheme=w.scheme)
    ctx = torch.tensor(w.lens, dtype=torch.int32, device=device)
    sig = torch.zeros((w.L, w.R * cap, w.Hq))
    t = 0
    for r, n in enumerate(w.lens):
        sig[:, r * cap:r * cap + n] = inp["sig_sum"][:, t:t + n]
        t += n
    for l in range(w.L):
        layer = {"L": 1, "R": w.R, "Hq": w.Hq, "Hkv": w.Hkv, "T": w.T, "lens": ctx,
                 "sig_cnt": inp["sig_cnt"].to(device), "k": keys[l:l + 1].contiguous().to(device)}
        for x in ("v", "sig_sum"):
            layer[x] = inp[x][l:l + 1].contiguous().to(device)
        dec.prefill_layer(layer, l, max(w.lens), w.alpha_h, w.alpha_l)
    dec.index(ctx)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    return dec, sig.to(device), ctx
