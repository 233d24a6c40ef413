"""Decode attention at capacities whose shared memory lies at the edge of what
a block may have: the kernel's own arrays count beside the call's."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, make_decoder

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G, caps", [(8, range(3680, 3744, 16)), (7, range(4160, 4416, 16)), (4, range(1984, 8192, 496))])
def test_capacities_at_the_edge(G, caps):
    """Groups of 8 from 3712 positions, pages of 16: 223 616 to 225 280 bytes beside 8 832 of the kernel's did not
    launch.  The outputs are those of a small capacity but for the order of the sums: every position's weight is
    positive, so a sum of n terms errs by at most n 2^-24 of the largest value on either side, and a weight by its
    logit's, 300 2^-24 |q| |k| scale."""
    w = W.small("edge", lens=[300], L=1, Hq=2 * G, Hkv=2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((1, 1, 2 * G, 128), generator=g).bfloat16().cuda()
    want = None
    for cap in (304, *caps):
        dec, sig, cnt, ctx = make_decoder(w, cap)
        out = torch.full((1, 1, 2 * G, 128), float("nan"), device="cuda")
        dec.attend(q, ctx, out, SCALE)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK, cap
        if want is None:
            want = out
            continue
        inp = W.make_inputs(w, 7)
        top = float(inp["v"].float().abs().max())
        dx = 300 * 2.0 ** -24 * SCALE * float(q.float().norm(dim=-1).max()) * float(inp["k"].float().norm(dim=-1).max())
        assert float((out - want).abs().max()) <= 2 * top * (2 * dx + 300 * 2.0 ** -24), cap
