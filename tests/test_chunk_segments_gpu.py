"""Significance of a chunk with several items a block: the keys of an item
replace the last one's in tensor memory behind its products."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from tests.chunk_helpers import Chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [dict(Hq=32, Hkv=8, B=16, ctx=[1500] * 6, new=[150] * 6),
                                   dict(Hq=16, Hkv=8, B=64, ctx=[300 + 61 * i for i in range(20)], new=[1 + i % 17 for i in range(20)], L=3,
                                        n_layers=3)])
def test_many_items_a_block(shape):
    """Right, and the same bits every time."""
    c = Chunk(seed=21, **shape)
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    ref = c.reference(lse_in=d["lse"].cpu().numpy())
    before = torch.zeros((c.L, c.R * c.cap, c.Hq))
    first = None
    for _ in range(20):
        sig = before.cuda()
        libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
        assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_OK
        if first is None:
            first = sig
            c.check_significance(sig.cpu().numpy(), before.numpy(), ref[4])
        assert torch.equal(sig, first)
