"""Lists of lengths that do not name every request of the tables are refused: a
unit's index counts all of them, and the kernels read as many."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import build as libbuild
from differentiated_kv_cache_dkv_gb300 import libdkv


def _i32(n):
    return torch.ones(n, dtype=torch.int32)


def _decoder(L, R):
    dec = libdkv.Decoder.__new__(libdkv.Decoder)  # no device state: the lists are looked at first
    dec.L, dec.R, dec.Hq, dec.Hkv, dec.cap, dec.device = L, R, 4, 2, 64, torch.device("cpu")
    dec.pool = dec.tables = None
    dec._ext_ws = []
    return dec


@pytest.mark.parametrize("new,ctx", [(2, 4), (3, 3), (5, 5), (4, 2), (4, 5), (0, 0)])
def test_a_decoder_wants_every_request_s_length(new, ctx):
    dec = _decoder(2, 4)
    q = torch.zeros((2, new, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dec.extend(q, _i32(new), _i32(ctx), 1, torch.empty_like(q), 0.1)
    with pytest.raises(ValueError):
        dec.extend_significance(q, _i32(new), _i32(new), _i32(ctx), 1, 0.1, torch.zeros((2, new, 4)),
                                torch.zeros((2, 256, 4)))


@pytest.mark.parametrize("acc", [0, 3, 5])
def test_accepted_lengths_of_every_request(acc):
    libbuild.build()
    q = torch.zeros((1, 4, 4, 128), dtype=torch.bfloat16)
    b = libdkv.make_extend_batch(1, 2, 64, q, _i32(4), _i32(4), 1, 0.1, lse=torch.zeros((1, 4, 4)))
    pool = libdkv.DevicePool(8, 16, "cpu")
    with pytest.raises(ValueError):
        libdkv.dkv_extend_significance(b, _i32(acc), torch.zeros((1, 256, 4)), pool, libdkv.DeviceTables(8, 5, "cpu"))
