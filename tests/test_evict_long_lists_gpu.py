"""Eviction of units whose lists have more pages than a block keeps ids of in
shared memory (1024) and than a plan block has threads (512)."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import make_decoder
from tests.page_ops_helpers import assert_untouched
from tests.test_evict_gpu import _check, _i32, _state

pytestmark = pytest.mark.gpu


def _long(alpha_h, alpha_l, lens=(6001,)):
    w = W.small("evict_pages", lens=list(lens), L=1, Hq=4, Hkv=2, P=2, alpha_h=alpha_h, alpha_l=alpha_l)
    cap = 6016
    return w, cap, *make_decoder(w, cap, F=16000)


@pytest.mark.parametrize("alpha_h, alpha_l, which", [(0.01, 0.0, 2), (2.0, 0.001, 3)])
def test_lists_of_more_than_a_thousand_pages(alpha_h, alpha_l, which):
    """Mostly high and mostly low tokens, three times: the later ones on lists whose slots are out of order."""
    w, cap, dec, sig, cnt, ctx = _long(alpha_h, alpha_l)
    assert int(dec.tables.unit_hdr[:, which].max()) > 1024
    g = torch.Generator("cuda").manual_seed(2)
    for b in (4500, 3500, 400):
        before = _state(dec)
        sig = sig[:, torch.randperm(sig.shape[1], generator=g, device="cuda")].contiguous()
        dec.evict(_i32([b]), ctx, sig, cnt, sinks=4, window=64)
        assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
        _check(dec, before, w, cap, [b], w.lens, sig, cnt, 4, 64, str(b))


@pytest.mark.parametrize("what", ["reverse index", "reverse unit", "page id"])
def test_an_error_behind_the_first_pages(what):
    w, cap, dec, sig, cnt, ctx = _long(0.01, 0.0)
    u, j = 1, int(dec.tables.unit_hdr[1, 2]) - 1
    assert j > 1024
    id_ = int(dec.tables.fwd[u, j])
    if what == "reverse index":
        dec.pool.rev_idx[id_] -= 1
    elif what == "reverse unit":
        dec.pool.rev_unit[id_] = 0
    else:
        dec.tables.fwd[u, j] = -1
    before = _state(dec)
    dec.evict(_i32([3000]), ctx, sig, cnt)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_E_INTERNAL
    assert_untouched(_state(dec), before, what)
