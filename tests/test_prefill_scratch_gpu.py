"""What Decoder.prefill_layer and the dequantisation allocate is memory of the
call's stream, and ids are converted there: the classes are given back while
kernels may still write them, and an earlier owner's work may still run."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.gpu_helpers import to_device
from tests.test_extend_scratch_gpu import _stream_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("side", ["current", "side", "another library's"])
def test_scratch_is_memory_of_the_call_s_stream(side, monkeypatch):
    w = W.small("scratch", L=1, lens=[2000, 300], Hq=8, Hkv=2)
    dec = libdkv.Decoder(1, 2, 8, 2, 2080, w.P, 2 * w.pool_pages)
    inp = to_device(W.make_inputs(w))
    keep = torch.cuda.Stream()
    s = {"current": None, "side": keep, "another library's": SimpleNamespace(cuda_stream=keep.cuda_stream)}[side]
    want = torch.cuda.current_stream().cuda_stream if s is None else s.cuda_stream
    seen, make = [], libdkv.make_batch

    def spy(inp, classes, *a, **kw):
        seen.append(_stream_of(classes))
        return make(inp, classes, *a, **kw)

    monkeypatch.setattr(libdkv, "make_batch", spy)
    torch.cuda.synchronize()
    dec.prefill_layer(inp, 0, 2000, 1.0, 0.2, stream=s)
    torch.cuda.synchronize()
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert seen == [want] and _stream_of(dec._pre_ws) == want


@pytest.mark.parametrize("side", ["current", "side", "another library's"])
def test_dequantised_pages_are_memory_of_the_call_s_stream(side):
    pool = libdkv.DevicePool(8, 16)
    libdkv.dkv_init_pool(pool)
    keep = torch.cuda.Stream()
    s = {"current": None, "side": keep, "another library's": SimpleNamespace(cuda_stream=keep.cuda_stream)}[side]
    want = torch.cuda.current_stream().cuda_stream if s is None else s.cuda_stream
    ids = torch.arange(8, device="cuda")
    torch.cuda.synchronize()
    outs = (*libdkv.dkv_dequant_pages(pool, ids, stream=s), *libdkv.dkv_dequant_page(pool, 3, stream=s))
    torch.cuda.synchronize()
    assert all(_stream_of(x) == want for x in outs)
    assert all(bool((x == (-1 if x.dtype == torch.int32 else 0)).all()) for x in outs)  # free pages
