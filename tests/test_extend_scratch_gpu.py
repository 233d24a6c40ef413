"""The scratch that a Decoder allocates for a call is memory of the call's
stream: another stream's could still be in use by work that had it before."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.extend_helpers import SCALE, draw_new, make_decoder

pytestmark = pytest.mark.gpu


def _stream_of(t: torch.Tensor) -> int:
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the caching allocator's memory")


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("side", ["current", "side", "another library's"])
def test_scratch_is_memory_of_the_call_s_stream(side):
    w = W.small("scratch", L=1, lens=[2000, 0], Hq=8, Hkv=2)
    dec, _, _, ctx = make_decoder(w, 2080)
    q, k, v = (x.cuda() for x in draw_new(w, [4, 0], 1, 3))
    q2, k2, v2 = (x.cuda() for x in draw_new(w, [40, 0], 1, 3))
    outs = [torch.empty_like(x) for x in (q, q2)]
    lens, lists = [_i32([4, 0]), _i32([40, 0])], [_i32([0]), _i32([1])]  # alive until the side stream is done
    torch.cuda.synchronize()
    keep = torch.cuda.Stream()
    s = {"current": None, "side": keep, "another library's": SimpleNamespace(cuda_stream=keep.cuda_stream)}[side]
    want = torch.cuda.current_stream().cuda_stream if s is None else s.cuda_stream
    # the second call outgrows the first one's
    dec.extend(q, lens[0], ctx, 4, outs[0], SCALE, k_new=k, v_new=v, stream=s)
    dec.extend(q2, lens[1], ctx, 40, outs[1], SCALE, k_new=k2, v_new=v2, stream=s)
    dec.fork(lists[0], lists[1], ctx, stream=s)
    dec.release(lists[1], stream=s)
    dec.defrag(stream=s)
    torch.cuda.synchronize()
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert len(dec._ext_ws) == 2
    assert all(_stream_of(x) == want for x in dec._ext_ws + [dec._ops_ws])
