"""Pages, significance rows and quantised pages whose offsets pass 32 bits: the
last pages of a pool of 17 GB, rows 2^31 sums and more behind the first."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from differentiated_kv_cache_dkv_gb300 import workloads as W
from tests.chunk_helpers import SCALE, Chunk, serial_evict
from tests.gpu_helpers import to_device
from tests.page_ops_helpers import assert_equal
from tests.test_evict_gpu import _i32, _state

pytestmark = pytest.mark.gpu


def test_pages_and_sums_far_behind_the_first():
    L, cap = 2, 1 << 24
    c = Chunk(64, 8, 16, [300, 0, 40], [20, 150, 1], seed=31)
    few, F = c.k.shape[1], (1 << 17) + 5
    k = torch.zeros((L, F, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k[0].numel() > 2 ** 31
    k[1, F - few:], v[1, F - few:] = c.k[0].cuda(), c.v[0].cuda()
    table = torch.full((3, cap // 16), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = torch.where(c.table < few, c.table + (F - few), c.table).cuda()
    q, kn, vn = (x.cuda() for x in (c.q, c.kn, c.vn))
    d = dict(out=torch.empty_like(q), lse=torch.empty((1, c.T, 64), device="cuda"), k=k[1:, F - few:], v=v[1:, F - few:])
    pool, pages = libdkv.DevicePool(1, 2), libdkv.ChunkPages.from_tensors(k, v, table)
    b = libdkv.make_chunk_batch(8, cap, q, _i32(c.new), _i32(c.ctx), c.max_new, SCALE, k_new=kn, v_new=vn, out=d["out"],
                                lse=d["lse"], layer0=1, L=L)
    ws = torch.empty(libdkv.dkv_chunk_workspace_size(b, pages), dtype=torch.uint8, device="cuda")
    libdkv.dkv_chunk_attention(b, pages, pool, ws)
    assert libdkv.dkv_get_status(pool) == libdkv.DKV_OK
    ref = c.reference(lse_in=d["lse"].cpu().numpy())
    c.check(d, ref)
    for x in (k, v):
        assert not bool(x[0].any()) and not bool(x[1, :F - few].any())
    sig = torch.zeros((L, 3 * cap, 64), device="cuda")
    assert sig[0].numel() > 2 ** 31
    libdkv.dkv_chunk_significance(b, pages, sig, pool)
    assert libdkv.dkv_get_status(pool) == libdkv.DKV_OK
    for r, n in enumerate(x + y for x, y in zip(c.ctx, c.new)):
        sums, bound = ref[4][0, r]
        got = sig[1, r * cap:r * cap + n].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - sums) <= bound + 2 ** -23 * sums)
        sig[1, r * cap:r * cap + n] = 0
    assert not any(bool(x.any()) for x in sig.view(-1).split(1 << 30))


class Rows:
    """Sums that are 0 but in the rows of one request."""

    def __init__(self, rows, at):
        self.rows, self.at = rows, at

    def __getitem__(self, key):
        _, where, heads = key
        return self.rows[:, heads] if where.start == self.at else np.zeros((where.stop - where.start, 1), np.float32)


def test_eviction_of_the_last_of_many_long_requests():
    R, Hq, cap, F, n = 65, 128, 1 << 18, 700000, 500
    w = W.small("far", lens=[0] * (R - 1) + [n], L=1, Hq=Hq, Hkv=1)
    dec = libdkv.Decoder(1, R, Hq, 1, cap, w.P, F)
    dec.pool.free_list.copy_(torch.arange(F - 1, -1, -1, dtype=torch.int32))  # the last pages first
    assert dec.pool.pages.numel() > 2 ** 31 and R * cap * Hq > 2 ** 31
    dec.prefill_layer(to_device(W.make_inputs(w)), 0, n, w.alpha_h, w.alpha_l)
    ctx = _i32(w.lens)
    dec.index(ctx)
    sig, at = torch.zeros((1, R * cap, Hq), device="cuda"), (R - 1) * cap
    g = torch.Generator("cuda").manual_seed(1)
    sig[0, at:at + n] = torch.rand((n, Hq), generator=g, device="cuda")
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    assert int(dec.tables.fwd[R - 1, 0]) == F - 1
    before, budgets = _state(dec), [-1] * (R - 1) + [120]
    dec.evict(_i32(budgets), ctx, sig, window=16, sinks=2)
    assert libdkv.dkv_get_status(dec.pool) == libdkv.DKV_OK
    rows = Rows(sig[0, at:at + cap].cpu().numpy(), at)
    want = serial_evict(before, 1, R, Hq, 1, cap, w.P, 8, 4, budgets, w.lens, rows, sinks=2, window=16)
    got = _state(dec)
    assert_equal(got, want, "far")
    assert all(np.array_equal(got[k], want[k].reshape(-1)) for k in ("classes", "slot_of"))
