"""What the bindings of the chunk and eviction calls refuse before the library
sees it: tensors of several devices, tables of fewer units than the batch has."""
from __future__ import annotations

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import build as libbuild
from differentiated_kv_cache_dkv_gb300 import libdkv

I32, BF16 = torch.int32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()


def _chunk(device):
    t = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device=device)  # noqa: E731
    return libdkv.make_chunk_batch(2, 64, t(1, 5, 4, 128), t(3, dtype=I32), t(3, dtype=I32), 5, 0.1, k_new=t(1, 5, 2, 128),
                                   v_new=t(1, 5, 2, 128), out=t(1, 5, 4, 128), lse=t(1, 5, 4, dtype=torch.float32))


def _pool(device):
    return libdkv.DevicePool(8, 2, device=device)


def _pages(device):
    return libdkv.ChunkPages(1, 3, 2, 64, 16, 12, device=device)


@pytest.mark.parametrize("at", range(4))
def test_tensors_of_two_devices(at):
    """One of batch, pages, pool and workspace lies elsewhere: refused before a launch."""
    d = ["meta" if i == at else "cpu" for i in range(4)]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=d[3])
    with pytest.raises(ValueError, match="one device"):
        libdkv.dkv_chunk_attention(_chunk(d[0]), _pages(d[1]), _pool(d[2]), ws, stream=0)
    if at < 3:
        sig = torch.zeros((1, 192, 4), device=d[1])
        with pytest.raises(ValueError, match="one device"):
            libdkv.dkv_chunk_significance(_chunk(d[0]), _pages(d[1]), sig, _pool(d[2]), stream=0)


def _evict(device="cpu", L=2):
    t = lambda n, dtype: torch.zeros(n, dtype=dtype, device=device)  # noqa: E731
    return libdkv.make_evict_batch(L, 3, 4, 2, 16, t(3, I32), t(3, I32), t(L * 48 * 4, torch.float32), t(L * 96, torch.uint8),
                                   t(L * 96, I32))


def test_eviction_on_two_devices():
    tables = libdkv.DeviceTables(12, 9, device="cpu")
    for b, p, w in (("meta", "cpu", "cpu"), ("cpu", "meta", "cpu"), ("cpu", "cpu", "meta")):
        with pytest.raises(ValueError, match="one device"):
            libdkv.dkv_evict(_evict(b), _pool(p), tables, torch.zeros(1 << 20, dtype=torch.uint8, device=w), stream=0)


def test_eviction_with_too_few_units():
    pool, ws = _pool("cpu"), torch.zeros(1 << 20, dtype=torch.uint8)
    whole = libdkv.DeviceTables(12, 9, device="cpu")
    assert libdkv.dkv_evict_workspace_size(_evict(), pool, whole) > 0
    assert libdkv.dkv_evict_workspace_size(_evict(L=1), pool, libdkv._TableView(whole, 6)) > 0
    for b, t in ((_evict(), libdkv.DeviceTables(11, 9, device="cpu")), (_evict(L=1), libdkv._TableView(whole, 7))):
        with pytest.raises(ValueError, match="units"):
            libdkv.dkv_evict_workspace_size(b, pool, t)
        with pytest.raises(ValueError, match="units"):
            libdkv.dkv_evict(b, pool, t, ws, stream=0)
