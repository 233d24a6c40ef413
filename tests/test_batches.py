"""A batch keeps the tensors whose addresses it has: one that is passed as a
temporary is not given back to the allocator before the call."""
from __future__ import annotations

import gc
import weakref

import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv

SHAPES = {
    "q": ((2, 5, 4, 128), torch.bfloat16), "kv": ((2, 5, 2, 128), torch.bfloat16), "lse": ((2, 5, 4), torch.float32),
    "i": ((3,), torch.int32), "sig": ((1, 48, 4), torch.float32), "cnt": ((48,), torch.int32),
    "cls": ((96,), torch.uint8), "slot": ((96,), torch.int32),
}


class Temporaries:
    """Tensors that only the callee may keep."""

    def __init__(self):
        self.refs = []

    def __call__(self, kind):
        shape, dtype = SHAPES[kind]
        t = torch.zeros(shape, dtype=dtype)
        self.refs.append(weakref.ref(t))
        return t


def _tokens(make, t, **kw):
    return make(q=t("q"), new_lens=t("i"), ctx_lens=t("i"), max_new=5, scale=0.1, k_new=t("kv"), v_new=t("kv"), out=t("q"),
                lse=t("lse"), **kw)


MAKE = {
    "chunk": lambda t: _tokens(libdkv.make_chunk_batch, t, Hkv=2, cap=64),
    "extend": lambda t: _tokens(libdkv.make_extend_batch, t, L=2, Hkv=2, cap=64),
    "evict": lambda t: libdkv.make_evict_batch(1, 3, 4, 2, 16, t("i"), t("i"), t("sig"), t("cls"), t("slot"), t("cnt")),
    "fork": lambda t: libdkv.make_fork_batch(1, 3, 4, 2, 16, t("i"), t("i"), t("i"), t("cls"), t("slot"), t("sig"), t("cnt")),
    "release": lambda t: libdkv.make_release_batch(1, 3, 2, t("i")),
    "compact": lambda t: libdkv.make_batch({"L": 1, "R": 3, "Hq": 4, "Hkv": 2, "T": 48, "k": t("kv"), "v": t("kv"),
                                            "sig_sum": t("sig"), "sig_cnt": t("cnt"), "lens": t("i")}, t("cls"), 16),
}


@pytest.mark.parametrize("kind", MAKE)
def test_a_batch_holds_its_tensors(kind):
    t = Temporaries()
    batch = MAKE[kind](t)
    gc.collect()
    assert t.refs and all(r() is not None for r in t.refs)
    del batch
    gc.collect()
    assert all(r() is None for r in t.refs)
