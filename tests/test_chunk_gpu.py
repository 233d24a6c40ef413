"""Attention of a chunk over bf16 pages and its significance on the GPU, against
float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from differentiated_kv_cache_dkv_gb300 import libdkv
from tests.chunk_helpers import SCALE, Chunk

pytestmark = pytest.mark.gpu

SHAPES = {
    "tiny": dict(Hq=8, Hkv=2, B=16, ctx=[512], new=[16]),
    "one head each, small pages": dict(Hq=4, Hkv=4, B=8, ctx=[0, 1, 7, 8, 9], new=[1, 1, 9, 0, 127]),
    "group of 7": dict(Hq=28, Hkv=4, B=32, ctx=[0, 129, 1000], new=[65, 1, 33], fused=True),
    "group of 16": dict(Hq=16, Hkv=1, B=64, ctx=[300], new=[40]),
    "group of 32": dict(Hq=32, Hkv=1, B=128, ctx=[5, 128], new=[130, 3]),
    "group of 128": dict(Hq=128, Hkv=1, B=16, ctx=[17], new=[3]),
    "single tokens": dict(Hq=6, Hkv=2, B=16, ctx=[2000, 3, 0, 127, 128, 4000], new=[1, 1, 1, 1, 1, 0], fused=True),
    "one long single token": dict(Hq=8, Hkv=2, B=16, ctx=[9001], new=[1]),
    "several rows, long": dict(Hq=4, Hkv=1, B=64, ctx=[5000, 100], new=[7, 2]),
    "prompts from the start": dict(Hq=4, Hkv=2, B=64, ctx=[0, 0, 0], new=[513, 64, 128]),
    "layers": dict(Hq=6, Hkv=3, B=32, ctx=[40, 0, 300], new=[9, 1, 70], L=4, layer0=1, n_layers=2),
    "layers of one projection": dict(Hq=4, Hkv=2, B=16, ctx=[33], new=[1], L=3, layer0=0, n_layers=3, fused=True),
    # enough of it that a block has several items, whole and cut, of one row tile, of two and of both in turn
    "many single tokens": dict(Hq=16, Hkv=8, B=16, ctx=[37 * i % 2000 for i in range(60)], new=[1] * 60),
    "many short items": dict(Hq=8, Hkv=8, B=16, ctx=[i % 300 for i in range(200)], new=[1 + i % 3 for i in range(200)]),
    "many of two row tiles": dict(Hq=16, Hkv=4, B=32, ctx=[0, 100, 2000], new=[700, 300, 500], fused=True),
    "one and two row tiles mixed": dict(Hq=16, Hkv=4, B=64, ctx=[211 * i % 1500 for i in range(40)],
                                        new=[(1, 33, 70, 5, 64)[i % 5] for i in range(40)]),
    # significance: one key tile and two in turn, few blocks of rows in each, several a block of the launch
    "short items of large groups": dict(Hq=64, Hkv=1, B=128, ctx=[0 if i % 3 == 0 else 83 * i % 300 for i in range(70)],
                                        new=[1 + i % 2 for i in range(70)], L=3, n_layers=3),
    "short items of the largest group": dict(Hq=128, Hkv=1, B=32, ctx=[0 if i % 5 == 0 else 131 * i % 301 for i in range(70)],
                                             new=[i % 6 for i in range(70)]),
    "none new": dict(Hq=2, Hkv=1, B=16, ctx=[5, 300, 17], new=[0, 2, 0]),
}


@pytest.mark.parametrize("name", SHAPES)
def test_attention_and_significance(name):
    c = Chunk(seed=len(name), **SHAPES[name])
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    ref = c.reference(lse_in=d["lse"].cpu().numpy())
    c.check(d, ref, name)
    g = torch.Generator().manual_seed(3)
    before = torch.rand((c.L, c.R * c.cap, c.Hq), generator=g)
    sig = before.cuda()
    libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
    assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_OK
    c.check_significance(sig.cpu().numpy(), before.numpy(), ref[4], name)


@pytest.mark.parametrize("name", ["group of 7", "several rows, long", "prompts from the start"])
def test_equal_bits_twice(name):
    c = Chunk(seed=5, **SHAPES[name])
    got = []
    for _ in range(2):
        d = c.device()
        assert c.attend(d) == libdkv.DKV_OK
        sig = torch.zeros((c.L, c.R * c.cap, c.Hq), device="cuda")
        libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
        got.append((d["out"].view(torch.int16), d["lse"], sig))
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_pages_that_hold_the_new_tokens_already():
    c = Chunk(8, 2, 16, [100, 0, 31], [20, 3, 1], seed=2)
    k, v = c.appended()
    d = c.device(k=k.cuda(), v=v.cuda(), kn=None, vn=None, lse=None)
    assert c.attend(d) == libdkv.DKV_OK
    c.check(d, c.reference())


def test_max_new_above_the_longest():
    c = Chunk(8, 2, 16, [100, 0], [20, 3], seed=2)
    d = c.device(max_new=500)
    assert c.attend(d) == libdkv.DKV_OK
    c.check(d, c.reference(lse_in=d["lse"].cpu().numpy()))


@pytest.mark.parametrize("q_size, k_size", [(30.0, 30.0), (1e18, 1.0), (1e-20, 1.0)])
def test_logits_of_any_size(q_size, k_size):
    """A row's largest logit far above its first, and far below: the reference follows."""
    c = Chunk(4, 1, 16, [700, 300], [70, 1], seed=9, outlier=1.0)
    c.q = (c.q.float() * q_size).bfloat16()
    c.kn = (c.kn.float() * k_size).bfloat16()
    c.k = (c.k.float() * k_size * torch.linspace(1e-3, 1.0, c.B).view(1, 1, -1, 1, 1)).bfloat16()
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    if q_size < 1e10:
        c.check(d, c.reference())
        return
    # logits of 1e18: the largest alone is left (the others are further away than fp32's exponent reaches)
    k, v = c.appended()
    t = 0
    for r, (ctx, n) in enumerate(zip(c.ctx, c.new)):
        x = np.einsum("ihd,td->hit", c.q[0, t:t + n].double().numpy(), c.rows(k, r, 0)[:, 0])
        x[:, np.arange(ctx + n) > ctx + np.arange(n)[:, None]] = -np.inf
        want = c.rows(v, r, 0)[:, 0][x.argmax(-1)].transpose(1, 0, 2)
        got = d["out"][0, t:t + n].double().cpu().numpy()
        two = np.sort(x, -1)[..., -2:]
        clear = (two[..., 1] - two[..., 0] > 1e-4 * np.abs(two[..., 1])) if ctx + n > 1 else np.ones(x.shape[:2], bool)
        assert clear.mean() > 0.9 and np.array_equal(got[clear.T], want[clear.T])
        t += n


def test_rising_logits_move_the_reference():
    """Every tile's logits lie above the tile's before by more than the exponent's reach."""
    c = Chunk(2, 1, 16, [1200], [5], seed=4, outlier=1.0)
    ones = torch.ones(128).bfloat16()
    c.q[:] = ones
    for x, base in ((c.k, 0), ):
        for p in range(1200):
            x[0, int(c.table[0, p // 16]), p % 16, 0] = (ones.float() * 0.25 * (p // 100)).bfloat16()
    c.kn[:] = (ones.float() * 3.0).bfloat16()
    d = c.device(scale=2.0)
    assert c.attend(d) == libdkv.DKV_OK
    c.check(d, c.reference(scale=2.0))


@pytest.mark.parametrize("new", [[1], [5], [20], [70]])
def test_large_values_under_a_first_reference_far_below(new):
    """Values of up to 2^100 whose logits lie 50 log2 units above those of a row's first positions: weights relative
    to those would add up to 2^58."""
    c = Chunk(2, 1, 16, [300], new, seed=14, outlier=1.0)
    c.q[:] = 1.0
    for p in range(300):
        c.k[0, int(c.table[0, p // 16]), p % 16, 0] = 0.0 if p < 32 else 0.27
    c.kn[:] = 0.27
    c.v = (c.v.float().clamp(-4, 4) * 2.0 ** 98).bfloat16()
    c.vn = (c.vn.float().clamp(-4, 4) * 2.0 ** 98).bfloat16()
    d = c.device(scale=1.0)
    assert c.attend(d) == libdkv.DKV_OK
    c.check(d, c.reference(scale=1.0))


def test_more_requests_than_the_plan_keeps_in_shared_memory():
    c = Chunk(16, 16, 8, [7 * i % 50 for i in range(1100)], [1 + (i % 97 == 0) for i in range(1100)], seed=15)
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    ref = c.reference(lse_in=d["lse"].cpu().numpy())
    c.check(d, ref)
    before = torch.ones((1, c.R * c.cap, c.Hq))
    sig = before.cuda()
    libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
    assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_OK
    c.check_significance(sig.cpu().numpy(), before.numpy(), ref[4])


def test_bad_lengths_write_nothing():
    c = Chunk(4, 2, 16, [30, 50], [10, 4], seed=1)
    for over in (dict(new=[10, 5]), dict(new=[-1, 15]), dict(ctx=[30, -1]), dict(ctx=[30, c.cap - 3]), dict(max_new=9)):
        over = {k: torch.tensor(v, dtype=torch.int32, device="cuda") if isinstance(v, list) else v
                for k, v in over.items()}
        d = c.device(**over)
        k, v = d["k"].clone(), d["v"].clone()
        assert c.attend(d) == libdkv.DKV_E_LENS, over
        assert bool((d["out"] == 7).all()) and bool((d["lse"] == 7).all())
        assert torch.equal(d["k"].view(torch.int16), k.view(torch.int16))
        assert torch.equal(d["v"].view(torch.int16), v.view(torch.int16))
        sig = torch.full((1, c.R * c.cap, c.Hq), 3.0, device="cuda")
        libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
        assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_E_LENS and bool((sig == 3).all())


def test_values_that_are_not_finite_are_stored_as_zero():
    c = Chunk(4, 2, 16, [30, 50], [10, 4], seed=1)
    d = c.device()
    d["kn"][0, 3, 1, 17] = float("nan")
    d["vn"][0, 12, 0, 5] = float("inf")
    c.kn[0, 3, 1, 17] = 0
    c.vn[0, 12, 0, 5] = 0
    assert c.attend(d) == libdkv.DKV_E_RANGE
    c.check(d, c.reference())


def test_a_page_id_out_of_range_harms_only_its_request():
    c = Chunk(4, 2, 16, [30, 50, 64], [10, 4, 1], seed=1)
    for bad in (-1, c.k.shape[1], 2 ** 31 - 1):
        d = c.device()
        d["table"][1, 1] = bad
        k, v = c.appended()
        assert c.attend(d) == libdkv.DKV_E_INTERNAL
        out, ob, *_ = c.reference()
        got = d["out"].double().cpu().numpy()
        for sl in (slice(0, 10), slice(14, 15)):
            assert np.all(np.abs(got[:, sl] - out[:, sl]) <= ob[:, sl])
        assert torch.equal(d["k"].cpu().view(torch.int16), k.view(torch.int16))  # the new tokens' page is another
        sig = torch.zeros((1, c.R * c.cap, c.Hq), device="cuda")
        libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
        assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_E_INTERNAL


def test_an_infinite_query_spoils_its_row_alone():
    c = Chunk(4, 2, 16, [300], [40], seed=6)
    d = c.device()
    d["q"][0, 7, 2, 3] = float("inf")
    assert c.attend(d) == libdkv.DKV_OK
    out, ob, *_ = c.reference()
    err = np.abs(d["out"].double().cpu().numpy() - out) - ob
    ok = np.ones(out.shape[:3], bool)
    ok[0, 7, 2] = False
    assert np.all(err[ok] <= 0)


def test_a_row_whose_lse_is_minus_infinity_adds_nothing():
    c = Chunk(4, 2, 16, [30], [6], seed=1)
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    d["lse"][0, 2] = float("-inf")
    sig = torch.zeros((1, c.cap, c.Hq), device="cuda")
    libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
    # the reference counts such a row with weights of exp(x - 1000) = 0
    ref = c.reference(lse_in=np.where(np.isinf(d["lse"].cpu().numpy()), np.float32(1e3), d["lse"].cpu().numpy()))
    c.check_significance(sig.cpu().numpy(), np.zeros(sig.shape, np.float32), ref[4])


def test_streams_and_graphs():
    """A captured call replayed with other contents and lengths; a call on a stream of its own."""
    c = Chunk(8, 2, 16, [200, 31], [12, 5], seed=3)
    d = c.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert c.attend(d) == libdkv.DKV_OK
    torch.cuda.current_stream().wait_stream(side)
    c.check(d, c.reference())
    sig = torch.zeros((1, c.R * c.cap, c.Hq), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        libdkv.dkv_chunk_attention(d["batch"], d["pages"], d["pool"], d["ws"])
        libdkv.dkv_chunk_significance(d["batch"], d["pages"], sig, d["pool"])
    e = Chunk(8, 2, 16, [205, 33], [7, 10], seed=11)  # as many pages and tokens
    assert e.k.shape == c.k.shape and e.table.shape == c.table.shape
    for n in ("k", "v", "table", "q", "kn", "vn"):
        d[n].copy_(getattr(e, n))
    d["new"].copy_(torch.tensor(e.new, dtype=torch.int32))
    d["ctx"].copy_(torch.tensor(e.ctx, dtype=torch.int32))
    for _ in range(2):
        sig.zero_()
        graph.replay()
        assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_OK
        ref = e.reference(lse_in=d["lse"].cpu().numpy())
        e.check(d, ref)
        e.check_significance(sig.cpu().numpy(), np.zeros(sig.shape, np.float32), ref[4])


def test_two_calls_at_once_with_a_workspace_each():
    cs = [Chunk(8, 2, 16, [3000 + 100 * i], [9], seed=i) for i in range(2)]
    ds = [c.device() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, s in zip(cs, ds, streams):
            libdkv.dkv_chunk_attention(d["batch"], d["pages"], d["pool"], d["ws"], stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cs, ds):
        assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_OK
        c.check(d, c.reference())


def test_a_shared_prefix():
    """Two requests whose tables name the same pages of a common prefix."""
    c = Chunk(4, 2, 16, [64, 64], [3, 5], seed=8)
    c.table[1, :4] = c.table[0, :4]
    d = c.device()
    assert c.attend(d) == libdkv.DKV_OK
    c.check(d, c.reference())


def test_nothing_to_do():
    c = Chunk(4, 2, 16, [64], [0], seed=8)
    d = c.device()
    k = d["k"].clone()
    assert c.attend(d) == libdkv.DKV_OK
    libdkv.dkv_chunk_significance(d["batch"], d["pages"], torch.zeros((1, c.cap, 4), device="cuda"), d["pool"])
    assert libdkv.dkv_get_status(d["pool"]) == libdkv.DKV_OK
    assert torch.equal(d["k"].view(torch.int16), k.view(torch.int16))


def test_a_prompt_in_chunks_is_the_prompt_at_once():
    """Outputs and significance over all chunks against one prefill attention over whole prompts."""
    Hq, Hkv, lens, B = 8, 2, [700, 259], 32
    g = torch.Generator().manual_seed(12)
    T = sum(lens)
    q, k, v = (torch.randn((1, T, h, 128), generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    pool = libdkv.DevicePool(1, 2)
    out = torch.empty((1, T, Hq, 128), device="cuda")
    sig, cnt = torch.empty((1, T, Hq), device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    libdkv.dkv_prefill_attention(q, k, v, i32(lens), max(lens), SCALE, out, sig, cnt, pool)
    cap = 704
    pages = libdkv.ChunkPages(1, 2, Hkv, cap, B, 2 * cap // B)
    pages.table.copy_(torch.randperm(2 * cap // B, generator=g).view(2, -1))
    mine, mysig = torch.empty_like(out), torch.zeros((1, 2 * cap, Hq), device="cuda")
    start, ctx = [0, lens[0]], [0, 0]
    while ctx != lens:
        new = [min(n - c, m) for n, c, m in zip(lens, ctx, (256, 100))]
        at = torch.cat([torch.arange(s + c, s + c + n) for s, c, n in zip(start, ctx, new)]).cuda()
        o, lse = torch.empty((1, sum(new), Hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, sum(new), Hq), device="cuda")
        qc, kc, vc, nc, cc = q[:, at], k[:, at], v[:, at], i32(new), i32(ctx)  # the batch holds their addresses alone
        b = libdkv.make_chunk_batch(Hkv, cap, qc, nc, cc, max(new), SCALE, k_new=kc, v_new=vc, out=o, lse=lse)
        ws = torch.empty(libdkv.dkv_chunk_workspace_size(b, pages), dtype=torch.uint8, device="cuda")
        libdkv.dkv_chunk_attention(b, pages, pool, ws)
        libdkv.dkv_chunk_significance(b, pages, mysig, pool)
        mine[:, at] = o.float()
        ctx = [c + n for c, n in zip(ctx, new)]
    assert libdkv.dkv_get_status(pool) == libdkv.DKV_OK
    # both round their weights to bf16, 2^-8 of at most the largest value each; out here is rounded to bf16, 2^-8.
    # A weight is off by twice what a logit is, 300 u scale sum |q| |k| <= 2e-4 for these sizes, on both sides.
    assert torch.all((mine - out).abs() <= 1.05 * (2.0 ** -7 * v.float().abs().max() + 2.0 ** -8 * out.abs()))
    for r, (s, n) in enumerate(zip(start, lens)):
        a, b = sig[0, s:s + n], mysig[0, r * cap:r * cap + n]
        assert torch.all((a - b).abs() <= 8e-4 * a)
