"""What three further cache operators are measured on: attention of a chunk of
new tokens a request over a paged bf16 cache that the call appends them to, the
significance that the chunk's rows give every token before and among them, and
the eviction of a unit's least attended tokens from the quantised pages.

The plain forms below state each operator in elementary tensor operations in
32 bits; with `own` set the same inputs go through libdkv's entry points.  A
unit is (layer l, request r, KV head h), u = (l R + r) Hkv + h; the layouts of
the bf16 and of the quantised pages are those of include/dkv.h.
"""
import torch

own = False

D = 128
SCALE = 0.08838834764831845
WIDTHS = ((8, 4), (8, 2), (4, 8))  # K and V bits of the high class of each scheme; the low class has half


def _up(x, m):
    return -(-int(x) // m) * m


def _page_bytes(case):
    kh, vh = WIDTHS[case["scheme"]]
    return (16 * (kh + vh) + 24) * case["P"]


# ------------------------------------------------------------------- cases --

def listed():
    tiny = dict(Hq=8, Hkv=2)
    llama = dict(Hq=32, Hkv=8)
    qwen = dict(Hq=28, Hkv=4)
    return [
        # one request of the tiny configuration takes sixteen tokens behind its 512: the smallest call, latency alone
        dict(tiny, name="chunk tiny", op="chunk", R=1, B=16, ctx_lo=512, ctx_hi=512, new_lo=16, new_hi=16, fused=False),
        # prompts that wait for their last chunk and meanwhile take single tokens: bound by the pages' bytes
        dict(llama, name="chunk single tokens", op="chunk", R=64, B=16, ctx_lo=2047, ctx_hi=8191, new_lo=1, new_hi=1,
             fused=False),
        # ragged suffixes, none for some requests, on an odd group of seven query heads, out of one projection's output
        dict(qwen, name="chunk ragged", op="chunk", R=16, B=32, ctx_lo=0, ctx_hi=5001, new_lo=0, new_hi=333,
             fused=True),
        # the first chunk of four prompts: nothing is held, every tile of keys is near the diagonal
        dict(llama, name="chunk first", op="chunk", R=4, B=64, ctx_lo=0, ctx_hi=0, new_lo=2048, new_hi=2048,
             fused=True),
        # a late chunk of four long prompts: bound by the two products
        dict(llama, name="chunk late", op="chunk", R=4, B=64, ctx_lo=16384, ctx_hi=16384, new_lo=1024, new_hi=1024,
             fused=False),
        # what the sixteen tokens of the tiny configuration give: latency
        dict(tiny, name="chunk significance tiny", op="chunk_sig", R=1, B=16, ctx_lo=512, ctx_hi=512, new_lo=16,
             new_hi=16, fused=False),
        # what the ragged suffixes give
        dict(qwen, name="chunk significance ragged", op="chunk_sig", R=16, B=32, ctx_lo=0, ctx_hi=5001, new_lo=0,
             new_hi=333, fused=True),
        # what a chunk of four prompts gives: bound by its one product and the exponentials
        dict(llama, name="chunk significance late", op="chunk_sig", R=4, B=64, ctx_lo=8192, ctx_hi=8192, new_lo=1024,
             new_hi=1024, fused=False),
        # one of four requests of the tiny configuration is cut to half of its tokens: latency
        dict(tiny, name="evict tiny", op="evict", L=1, R=4, P=16, scheme=0, hi=0.5, lo=0.4, ctx_lo=512, ctx_hi=512,
             keep=0.5, share=0.25, sinks=4, window=64, average=True),
        # a batch is cut to what its pool can hold: bound by the significance's bytes and the moved tokens'
        dict(llama, name="evict batch", op="evict", L=8, R=16, P=16, scheme=0, hi=0.5, lo=0.39, ctx_lo=2048,
             ctx_hi=8192, keep=0.5, share=1.0, sinks=4, window=64, average=True),
        # most tokens of a 28-layer ragged batch stay, on larger pages with 4-bit keys, by the sum instead of the average
        dict(qwen, name="evict ragged", op="evict", L=28, R=7, P=32, scheme=2, hi=0.22, lo=0.336, ctx_lo=1, ctx_hi=6001,
             keep=0.85, share=0.8, sinks=0, window=33, average=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("chunk", "chunk", "chunk", "chunk_sig", "chunk_sig", "evict", "evict", "evict"))
    g, hkv = rng.choice(((1, 8), (2, 5), (3, 2), (4, 8), (4, 2), (5, 3), (7, 4), (8, 8), (8, 1), (16, 1)))
    case = dict(op=op, Hq=g * hkv, Hkv=hkv)
    if op != "evict":
        case.update(B=rng.choice((8, 16, 32, 64, 128)), fused=rng.random() < 0.5, R=log(1, 64), ctx_hi=log(1, 16384),
                    new_hi=log(1, 1024))
        case["ctx_lo"] = rng.choice((0, case["ctx_hi"] // 3, case["ctx_hi"]))
        case["new_lo"] = rng.choice((0, 1, case["new_hi"]))
        most = 4 * 32 * 1024 * (17408 if op == "chunk" else 9216)
        while case["R"] * case["Hq"] * case["new_hi"] * (case["ctx_hi"] + case["new_hi"]) > most or \
                case["R"] * case["Hkv"] * case["ctx_hi"] > 64 * 8 * 8192:
            k = rng.choice(("R", "new_hi", "ctx_hi"))
            case[k] = max(1, case[k] // 2)
            case["ctx_lo"] = min(case["ctx_lo"], case["ctx_hi"])
            case["new_lo"] = min(case["new_lo"], case["new_hi"])
        return case
    hi = rng.choice((0.05, 0.22, 0.5, 0.9, 1.0))
    case.update(L=log(1, 28), R=log(1, 32), P=rng.choice((2, 6, 8, 16, 16, 32, 64)), scheme=rng.randrange(3), hi=hi,
                lo=rng.choice((0.0, 0.3, 1.0)) * (1.0 - hi), ctx_hi=log(1, 8192), keep=rng.choice((0.0, 0.1, 0.5, 0.9)),
                share=rng.choice((0.3, 1.0)), sinks=rng.choice((0, 1, 4)), window=rng.choice((0, 1, 33, 64, 500)),
                average=rng.random() < 0.5)
    case["ctx_lo"] = rng.choice((0, case["ctx_hi"] // 3, case["ctx_hi"]))
    while case["L"] * case["R"] * case["Hkv"] * (case["ctx_hi"] + 4 * case["P"]) > 8 * 16 * 8 * 5120:
        k = rng.choice(("L", "R", "ctx_hi"))
        case[k] = max(1, case[k] // 2)
        case["ctx_lo"] = min(case["ctx_lo"], case["ctx_hi"])
    return case


def work(case):
    ctx, hq, hkv, R = 0.5 * (case["ctx_lo"] + case["ctx_hi"]), case["Hq"], case["Hkv"], case["R"]
    if case["op"] != "evict":
        n = max(0.5 * (case["new_lo"] + case["new_hi"]), 1e-3)
        rows = R * n * hq
        pairs = rows * (ctx + 0.5 * n)
        if case["op"] == "chunk":  # K and V held, q, the new K and V read and stored in their pages, outputs
            held = R * ctx * hkv * 512
            return {"bytes": held + rows * (256 + 256 + 4) + R * n * hkv * 1024, "flops": 4.0 * D * pairs}
        sums = R * ctx * hq * 8 + R * n * hq * 4  # held rows read and written, new rows written
        return {"bytes": R * (ctx + n) * hkv * 256 + sums + rows * 260, "flops": 2.0 * D * pairs}
    # the requests that are cut: the significance of their held tokens' positions, classes and slots of them, and of
    # each list the tokens behind the cut that stay, moved
    kh, vh = WIDTHS[case["scheme"]]
    hi, lo, keep = case["hi"], case["lo"], case["keep"]
    cut = case["L"] * case["R"] * case["share"] * ctx
    token = hi * (16 * (kh + vh) + 12) + lo * (8 * (kh + vh) + 12)
    moved = cut * hkv * token * keep * (1 - keep)
    pages = cut * hkv * (hi / case["P"] + lo / (2 * case["P"])) * (1 - keep)
    gone = cut * hkv * (hi + lo) * (1 - keep)
    return {"bytes": cut * (4 * hq + hkv) + cut * hkv * (hi + lo) * 4 + 2 * moved + gone * 5 + pages * 21, "flops": 0}


# ------------------------------------------------------------------ inputs --

def _ragged(lo, hi, n, g):
    """n lengths spread over [lo, hi], both ends among them, in a drawn order (their sum is the case's own)."""
    x = hi - (torch.arange(n, device="cuda") * (hi - lo)) // max(n - 1, 1)
    return x[torch.randperm(n, generator=g, device="cuda")].to(torch.int32)


def _chunk_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    R, Hq, Hkv, B = case["R"], case["Hq"], case["Hkv"], case["B"]
    ctx = _ragged(case["ctx_lo"], case["ctx_hi"], R, g)
    new = _ragged(case["new_lo"], case["new_hi"], R, g)
    T = int(new.sum())
    cap = _up(case["ctx_hi"] + case["new_hi"], 16)
    tmax = -(-cap // B)
    used = (ctx + new + B - 1) // B
    total = int(used.sum())
    F = R * tmax + 3
    # each request's pages lie scattered over the pool; entries behind its last page are not set
    order = torch.randperm(F, generator=g, device="cuda").to(torch.int32)
    table = torch.full((R, tmax), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(tmax, device="cuda") < used.view(-1, 1)] = order[:total]
    # three channels of a KV head are ten times as large
    outlier = torch.ones((2, Hkv, D), device="cuda").scatter_(
        2, torch.rand((2, Hkv, D), generator=g, device="cuda").argsort(2)[..., :3], 10.0)
    kv = [torch.empty((1, F, B, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, o in zip(kv, outlier):
        for a in range(0, F, 1024):
            y = x[0, a:a + 1024]
            y.copy_(torch.randn(y.shape, generator=g, device="cuda") * o)
    new_rows = torch.randn((1, T, Hq + 2 * Hkv, D), generator=g, device="cuda")
    new_rows[:, :, Hq:Hq + Hkv] *= outlier[0]
    new_rows[:, :, Hq + Hkv:] *= outlier[1]
    new_rows = new_rows.bfloat16()  # q, K and V heads of a token side by side, as one projection leaves them
    q, kn, vn = new_rows[:, :, :Hq], new_rows[:, :, Hq:Hq + Hkv], new_rows[:, :, Hq + Hkv:]
    if not case["fused"]:
        q, kn, vn = q.contiguous(), kn.contiguous(), vn.contiguous()
    s = dict(case=case, R=R, Hq=Hq, Hkv=Hkv, B=B, T=T, cap=cap, F=F, ctx=ctx, new=new, table=table, k=kv[0], v=kv[1],
             q=q, kn=kn, vn=vn, max_new=case["new_hi"], max_len=max(1, case["ctx_hi"] + case["new_hi"]))
    if case["op"] == "chunk_sig":
        s["lse"] = _plain_attention(s)[1]  # what the attention of these tokens left (and its append to the pages)
        s["sig"] = torch.rand((1, R * cap, Hq), generator=g, device="cuda") * 0.1
    return s


def _evict_inputs(case, seed):
    """A decode state in the middle of its life: scattered pages, slots out of order, a ring that has wrapped."""
    g = torch.Generator("cuda").manual_seed(seed)
    L, R, Hq, Hkv, P = case["L"], case["R"], case["Hq"], case["Hkv"], case["P"]
    kh, vh = WIDTHS[case["scheme"]]
    ctx = _ragged(case["ctx_lo"], case["ctx_hi"], R, g)
    cap = _up(max(1, case["ctx_hi"]), 16)
    pmax = -(-cap // P) + 1
    U = L * R * Hkv
    pos = torch.arange(cap, device="cuda")
    held = (pos < ctx.view(1, R, 1, 1)).expand(L, R, Hkv, cap).reshape(U, cap)
    x = torch.rand((U, cap), generator=g, device="cuda")
    cls = ((x < case["hi"]).to(torch.int8) + (x < case["hi"] + case["lo"]).to(torch.int8)) * held
    n_hi, n_lo = (cls == 2).sum(1), (cls == 1).sum(1)
    hdr = torch.stack([n_hi, n_lo, (n_hi + P - 1) // P, (n_lo + 2 * P - 1) // (2 * P)], 1).to(torch.int32)
    d = (hdr[:, 2] + hdr[:, 3]).long()
    total = int(d.sum())
    # one page of room and one in a hundred, and an eighth of the pool free
    F = int(1.01 * 1.125 * U * (case["hi"] / P + case["lo"] / (2 * P)) * 0.5 * (case["ctx_lo"] + case["ctx_hi"]))
    F = max(F + 4 * U + 16, total + 16)
    order = torch.randperm(F, generator=g, device="cuda").to(torch.int32)
    ids, free_ids = order[:total], order[total:]
    u = torch.repeat_interleave(torch.arange(U, device="cuda"), d)
    k = torch.arange(total, device="cuda") - (d.cumsum(0) - d)[u]
    head = 5 * F + int(torch.randint(0, F, (1,), generator=g, device="cuda"))
    slot_of = torch.full((U, cap), -1, dtype=torch.int32, device="cuda")
    pages = torch.randint(-2 ** 62, 2 ** 62, (F * _page_bytes(case) // 8,), generator=g, device="cuda")
    pages = pages.view(torch.uint8).view(F, -1)
    where = pages[:, 16 * (kh + vh + 1) * P:].unflatten(1, (2 * P, 4))
    where.fill_(255)  # position -1 in the unused slots
    small = dict(cursors=torch.tensor([head, head + F - total], dtype=torch.int64, device="cuda"), hdr=hdr,
                 fwd=torch.full((U, pmax), -1, dtype=torch.int32, device="cuda"),
                 free_list=torch.full((F,), -1, dtype=torch.int32, device="cuda"),
                 rev_unit=torch.full((F,), -1, dtype=torch.int32, device="cuda"),
                 rev_idx=torch.full((F,), -1, dtype=torch.int32, device="cuda"),
                 page_cls=torch.zeros(F, dtype=torch.uint8, device="cuda"))
    small["fwd"][u, k] = ids
    small["free_list"][(head + torch.arange(F - total, device="cuda")) % F] = free_ids
    small["rev_unit"][ids.long()], small["rev_idx"][ids.long()] = u.to(torch.int32), k.to(torch.int32)
    small["page_cls"][ids.long()] = torch.where(k < hdr[:, 2][u], 2, 1).to(torch.uint8)
    for c, slots in ((2, P), (1, 2 * P)):  # each list's tokens in a drawn order: earlier steps filled its holes
        unit, at = (cls == c).nonzero(as_tuple=True)
        n = (cls == c).sum(1)
        mixed = (unit + torch.rand(unit.numel(), generator=g, device="cuda", dtype=torch.float64)).argsort()
        at = at[mixed]
        rank = torch.arange(unit.numel(), device="cuda") - (n.cumsum(0) - n)[unit]
        slot_of[unit, at] = rank.to(torch.int32)
        page = small["fwd"][unit, (hdr[:, 2].long()[unit] if c == 1 else 0) + rank // slots].long()
        where[page, rank % slots] = at.to(torch.int32).view(-1, 1).view(torch.uint8)
    rows = lambda t: t.view(L, R, Hkv, cap).permute(0, 1, 3, 2).contiguous()  # noqa: E731
    small["classes"], small["slot_of"] = rows(cls.to(torch.uint8)), rows(slot_of)
    # log-normal significance whose mean falls with a token's age; counts of a prompt's positions
    sig = torch.exp(2.0 * torch.randn((L, R, cap, Hq), generator=g, device="cuda"))
    cnt = (ctx.view(R, 1) - pos.view(1, cap)).clamp(min=1).to(torch.int32)
    sig *= cnt.view(1, R, cap, 1) / ctx.clamp(min=1).view(1, R, 1, 1)
    budgets = (case["keep"] * (case["hi"] + case["lo"]) * ctx).to(torch.int32)
    n_cut = max(1, int(round(case["share"] * R)))
    budgets[torch.randperm(R, generator=g, device="cuda")[n_cut:]] = -1
    # the tables and rows lie in one piece, so that a pass can start from the same state again with one copy
    at, size = {}, 0
    for name, t in small.items():
        at[name] = (size, t)
        size = _up(size + t.numel() * t.element_size(), 256)
    arena = torch.zeros(size, dtype=torch.uint8, device="cuda")
    s = dict(case=case, L=L, R=R, Hq=Hq, Hkv=Hkv, U=U, cap=cap, pmax=pmax, F=F, ctx=ctx, budgets=budgets, sig=sig,
             cnt=cnt, pages=pages)
    for name, (o, t) in at.items():
        s[name] = arena[o:o + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        s[name].copy_(t)
    s["live"], s["start"] = arena, arena.clone()
    # of the pages' bytes a pass changes holes, which the next pass fills again with the same, and the last kept page
    # of each list, whose end it clears: those pages are put back
    kept = _kept(s)
    edge = []
    for c, slots, first in ((2, P, 0 * hdr[:, 2]), (1, 2 * P, hdr[:, 2])):
        need = ((kept & (cls == c)).sum(1) + slots - 1) // slots
        e = s["fwd"].gather(1, (first + need - 1).clamp(min=0).long().view(-1, 1))[:, 0]
        edge.append(e[need > 0])
    s["edge"] = torch.cat(edge).long()
    s["edge_start"] = pages.view(torch.int64)[s["edge"]]
    return s


def prepare(case, seed):
    evict = case["op"] == "evict"
    s = (_evict_inputs if evict else _chunk_inputs)(dict(case), int(seed))
    if own:  # the handles that a program keeps: the pool, tables, pages, outputs, a workspace
        from differentiated_kv_cache_dkv_gb300 import libdkv
        s["lib"] = libdkv
        if evict:
            s["pool"] = libdkv.DevicePool.from_tensors(
                case["P"], case["scheme"], s["free_list"], s["cursors"], s["rev_unit"], s["rev_idx"], s["page_cls"],
                s["pages"], torch.zeros(1, dtype=torch.int32, device="cuda"))
            s["tables"] = libdkv.DeviceTables.from_tensors(s["fwd"], s["hdr"])
            size = libdkv.dkv_evict_workspace_size(_evict_batch(s), s["pool"], s["tables"])
        else:
            s["pool"] = libdkv.DevicePool(1, 2)  # its status word alone is used
            s["pages"] = libdkv.ChunkPages.from_tensors(s["k"], s["v"], s["table"])
            s["out"] = torch.empty((1, s["T"], s["Hq"], D), dtype=torch.bfloat16, device="cuda")
            if case["op"] == "chunk":
                s["lse"] = torch.empty((1, s["T"], s["Hq"]), dtype=torch.float32, device="cuda")
            size = libdkv.dkv_chunk_workspace_size(_chunk_batch(s), s["pages"])
        s["work"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s


def _chunk_batch(s):
    return s["lib"].make_chunk_batch(s["Hkv"], s["cap"], s["q"], s["new"], s["ctx"], s["max_new"], SCALE,
                                     k_new=s["kn"], v_new=s["vn"], out=s["out"], lse=s["lse"])


def _evict_batch(s):
    case = s["case"]
    return s["lib"].make_evict_batch(s["L"], s["R"], s["Hq"], s["Hkv"], s["cap"], s["budgets"], s["ctx"], s["sig"],
                                     s["classes"], s["slot_of"], sig_cnt=s["cnt"] if case["average"] else None,
                                     sinks=case["sinks"], window=case["window"])


# ---------------------------------------------------------------- operators --

def run(s):
    op = s["case"]["op"]
    if op == "evict":  # the same state again (both sides pay for it)
        s["live"].copy_(s["start"])
        s["pages"].view(torch.int64)[s["edge"]] = s["edge_start"]
    return (_RUN_OWN if own else _RUN)[op](s)


def _run_chunk(s):
    s["lib"].dkv_chunk_attention(_chunk_batch(s), s["pages"], s["pool"], s["work"])
    return _attended(s, s["out"], s["lse"])


def _run_chunk_sig(s):
    s["lib"].dkv_chunk_significance(_chunk_batch(s), s["pages"], s["sig"], s["pool"])
    return s["sig"]


def _run_evict(s):
    s["lib"].dkv_evict(_evict_batch(s), s["pool"], s["tables"], s["work"])
    return _evicted(s)


_RUN_OWN = {"chunk": _run_chunk, "chunk_sig": _run_chunk_sig, "evict": _run_evict}


def _attended(s, out, lse):
    return {"out": out, "lse": lse, "k_pages": s["k"].view(torch.int64), "v_pages": s["v"].view(torch.int64)}


def _evicted(s):
    return dict({k: s[k] for k in ("cursors", "hdr", "fwd", "free_list", "rev_unit", "rev_idx", "page_cls", "classes",
                                   "slot_of")}, pages=s["pages"].view(torch.int64))


# -------------------------------------------------------------- plain forms --

def _padded(s):
    """Where token i of request r lies among the packed tokens [R][max_new], and which exist."""
    i = torch.arange(s["max_new"], device="cuda")
    new = s["new"].long()
    ok = i < new.view(-1, 1)
    return ((new.cumsum(0) - new).view(-1, 1) + i).clamp(max=max(s["T"] - 1, 0)), ok


def _append(s):
    """The new tokens' K and V go to their positions' places in the pages."""
    at, ok = _padded(s)
    pos = (s["ctx"].view(-1, 1) + torch.arange(s["max_new"], device="cuda")).clamp(max=s["cap"] - 1)
    page = s["table"].gather(1, pos // s["B"])[ok].long()
    slot = (pos % s["B"])[ok]
    s["k"][0, page, slot] = s["kn"][0, at[ok]]
    s["v"][0, page, slot] = s["vn"][0, at[ok]]


def _rows(s, x):
    """fp32 rows [R][Hkv][N][128] of every position, zeros behind a request's last."""
    n = torch.arange(s["max_len"], device="cuda")
    ok = n < (s["ctx"] + s["new"]).view(-1, 1)
    page = s["table"][:, n // s["B"]].clamp(min=0).long()
    y = torch.where(ok.view(*ok.shape, 1, 1), x[0, page, n % s["B"]].float(), 0.0)
    return y.permute(0, 2, 1, 3)


def _logits(s):
    """Logits [R][Hkv][i, g][N] of every new token, and which pairs exist."""
    at, ok = _padded(s)
    G, n = s["Hq"] // s["Hkv"], s["max_new"]
    q = s["q"][0, at].float().view(s["R"], n, s["Hkv"], G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = (q * SCALE) @ _rows(s, s["k"]).transpose(2, 3)
    last = s["ctx"].view(-1, 1) + torch.arange(n, device="cuda")
    seen = (torch.arange(s["max_len"], device="cuda") <= last.unsqueeze(-1)) & ok.unsqueeze(-1)
    return x, seen.repeat_interleave(G, 1).unsqueeze(1), at, ok


def _plain_attention(s):
    _append(s)
    x, seen, at, ok = _logits(s)
    x.masked_fill_(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = (x @ _rows(s, s["v"])) / torch.where(z > 0, z, torch.ones_like(z))
    G = s["Hq"] // s["Hkv"]
    o = o.unflatten(2, (s["max_new"], G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = (m + z.log()).squeeze(-1).unflatten(2, (s["max_new"], G)).permute(0, 2, 1, 3).flatten(2, 3)
    return o[ok].bfloat16().unsqueeze(0), lse[ok].unsqueeze(0)


def _plain_chunk(s):
    return _attended(s, *_plain_attention(s))


def _plain_chunk_sig(s):
    x, seen, at, ok = _logits(s)
    R, Hkv, n, G = s["R"], s["Hkv"], s["max_new"], s["Hq"] // s["Hkv"]
    lse = s["lse"][0, at].view(R, n, Hkv, G).permute(0, 2, 1, 3).flatten(2, 3)
    x.sub_(lse.unsqueeze(-1)).exp_()
    x.masked_fill_(~seen, 0.0)
    p = x.unflatten(2, (n, G)).sum(2).permute(0, 3, 1, 2).flatten(2, 3)  # [R][N][Hq]
    pos = torch.arange(s["max_len"], device="cuda")
    held, end = s["ctx"].view(-1, 1), (s["ctx"] + s["new"]).view(-1, 1)
    sig = s["sig"].view(R, s["cap"], s["Hq"])[:, :s["max_len"]]
    fresh = torch.where(((pos >= held) & (pos < end)).unsqueeze(-1), p, sig)
    sig.copy_(torch.where((pos < held).unsqueeze(-1), sig + p, fresh))
    return s["sig"]


def _units(s, rows):
    """[L][R][cap][Hkv] as [U][cap]."""
    return rows.permute(0, 1, 3, 2).reshape(s["U"], s["cap"])


def _kept(s):
    """Which positions of each unit stay [U][cap]."""
    case, R, Hkv, cap = s["case"], s["R"], s["Hkv"], s["cap"]
    score = s["sig"].unflatten(3, (Hkv, -1)).amax(-1)
    if case["average"]:
        score = score / s["cnt"].float().view(1, R, cap, 1)
    unit = lambda t: t.view(1, R, 1).expand(s["L"], R, Hkv).reshape(-1, 1)  # noqa: E731
    ctx, budget = unit(s["ctx"]), unit(s["budgets"])
    pos = torch.arange(cap, device="cuda")
    held = (_units(s, s["classes"]) != 0) & (pos < ctx)
    safe = held & ((pos < case["sinks"]) | (pos >= ctx - case["window"]))
    key = torch.where(safe, float("inf"), torch.where(held, _units(s, score), -1.0))
    order = key.sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, pos.expand_as(order))
    return held & ((rank < budget) | safe | (budget < 0))


def _plain_evict(s):
    case, P, F = s["case"], s["case"]["P"], s["F"]
    kh, vh = WIDTHS[case["scheme"]]
    keep, cls, slot = _kept(s), _units(s, s["classes"]), _units(s, s["slot_of"])
    gone = (cls != 0) & ~keep & (torch.arange(s["cap"], device="cuda") <
                                 s["ctx"].view(1, -1, 1).expand(s["L"], -1, s["Hkv"]).reshape(-1, 1))
    pages, old = s["pages"], s["hdr"].clone()
    meta = pages[:, 16 * (kh + vh) * P:].unflatten(1, (3 * P, 8))[:, :2 * P]
    where = pages[:, 16 * (kh + vh + 1) * P:].unflatten(1, (2 * P, 4))
    for c, slots, half, first in ((2, P, 1, 0 * old[:, 2]), (1, 2 * P, 2, old[:, 2])):
        n = old[:, 2 - c]
        regions = (pages[:, :16 * kh * P].unflatten(1, (slots, 16 * kh // half)),
                   pages[:, 16 * kh * P:16 * (kh + vh) * P].unflatten(1, (slots, 16 * vh // half)), meta, where)
        u, p = (keep & (cls == c)).nonzero(as_tuple=True)
        stays = torch.zeros((s["U"], s["cap"]), dtype=torch.bool, device="cuda")
        stays[u, slot[u, p].long()] = True
        at = torch.empty((s["U"], s["cap"]), dtype=torch.int64, device="cuda")
        at[u, slot[u, p].long()] = p
        k = stays.sum(1, keepdim=True)
        i = torch.arange(s["cap"], device="cuda")
        hu, hole = (~stays & (i < k)).nonzero(as_tuple=True)
        mu, mover = (stays & (i >= k)).nonzero(as_tuple=True)  # as many a unit, both ascending
        page = lambda u, x: s["fwd"][u, first[u] + x // slots].long()  # noqa: E731
        src, dst = page(mu, mover), page(hu, hole)
        for r in regions:
            r[dst, hole % slots] = r[src, mover % slots]
        slot[mu, at[mu, mover]] = hole.to(torch.int32)
        need = (k + slots - 1) // slots
        cu, x = ((i >= k) & (i < n.view(-1, 1)) & (i < need * slots)).nonzero(as_tuple=True)
        for r, fill in zip(regions, (0, 0, 0, 255)):
            r[page(cu, x), x % slots] = fill
        s["hdr"][:, 2 - c], s["hdr"][:, 4 - c] = k[:, 0].to(torch.int32), need[:, 0].to(torch.int32)
    back = lambda t: t.view(s["L"], s["R"], s["Hkv"], s["cap"]).permute(0, 1, 3, 2)  # noqa: E731
    s["classes"].masked_fill_(back(gone), 0)
    s["slot_of"].copy_(back(slot.masked_fill(gone, -1)))
    j = torch.arange(s["pmax"], device="cuda")
    have, need = old[:, 2:].long(), s["hdr"][:, 2:].long()
    of_hi, of_lo = j < have[:, :1], (j >= have[:, :1]) & (j < have.sum(1, keepdim=True))
    stays = (of_hi & (j < need[:, :1])) | (of_lo & (j < have[:, :1] + need[:, 1:]))
    free = s["fwd"][(of_hi | of_lo) & ~stays]  # in the order of units and of their rows
    tail = s["cursors"][1]
    s["free_list"][(tail + torch.arange(free.numel(), device="cuda")) % F] = free
    s["rev_unit"][free.long()], s["rev_idx"][free.long()], s["page_cls"][free.long()] = -1, -1, 0
    u, x = stays.nonzero(as_tuple=True)
    ids = s["fwd"][u, x]
    to = (stays.cumsum(1) - 1)[u, x]
    s["fwd"].fill_(-1)
    s["fwd"][u, to] = ids
    s["rev_idx"][ids.long()] = to.to(torch.int32)
    s["cursors"][1] += free.numel()
    return _evicted(s)


_RUN = {"chunk": _plain_chunk, "chunk_sig": _plain_chunk_sig, "evict": _plain_evict}


# ------------------------------------------------------------------ 64 bits --

def exact(case, seed):
    if case["op"] == "evict":
        return None  # nothing is computed: whole numbers and copies
    s = _chunk_inputs(dict(case), int(seed))
    Hq, Hkv, G, B, cap = s["Hq"], s["Hkv"], s["Hq"] // s["Hkv"], s["B"], s["cap"]
    out = torch.zeros((1, s["T"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((1, s["T"], Hq), dtype=torch.float64, device="cuda")
    sig = s["sig"].double() if "sig" in s else None
    ctx, new, t0 = s["ctx"].tolist(), s["new"].tolist(), 0
    for r in range(s["R"]):
        c, n, t1 = ctx[r], new[r], t0 + new[r]
        if n == 0:
            continue
        ids = s["table"][r, :-(-(c + n) // B)].long()
        k, v = (torch.cat([x[0, ids].flatten(0, 1)[:c], y[0, t0:t1]]).double()
                for x, y in ((s["k"], s["kn"]), (s["v"], s["vn"])))
        later = torch.ones((n, n), device="cuda").triu(1).bool()
        for h in range(Hq):
            x = s["q"][0, t0:t1, h].double() @ k[:, h // G].T * SCALE
            x[:, c:].masked_fill_(later, float("-inf"))
            if sig is None:
                e = torch.logsumexp(x, 1)
                lse[0, t0:t1, h] = e
                out[0, t0:t1, h] = torch.exp(x - e.view(-1, 1)) @ v[:, h // G]
            else:
                p = torch.exp(x - s["lse"][0, t0:t1, h].double().view(-1, 1)).sum(0)
                rows = sig[0, r * cap:(r + 1) * cap, h]
                rows[:c] += p[:c]
                rows[c:c + n] = p[c:]
        t0 = t1
    return sig if sig is not None else {"out": out, "lse": lse, "k_pages": None, "v_pages": None}
