"""What the cache operators are measured on: several tokens a request over the
quantised pages (attention, and the significance its tokens receive), and the
page operations of a pool that serves many requests (fork, release, defrag).

The plain forms below state each operator in elementary tensor operations in
32 bits; with `own` set the same inputs go through libdkv's entry points.  A
unit is (layer l, request r, KV head h), u = (l R + r) Hkv + h; the page
layout, the precision schemes and the tables are those of include/dkv.h.
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
    tiny = dict(L=1, Hq=8, Hkv=2, P=16, scheme=0, hi=0.5, lo=0.4)
    llama = dict(L=1, Hq=32, Hkv=8, P=16, scheme=0, hi=0.5, lo=0.39)
    qwen = dict(L=1, Hq=28, Hkv=4, P=32, scheme=0, hi=0.22, lo=0.336)
    return [
        # one request of the tiny configuration takes four tokens at once: the smallest call, latency alone
        dict(tiny, name="extend tiny", op="extend", R=1, ctx_lo=512, ctx_hi=512, new_lo=4, new_hi=4),
        # a decode batch scores up to eight drafted tokens a request over ragged contexts: bound by the pages' bytes
        dict(llama, name="extend drafts", op="extend", R=64, ctx_lo=2048, ctx_hi=8192, new_lo=1, new_hi=8),
        # turns of a conversation: ragged suffixes, none for some requests, on an odd group of seven query heads,
        # 4-bit keys
        dict(qwen, name="extend ragged", op="extend", R=16, ctx_lo=0, ctx_hi=5001, new_lo=0, new_hi=333, scheme=2),
        # a chunk of a long prompt over what the earlier chunks left in the cache: bound by the two products
        dict(llama, name="extend chunk", op="extend", R=4, ctx_lo=16384, ctx_hi=16384, new_lo=1024, new_hi=1024),
        # the accepted drafts of that decode batch give their tokens' significance
        dict(llama, name="significance drafts", op="significance", R=64, ctx_lo=2048, ctx_hi=8192, new_lo=1,
             new_hi=8),
        # a whole chunk does
        dict(llama, name="significance chunk", op="significance", R=4, ctx_lo=8192, ctx_hi=8192, new_lo=1024,
             new_hi=1024),
        # one request of the tiny configuration is forked once: latency
        dict(tiny, name="fork tiny", op="fork", R=4, ctx_lo=512, ctx_hi=512, n=1),
        # eight sequences of a 32-layer cache are forked (parallel sampling after a shared prompt)
        dict(llama, name="fork prompts", op="fork", L=32, R=16, ctx_lo=2048, ctx_hi=6144, n=8),
        # one finished request of the tiny configuration leaves
        dict(tiny, name="release tiny", op="release", R=4, ctx_lo=512, ctx_hi=512, n=1),
        # eight finished requests of a 32-layer batch leave at once
        dict(llama, name="release batch", op="release", L=32, R=16, ctx_lo=1024, ctx_hi=8192, n=8),
        # the pool of the tiny configuration is packed
        dict(tiny, name="defrag tiny", op="defrag", R=4, ctx_lo=512, ctx_hi=512, live=0.5),
        # a scattered 32-layer pool of odd page size is packed to hand its upper part back
        dict(qwen, name="defrag pool", op="defrag", L=28, R=24, ctx_lo=1024, ctx_hi=8192, live=0.6),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("extend", "extend", "extend", "significance", "significance", "fork", "release", "defrag"))
    g, hkv = rng.choice(((1, 8), (2, 5), (3, 2), (4, 8), (4, 2), (5, 3), (7, 4), (8, 8), (8, 1)))
    hi = rng.choice((0.0, 0.1, 0.22, 0.5, 0.9, 1.0))
    case = dict(op=op, L=1, Hq=g * hkv, Hkv=hkv, P=rng.choice((2, 6, 8, 16, 16, 32, 64)), scheme=rng.randrange(3),
                hi=hi, lo=rng.choice((0.0, 0.3, 1.0)) * (1.0 - hi))
    if op in ("extend", "significance"):
        case["R"] = log(1, 64)
        case["ctx_hi"] = log(1, 16384)
        case["ctx_lo"] = rng.choice((0, case["ctx_hi"] // 3, case["ctx_hi"]))
        case["new_hi"] = log(1, 1024)
        case["new_lo"] = rng.choice((0, 1, case["new_hi"]))
        most = 4 * 32 * 1024 * (17408 if op == "extend" else 9216)
        while case["R"] * case["Hq"] * case["new_hi"] * (case["ctx_hi"] + case["new_hi"]) > most or \
                case["R"] * case["Hkv"] * case["ctx_hi"] > 64 * 8 * 8192:
            k = rng.choice(("R", "new_hi", "ctx_hi"))
            case[k] = max(1, case[k] // 2)
            case["ctx_lo"] = min(case["ctx_lo"], case["ctx_hi"])
            case["new_lo"] = min(case["new_lo"], case["new_hi"])
        return case
    case["L"] = log(1, 32)
    case["R"] = log(2, 32)
    case["ctx_hi"] = log(1, 8192)
    case["ctx_lo"] = rng.choice((0, case["ctx_hi"] // 3, case["ctx_hi"]))
    case["hi"] = hi or 0.05
    while case["L"] * case["R"] * case["Hkv"] * (case["ctx_hi"] + 4 * case["P"]) > 32 * 16 * 8 * 4096:
        k = rng.choice(("L", "R", "ctx_hi"))
        case[k] = max(2 if k == "R" else 1, case[k] // 2)
        case["ctx_lo"] = min(case["ctx_lo"], case["ctx_hi"])
    if op == "defrag":
        case["live"] = rng.choice((0.1, 0.5, 0.8, 0.97))
    else:
        case["n"] = rng.randint(1, case["R"] // 2 if op == "fork" else case["R"])
    return case


def work(case):
    ctx, P, hq, hkv = 0.5 * (case["ctx_lo"] + case["ctx_hi"]), case["P"], case["Hq"], case["Hkv"]
    kh, vh = WIDTHS[case["scheme"]]
    hi, lo = case["hi"], case["lo"]
    if case["op"] in ("extend", "significance"):
        n = max(0.5 * (case["new_lo"] + case["new_hi"]), 1e-3)
        rows, units = case["R"] * n * hq, case["R"] * hkv
        pairs = rows * ((hi + lo) * ctx + 0.5 * n)
        if case["op"] == "extend":  # codes and metadata of each held token, q, the new K and V, the outputs
            held = units * ctx * (hi * (16 * (kh + vh) + 8) + lo * (8 * (kh + vh) + 8))
            return {"bytes": held + rows * (256 + 256 + 4) + case["R"] * n * hkv * 512, "flops": 4.0 * D * pairs}
        held = units * ctx * (hi * (16 * kh + 8) + lo * (8 * kh + 8))  # K codes, metadata's K half, positions
        sums = case["R"] * ctx * (hi + lo) * hq * 8 + case["R"] * n * hq * 4
        return {"bytes": held + sums + rows * 260 + case["R"] * n * hkv * 256, "flops": 2.0 * D * pairs}
    per_unit = hi * ctx / P + lo * ctx / (2 * P)
    if case["op"] == "fork":
        units = case["L"] * case["n"] * hkv
        rows = case["L"] * case["n"] * ctx * (5 * hkv + 4 * hq)  # classes, slots, significance of the context
        return {"bytes": units * (per_unit * (2 * _page_bytes(case) + 4 + 4 + 4 + 9) + 32) + 2 * rows, "flops": 0}
    if case["op"] == "release":
        return {"bytes": case["L"] * case["n"] * hkv * (per_unit * (4 + 4 + 4 + 4 + 9) + 32), "flops": 0}
    pages = case["L"] * case["R"] * hkv * per_unit
    moved = pages * (1 - case["live"])
    total = pages / case["live"]
    return {"bytes": moved * (2 * _page_bytes(case) + 4 + 4 + 18) + total * 1 + (total - pages) * 4, "flops": 0}


# ------------------------------------------------------------------ inputs --

def _ragged(lo, hi, n, g):
    """n lengths spread over [lo, hi], both ends among them, in a drawn order (their sum is the case's own)."""
    x = hi - (torch.arange(n, device="cuda") * (hi - lo)) // max(n - 1, 1)
    return x[torch.randperm(n, generator=g, device="cuda")].to(torch.int32)


def _pool_pages(case, requests):
    """Pages that hold the lists of so many requests of the mean length, with room for the draw of their classes."""
    ctx, units = 0.5 * (case["ctx_lo"] + case["ctx_hi"]), case["L"] * requests * case["Hkv"]
    mean = units * ctx * (case["hi"] / case["P"] + case["lo"] / (2 * case["P"]))
    return int(1.02 * mean + 8 * mean ** 0.5) + 2 * units + 16


def _quantise(x, bits):
    """Codes [n][128 bits / 8], and fp16 scale and zero, of rows x [n][128]."""
    n = float(2 ** bits - 1)
    mn, mx = x.amin(1, keepdim=True), x.amax(1, keepdim=True)
    s = ((mx - mn) / n).half()
    s = torch.where((s == 0) & (mx > mn), torch.full_like(s, 2.0 ** -24), s)
    z = mn.half()
    sf = s.float()
    q = ((x - z.float()) / torch.where(sf == 0, torch.ones_like(sf), sf)).round().clamp(0, n)
    q = q.to(torch.int32).view(x.shape[0], -1, 8 // bits)
    sh = torch.arange(0, 8, bits, device=x.device, dtype=torch.int32)
    return (q << sh).sum(-1).to(torch.uint8), torch.cat([s, z], 1)


def _fill(pages, case, ids, slot, pos, kbits, vbits, slots, base, which, outlier, g):
    """Writes drawn K and V rows of one class into (page, slot) of the pages."""
    kh, vh = WIDTHS[case["scheme"]]
    P = case["P"]
    moff = 16 * (kh + vh) * P
    at = 0
    for bits, width in ((kbits, kh), (vbits, vh)):
        region = pages[:, at:at + 16 * width * P].unflatten(1, (slots, 16 * bits))
        meta = pages[:, moff:moff + 16 * P].unflatten(1, (2 * P, 8))
        for a in range(0, ids.numel(), 1 << 20):
            sl = slice(a, a + (1 << 20))
            x = torch.randn((ids[sl].numel(), D), generator=g, device="cuda") * outlier[which][base[sl]]
            c, m = _quantise(x.bfloat16().float(), bits)
            region[ids[sl], slot[sl]] = c
            meta[:, :, 4 * which:4 * which + 4][ids[sl], slot[sl]] = m.view(torch.uint8)
        at += 16 * width * P
        which += 1
    where = pages[:, moff + 16 * P:].unflatten(1, (2 * P, 4))
    where[ids, slot] = pos.to(torch.int32).view(-1, 1).view(torch.uint8)


def _lists(case, ctx, L, g):
    """Classes of every position [U][N] (2 high, 1 low, 0 pruned), the lists' lengths and pages [U] of L layers."""
    N = max(1, int(ctx.max()))
    U = L * ctx.numel() * case["Hkv"]
    x = torch.rand((U, N), generator=g, device="cuda")
    held = torch.arange(N, device="cuda") < ctx.view(1, -1, 1, 1).expand(L, -1, case["Hkv"], 1).reshape(U, 1)
    cls = ((x < case["hi"]).to(torch.int8) + (x < case["hi"] + case["lo"]).to(torch.int8)) * held
    n_hi, n_lo = (cls == 2).sum(1), (cls == 1).sum(1)
    P = case["P"]
    hdr = torch.stack([n_hi, n_lo, (n_hi + P - 1) // P, (n_lo + 2 * P - 1) // (2 * P)], 1).to(torch.int32)
    return cls, hdr


def _tables(hdr, pmax, ids):
    """Forward rows of the units whose pages are ids, in unit order."""
    d = (hdr[:, 2] + hdr[:, 3]).long()
    u = torch.repeat_interleave(torch.arange(d.numel(), device="cuda"), d)
    k = torch.arange(u.numel(), device="cuda") - (d.cumsum(0) - d)[u]
    fwd = torch.full((d.numel(), pmax), -1, dtype=torch.int32, device="cuda")
    fwd[u, k] = ids
    return fwd, u, k


def _attention_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    R, Hq, Hkv, P = case["R"], case["Hq"], case["Hkv"], case["P"]
    ctx = _ragged(case["ctx_lo"], case["ctx_hi"], R, g)
    new = _ragged(case["new_lo"], case["new_hi"], R, g)
    T = int(new.sum())
    cap = _up(case["ctx_hi"] + case["new_hi"], 16)
    pmax = -(-cap // P) + 1
    cls, hdr = _lists(case, ctx, 1, g)
    total = int((hdr[:, 2] + hdr[:, 3]).sum())
    F = _pool_pages(case, R + 1)
    ids = torch.randperm(F, generator=g, device="cuda")[:total].to(torch.int32)
    fwd, u, k = _tables(hdr, pmax, ids)
    kh, vh = WIDTHS[case["scheme"]]
    pages = torch.zeros((F, _page_bytes(case)), dtype=torch.uint8, device="cuda")
    pages[:, 16 * (kh + vh) * P + 16 * P:] = 255  # position -1 in the unused slots
    outlier = [torch.ones((R * Hkv, D), device="cuda") for _ in range(2)]
    for o in outlier:  # three channels of a KV head are ten times as large
        o.view(R, Hkv, D).scatter_(2, torch.rand((Hkv, D), generator=g, device="cuda").argsort(1)[:, :3]
                                   .expand(R, -1, -1), 10.0)
    for c, kb, vb, slots in ((2, kh, vh, P), (1, kh // 2, vh // 2, 2 * P)):
        unit, pos = (cls == c).nonzero(as_tuple=True)
        n = (cls == c).sum(1)
        rank = torch.arange(unit.numel(), device="cuda") - (n.cumsum(0) - n)[unit]
        first = hdr[:, 2].long()[unit] if c == 1 else 0
        page = fwd[unit, first + rank // slots].long()
        _fill(pages, case, page, rank % slots, pos, kb, vb, slots, unit, 0, outlier, g)
    q = torch.randn((1, T, Hq, D), generator=g, device="cuda").bfloat16()
    kn = (torch.randn((1, T, Hkv, D), generator=g, device="cuda") * outlier[0][:Hkv]).bfloat16()
    vn = (torch.randn((1, T, Hkv, D), generator=g, device="cuda") * outlier[1][:Hkv]).bfloat16()
    rev_unit = torch.full((F,), -1, dtype=torch.int32, device="cuda")
    rev_idx = rev_unit.clone()
    page_cls = torch.zeros(F, dtype=torch.uint8, device="cuda")
    rev_unit[ids.long()], rev_idx[ids.long()] = u.to(torch.int32), k.to(torch.int32)
    page_cls[ids.long()] = torch.where(k < hdr[:, 2][u], 2, 1).to(torch.uint8)
    free = torch.full((F,), -1, dtype=torch.int32, device="cuda")
    free[:F - total] = (page_cls == 0).nonzero()[:, 0].to(torch.int32)
    s = dict(case=case, R=R, Hq=Hq, Hkv=Hkv, cap=cap, pmax=pmax, F=F, T=T, ctx=ctx, new=new, fwd=fwd, hdr=hdr,
             pages=pages, q=q, kn=kn, vn=vn, rev_unit=rev_unit, rev_idx=rev_idx, page_cls=page_cls, free_list=free,
             cursors=torch.tensor([0, F - total], dtype=torch.int64, device="cuda"), max_new=case["new_hi"],
             max_ctx=max(1, case["ctx_hi"]))
    if case["op"] == "significance":
        s["lse"] = _plain_attention(s)[1]  # what the attention over these tokens left
        s["acc"] = torch.minimum(new, _ragged(0, case["new_hi"], R, g)) if case["new_hi"] < 64 else new
        s["sig"] = torch.rand((1, R * cap, Hq), generator=g, device="cuda") * 0.1
    return s


def _pool_inputs(case, seed):
    """A pool in the middle of its life: scattered pages, a ring of free pages that has wrapped."""
    g = torch.Generator("cuda").manual_seed(seed)
    L, R, Hq, Hkv, P, op = case["L"], case["R"], case["Hq"], case["Hkv"], case["P"], case["op"]
    ctx = _ragged(case["ctx_lo"], case["ctx_hi"], R, g)
    who = torch.randperm(R, generator=g, device="cuda")
    src = dst = who[:0]
    if op == "fork":
        dst = who[:case["n"]]
        src = who[case["n"]:][torch.randint(0, R - case["n"], (case["n"],), generator=g, device="cuda")]
        ctx[dst] = 0
    if op == "release":
        src = who[:case["n"]]
    cap = _up(max(1, case["ctx_hi"]), 16)
    pmax = -(-cap // P) + 1
    U = L * R * Hkv
    cls, hdr = _lists(case, ctx, L, g)
    d = (hdr[:, 2] + hdr[:, 3]).long()
    total = int(d.sum())
    if op == "fork":
        F = _pool_pages(case, R) + _pool_pages(dict(case, ctx_lo=case["ctx_hi"]), case["n"])
    else:
        F = int(_pool_pages(case, R + 1) / case.get("live", 1.0))
    order = torch.randperm(F, generator=g, device="cuda").to(torch.int32)
    ids, free_ids = order[:total], order[total:]
    fwd, u, k = _tables(hdr, pmax, ids)
    head = 5 * F + int(torch.randint(0, F, (1,), generator=g, device="cuda"))
    slots = (head + torch.arange(F - total, device="cuda")) % F
    small = dict(cursors=torch.tensor([head, head + F - total], dtype=torch.int64, device="cuda"), hdr=hdr, fwd=fwd,
                 free_list=torch.full((F,), -1, dtype=torch.int32, device="cuda"),
                 rev_unit=torch.full((F,), -1, dtype=torch.int32, device="cuda"),
                 rev_idx=torch.full((F,), -1, dtype=torch.int32, device="cuda"),
                 page_cls=torch.zeros(F, dtype=torch.uint8, device="cuda"))
    small["free_list"][slots] = free_ids
    small["rev_unit"][ids.long()], small["rev_idx"][ids.long()] = u.to(torch.int32), k.to(torch.int32)
    small["page_cls"][ids.long()] = torch.where(k < hdr[:, 2][u], 2, 1).to(torch.uint8)
    # the pool's tables lie in one piece, so that a pass can start from the same state again with one small copy
    at, size = {}, 0
    for name, t in small.items():
        at[name] = (size, t)
        size = _up(size + t.numel() * t.element_size(), 256)
    arena = torch.zeros(size, dtype=torch.uint8, device="cuda")
    s = dict(case=case, L=L, R=R, Hq=Hq, Hkv=Hkv, U=U, cap=cap, pmax=pmax, F=F, src=src.to(torch.int32),
             dst=dst.to(torch.int32), ctx=ctx)
    for name, (o, t) in at.items():
        s[name] = arena[o:o + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        s[name].copy_(t)
    s["live"] = arena[:at["fwd"][0]] if op == "fork" else arena
    s["start"] = s["live"].clone()
    words = F * _page_bytes(case) // 8
    s["pages"] = torch.randint(-2 ** 62, 2 ** 62, (words,), generator=g, device="cuda").view(torch.uint8).view(F, -1)
    if op == "fork":  # the decode state that goes with the pages
        rows = L * R * cap
        s["classes"] = torch.randint(0, 3, (L, R, cap, Hkv), generator=g, device="cuda", dtype=torch.uint8)
        s["slot_of"] = torch.randint(-1, 999, (L, R, cap, Hkv), generator=g, device="cuda", dtype=torch.int32)
        s["sig"] = torch.rand(rows * Hq, generator=g, device="cuda").view(L, R, cap, Hq)
        s["cnt"] = torch.randint(1, 999, (R, cap), generator=g, device="cuda", dtype=torch.int32)
    return s


def prepare(case, seed):
    s = (_attention_inputs if case["op"] in ("extend", "significance") else _pool_inputs)(dict(case), int(seed))
    if own:  # the handles that a program keeps: the pool, its tables, a workspace
        from differentiated_kv_cache_dkv_gb300 import libdkv
        s["lib"] = libdkv
        s["pool"] = libdkv.DevicePool.from_tensors(
            case["P"], case["scheme"], s["free_list"], s["cursors"], s["rev_unit"], s["rev_idx"], s["page_cls"],
            s["pages"], torch.zeros(1, dtype=torch.int32, device="cuda"))
        s["tables"] = libdkv.DeviceTables.from_tensors(s["fwd"], s["hdr"])
        if case["op"] == "extend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:3], dtype=torch.float32, device="cuda")
            size = libdkv.dkv_extend_workspace_size(_batch(s), s["pool"], s["tables"])
        elif case["op"] == "significance":
            size = 0
        else:
            size = libdkv.dkv_page_ops_workspace_size(s["pool"], s["tables"])
        s["work"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s


def _batch(s):
    return s["lib"].make_extend_batch(1, s["Hkv"], s["cap"], s["q"], s["new"], s["ctx"], s["max_new"], SCALE,
                                      k_new=s["kn"], v_new=s["vn"], out=s.get("out"), lse=s["lse"])


# ---------------------------------------------------------------- operators --

def run(s):
    op = s["case"]["op"]
    if op in ("fork", "release", "defrag"):
        s["live"].copy_(s["start"])  # the same pool again (both sides pay for it)
    if own:
        return _RUN_OWN[op](s)
    return _RUN[op](s)


def _run_extend(s):
    lib = s["lib"]
    lib.dkv_extend_attention(_batch(s), s["pool"], s["tables"], s["work"])
    return {"out": s["out"], "lse": s["lse"]}


def _run_significance(s):
    lib = s["lib"]
    lib.dkv_extend_significance(_batch(s), s["acc"], s["sig"], s["pool"], s["tables"])
    return s["sig"]


def _run_fork(s):
    lib = s["lib"]
    lib.dkv_fork(lib.make_fork_batch(s["L"], s["R"], s["Hq"], s["Hkv"], s["cap"], s["src"], s["dst"], s["ctx"],
                                     classes=s["classes"], slot_of=s["slot_of"], sig_sum=s["sig"], sig_cnt=s["cnt"]),
                 s["pool"], s["tables"], s["work"])
    return _forked(s)


def _run_release(s):
    lib = s["lib"]
    lib.dkv_release(lib.make_release_batch(s["L"], s["R"], s["Hkv"], s["src"]), s["pool"], s["tables"], s["work"])
    return _small(s)


def _run_defrag(s):
    s["lib"].dkv_defrag(s["pool"], s["tables"], s["work"])
    return dict(_small(s), pages=s["pages"].view(torch.int64))


_RUN_OWN = {"extend": _run_extend, "significance": _run_significance, "fork": _run_fork, "release": _run_release,
            "defrag": _run_defrag}


def _small(s):
    return {k: s[k] for k in ("cursors", "hdr", "fwd", "free_list", "rev_unit", "rev_idx", "page_cls")}


def _forked(s):
    return dict(_small(s), pages=s["pages"].view(torch.int64), classes=s["classes"], slot_of=s["slot_of"],
                sig=s["sig"], cnt=s["cnt"])


# -------------------------------------------------------------- plain forms --

def _codes(b, bits):
    sh = torch.arange(0, 8, bits, device=b.device, dtype=torch.uint8)
    return ((b.unsqueeze(-1) >> sh) & (2 ** bits - 1)).flatten(-2).float()


def _held(s, need_v):
    """fp32 K, V [R][Hkv][N][128], positions and which are held, of the two lists one after the other."""
    case, pages, P = s["case"], s["pages"], s["case"]["P"]
    kh, vh = WIDTHS[case["scheme"]]
    meta = pages[:, 16 * (kh + vh) * P:].unflatten(1, (3 * P, 8))[:, :2 * P].view(torch.float16)
    posn = pages[:, 16 * (kh + vh + 1) * P:].unflatten(1, (2 * P, 4)).view(torch.int32)

    def part(slots, half, n, first):
        i = torch.arange(max(1, s["max_ctx"]), device="cuda")
        ok = i < n.view(-1, 1)
        page = s["fwd"].gather(1, (first.view(-1, 1) + i // slots).clamp(max=s["pmax"] - 1).long())
        page, slot = torch.where(ok, page, torch.zeros_like(page)).long(), (i % slots).expand_as(ok)
        m = meta[page, slot].float()
        kr = pages[:, :16 * kh * P].unflatten(1, (slots, 16 * kh // half))
        k = _codes(kr[page, slot], kh // half) * m[..., 0:1] + m[..., 1:2]
        v = None
        if need_v:
            vr = pages[:, 16 * kh * P:16 * (kh + vh) * P].unflatten(1, (slots, 16 * vh // half))
            v = _codes(vr[page, slot], vh // half) * m[..., 2:3] + m[..., 3:4]
            v = v * ok.unsqueeze(-1)
        return k * ok.unsqueeze(-1), v, posn[page, slot, 0], ok

    hdr = s["hdr"]
    a, b = part(P, 1, hdr[:, 0], hdr[:, 2] * 0), part(2 * P, 2, hdr[:, 1], hdr[:, 2])
    shape = (s["R"], s["Hkv"])
    return [None if x is None else torch.cat([x, y], 1).unflatten(0, shape) for x, y in zip(a, b)]


def _padded(s):
    """Where token i of request r lies among the packed tokens [R][max_new], and which exist."""
    i = torch.arange(s["max_new"], device="cuda")
    new = s["new"].long()
    ok = i < new.view(-1, 1)
    return ((new.cumsum(0) - new).view(-1, 1) + i).clamp(max=max(s["T"] - 1, 0)), ok


def _logits(s, k):
    """Logits [R][Hkv][i, g][held + new] of every new token, and which pairs exist."""
    at, ok = _padded(s)
    G, n = s["Hq"] // s["Hkv"], s["max_new"]
    q = s["q"][0, at].float().view(s["R"], n, s["Hkv"], G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    kn = s["kn"][0, at].float().permute(0, 2, 1, 3)
    x = (q * SCALE) @ torch.cat([k, kn], 2).transpose(2, 3)
    i = torch.arange(n, device="cuda")
    causal = (i.view(1, -1, 1) >= i.view(1, 1, -1)) & ok.view(s["R"], n, 1)
    return x, causal.repeat_interleave(G, 1).unsqueeze(1), at, ok


def _plain_attention(s):
    k, v, _, held = _held(s, True)
    x, causal, at, ok = _logits(s, k)
    n = held.shape[2]
    x[..., :n].masked_fill_(~held.unsqueeze(2), float("-inf"))
    x[..., n:].masked_fill_(~causal, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    vn = s["vn"][0, at].float().permute(0, 2, 1, 3)
    o = (x @ torch.cat([v, vn * ok.view(s["R"], 1, -1, 1)], 2)) / torch.where(z > 0, z, torch.ones_like(z))
    G = s["Hq"] // s["Hkv"]
    o = o.unflatten(2, (s["max_new"], G)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = (m + z.log()).squeeze(-1).unflatten(2, (s["max_new"], G)).permute(0, 2, 1, 3).flatten(2, 3)
    return o[ok].bfloat16().unsqueeze(0), lse[ok].unsqueeze(0)


def _plain_extend(s):
    out, lse = _plain_attention(s)
    return {"out": out, "lse": lse}


def _plain_significance(s):
    k, _, pos, held = _held(s, False)
    x, causal, at, ok = _logits(s, k)
    R, Hkv, n, G, N = s["R"], s["Hkv"], s["max_new"], s["Hq"] // s["Hkv"], held.shape[2]
    acc = torch.arange(n, device="cuda") < s["acc"].view(-1, 1)
    lse = s["lse"][0, at].view(R, n, Hkv, G).permute(0, 2, 1, 3).flatten(2, 3)
    x.sub_(lse.unsqueeze(-1)).exp_()
    x.mul_(acc.repeat_interleave(G, 1).view(R, 1, n * G, 1))
    x[..., N:].mul_(causal)
    p = x.unflatten(2, (n, G)).sum(2).permute(0, 3, 1, 2)  # [R][held + new][Hkv][G]
    sig = s["sig"].view(R, s["cap"], Hkv, G)
    r, h, t = held.nonzero(as_tuple=True)
    sig[r, pos[r, h, t].long(), h] += p[r, t, h]
    r, i = acc.nonzero(as_tuple=True)
    sig[r, s["ctx"].long()[r] + i] = p[r, N + i]
    return s["sig"]


def _units_of(s, who):
    """Units of the requests `who`, layer by layer in the order given."""
    l = torch.arange(s["L"], device="cuda").view(-1, 1, 1)
    return ((l * s["R"] + who.long().view(1, -1, 1)) * s["Hkv"] + torch.arange(s["Hkv"], device="cuda")).flatten()


def _runs(d):
    """For runs of lengths d: the run of each element, its index in the run and in all."""
    v = torch.repeat_interleave(torch.arange(d.numel(), device="cuda"), d)
    j = torch.arange(v.numel(), device="cuda")
    return v, j - (d.cumsum(0) - d)[v], j


def _plain_fork(s):
    su, du = _units_of(s, s["src"]), _units_of(s, s["dst"])
    hdr = s["hdr"][su]
    v, k, j = _runs((hdr[:, 2] + hdr[:, 3]).long())
    old = s["fwd"][su[v], k].long()
    new32 = s["free_list"][(s["cursors"][0] + j) % s["F"]]
    new = new32.long()
    s["pages"].view(torch.int64)[new] = s["pages"].view(torch.int64)[old]
    s["rev_unit"][new], s["rev_idx"][new] = du[v].to(torch.int32), k.to(torch.int32)
    s["page_cls"][new] = s["page_cls"][old]
    s["fwd"][du] = -1
    s["fwd"][du[v], k] = new32
    s["hdr"][du] = hdr
    s["cursors"][0] += v.numel()
    src, dst = s["src"].long(), s["dst"].long()
    held = torch.arange(s["cap"], device="cuda") < s["ctx"][src].view(-1, 1)
    for t in (s["classes"], s["slot_of"], s["sig"]):
        t[:, dst] = torch.where(held.view(1, -1, s["cap"], 1), t[:, src], t[:, dst])
    s["cnt"][dst] = torch.where(held, s["cnt"][src], s["cnt"][dst])
    return _forked(s)


def _plain_release(s):
    u = _units_of(s, s["src"])
    v, k, j = _runs((s["hdr"][u, 2] + s["hdr"][u, 3]).long())
    ids = s["fwd"][u[v], k]
    s["free_list"][(s["cursors"][1] + j) % s["F"]] = ids
    s["rev_unit"][ids.long()] = -1
    s["rev_idx"][ids.long()] = -1
    s["page_cls"][ids.long()] = 0
    s["fwd"][u] = -1
    s["hdr"][u] = 0
    s["cursors"][1] += v.numel()
    return _small(s)


def _plain_defrag(s):
    live = s["page_cls"] != 0
    n = int(live.sum())
    hole = (~live[:n]).nonzero()[:, 0]
    high = n + live[n:].nonzero()[:, 0]
    s["pages"].view(torch.int64)[hole] = s["pages"].view(torch.int64)[high]
    s["fwd"][s["rev_unit"][high].long(), s["rev_idx"][high].long()] = hole.to(torch.int32)
    for t, gone in ((s["rev_unit"], -1), (s["rev_idx"], -1), (s["page_cls"], 0)):
        t[hole] = t[high]
        t[high] = gone
    F = s["F"]
    s["free_list"][n:] = torch.arange(n, F, device="cuda", dtype=torch.int32)
    s["cursors"][0] += (n - s["cursors"][0]) % F
    s["cursors"][1] = s["cursors"][0] + (F - n)
    return dict(_small(s), pages=s["pages"].view(torch.int64))


_RUN = {"extend": _plain_extend, "significance": _plain_significance, "fork": _plain_fork, "release": _plain_release,
        "defrag": _plain_defrag}


# ------------------------------------------------------------------ 64 bits --

def _bits_row(page, at, slot, bits):
    """Codes of the rows (page, slot) of a region that starts at byte `at`, from their single bits."""
    b = page.gather(1, at + slot.view(-1, 1) * 16 * bits + torch.arange(16 * bits, device="cuda"))
    b = (b.unsqueeze(2) >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
    return (b.view(len(slot), D, bits).double() * (2.0 ** torch.arange(bits, device="cuda").double())).sum(2)


def _unit_rows(s, u):
    """fp64 K and V rows and the positions of one unit."""
    P = s["case"]["P"]
    kh, vh = WIDTHS[s["case"]["scheme"]]
    n_hi, n_lo, p_hi, _ = (int(x) for x in s["hdr"][u])
    ks, vs, ps = [], [], []
    for n, first, slots, half in ((n_hi, 0, P, 1), (n_lo, p_hi, 2 * P, 2)):
        if n == 0:
            continue
        i = torch.arange(n, device="cuda")
        page, slot = s["pages"][s["fwd"][u][first + i // slots].long()], i % slots
        base = 16 * (kh + vh) * P
        m = page.gather(1, base + slot.view(-1, 1) * 8 + torch.arange(8, device="cuda")).view(torch.float16).double()
        ks.append(_bits_row(page, 0, slot, kh // half) * m[:, 0:1] + m[:, 1:2])
        vs.append(_bits_row(page, 16 * kh * P, slot, vh // half) * m[:, 2:3] + m[:, 3:4])
        where = base + 16 * P + slot.view(-1, 1) * 4 + torch.arange(4, device="cuda")
        ps.append(page.gather(1, where).view(torch.int32)[:, 0].long())
    empty = torch.zeros((0, D), dtype=torch.float64, device="cuda")
    return (torch.cat(ks + [empty]), torch.cat(vs + [empty]),
            torch.cat(ps + [torch.zeros(0, dtype=torch.long, device="cuda")]))


def exact(case, seed):
    if case["op"] not in ("extend", "significance"):
        return None  # nothing is computed: whole numbers and copies
    s = _attention_inputs(dict(case), int(seed))
    Hq, Hkv, G = s["Hq"], s["Hkv"], s["Hq"] // s["Hkv"]
    out = torch.zeros((1, s["T"], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((1, s["T"], Hq), dtype=torch.float64, device="cuda")
    sig = s["sig"].double() if "sig" in s else None
    ctx, new, t0 = s["ctx"].tolist(), s["new"].tolist(), 0
    acc = s["acc"].tolist() if "acc" in s else None
    for r in range(s["R"]):
        n, t1 = new[r], t0 + new[r]
        if n == 0:
            continue
        later = torch.ones((n, n), device="cuda").triu(1).bool()
        for h in range(Hkv):
            k, v, pos = _unit_rows(s, r * Hkv + h)
            k = torch.cat([k, s["kn"][0, t0:t1, h].double()])
            v = torch.cat([v, s["vn"][0, t0:t1, h].double()])
            for g in range(G):
                x = s["q"][0, t0:t1, h * G + g].double() @ k.T * SCALE
                x[:, len(pos):].masked_fill_(later, float("-inf"))
                if sig is None:
                    e = torch.logsumexp(x, 1)
                    lse[0, t0:t1, h * G + g] = e
                    out[0, t0:t1, h * G + g] = torch.exp(x - e.view(-1, 1)) @ v
                else:
                    a = acc[r]
                    p = torch.exp(x[:a] - s["lse"][0, t0:t0 + a, h * G + g].double().view(-1, 1)).sum(0)
                    rows = sig[0, r * s["cap"]:(r + 1) * s["cap"], h * G + g]
                    rows[pos] += p[:len(pos)]
                    rows[ctx[r]:ctx[r] + a] = p[len(pos):len(pos) + a]
        t0 = t1
    return {"out": out, "lse": lse} if sig is None else sig
