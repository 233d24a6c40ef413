"""Test-side restatement of the page operations (fork, release, defrag): one
page after the other over numpy copies of a pool's state.  `st` has free_list,
cursors, rev_unit, rev_idx, page_cls, pages, fwd, unit_hdr."""
from __future__ import annotations

import numpy as np


def list_units(L, R, Hkv, reqs):
    return [(l * R + int(r)) * Hkv + h for l in range(L) for r in reqs for h in range(Hkv)]


def copy_state(st: dict) -> dict:
    return {k: v.copy() for k, v in st.items()}


def serial_fork(st: dict, L, R, Hkv, src, dst, unit_base=0) -> dict:
    st = copy_state(st)
    F = st["free_list"].size
    head = int(st["cursors"][0])
    for u, w in zip(list_units(L, R, Hkv, src), list_units(L, R, Hkv, dst)):
        p_hi, p_lo = int(st["unit_hdr"][u][2]), int(st["unit_hdr"][u][3])
        st["fwd"][w] = -1
        for j in range(p_hi + p_lo):
            new, old = int(st["free_list"][head % F]), int(st["fwd"][u][j])
            head += 1
            st["fwd"][w][j] = new
            st["pages"][new] = st["pages"][old]
            st["page_cls"][new] = st["page_cls"][old]
            st["rev_unit"][new], st["rev_idx"][new] = unit_base + w, j
        st["unit_hdr"][w] = st["unit_hdr"][u]
    st["cursors"][0] = head
    return st


def serial_release(st: dict, L, R, Hkv, reqs) -> dict:
    st = copy_state(st)
    F = st["free_list"].size
    tail = int(st["cursors"][1])
    for u in list_units(L, R, Hkv, reqs):
        for j in range(int(st["unit_hdr"][u][2]) + int(st["unit_hdr"][u][3])):
            p = int(st["fwd"][u][j])
            st["free_list"][tail % F] = p
            tail += 1
            st["rev_unit"][p] = st["rev_idx"][p] = -1
            st["page_cls"][p] = 0
        st["fwd"][u] = -1
        st["unit_hdr"][u] = 0
    st["cursors"][1] = tail
    return st


def serial_defrag(st: dict, unit_base=0) -> dict:
    st = copy_state(st)
    F = st["free_list"].size
    head, tail = int(st["cursors"][0]), int(st["cursors"][1])
    n = F - (tail - head)
    holes = [p for p in range(n) if st["page_cls"][p] == 0]
    movers = [p for p in range(n, F) if st["page_cls"][p] != 0]
    assert len(holes) == len(movers)
    for to, p in zip(holes, movers):
        st["pages"][to] = st["pages"][p]
        for k in ("rev_unit", "rev_idx", "page_cls"):
            st[k][to] = st[k][p]
        st["rev_unit"][p] = st["rev_idx"][p] = -1
        st["page_cls"][p] = 0
        st["fwd"][int(st["rev_unit"][to]) - unit_base][int(st["rev_idx"][to])] = to
    while head % F != n % F:
        head += 1
    st["cursors"][0], st["cursors"][1] = head, head + F - n
    st["free_list"][n:] = np.arange(n, F)
    return st


def pool_state(pool, tables) -> dict:
    """numpy copies of a device pool's and its tables' state."""
    return {"free_list": pool.free_list.cpu().numpy(), "cursors": pool.cursors.cpu().numpy().astype(np.int64),
            "rev_unit": pool.rev_unit.cpu().numpy(), "rev_idx": pool.rev_idx.cpu().numpy(),
            "page_cls": pool.page_cls.cpu().numpy(), "pages": pool.pages.cpu().numpy(),
            "fwd": tables.fwd.cpu().numpy(), "unit_hdr": tables.unit_hdr.cpu().numpy()}


def assert_equal(got: dict, want: dict, what: str, ring_only: bool = True):
    """Everything equal: the free list over its live slots, pages where owned."""
    for k in ("cursors", "rev_unit", "rev_idx", "page_cls", "fwd", "unit_hdr"):
        assert np.array_equal(got[k], want[k]), f"{what}: {k}"
    F = want["free_list"].size
    ring = np.arange(int(want["cursors"][0]), int(want["cursors"][1])) % F
    assert np.array_equal(got["free_list"][ring], want["free_list"][ring]), f"{what}: free list"
    live = np.nonzero(want["page_cls"])[0]
    assert np.array_equal(got["pages"][live], want["pages"][live]), f"{what}: pages"


def assert_untouched(got: dict, before: dict, what: str):
    for k in before:
        assert np.array_equal(got[k], before[k]), f"{what}: {k} changed"
