"""Thin ctypes binding over libdkv.so (argument marshalling only).

Every function here forwards to the C entry point of the same name declared
in ``include/dkv.h``; all compute runs in the library's CUDA kernels.  PyTorch
only provides device memory and the current stream.  There is no fallback:
if ``libdkv.so`` has not been built, loading raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# DKV_LIBRARY=checked selects the bounds-checked build (lib/libdkv_checked.so),
# DKV_LIBRARY=sanitized the one with sanitized host code (lib/libdkv_san.so)
LIB_PATH = os.path.join(HERE, "lib", {"checked": "libdkv_checked.so", "sanitized": "libdkv_san.so"}.get(
    os.environ.get("DKV_LIBRARY", ""), "libdkv.so"))

DKV_OK = 0
DKV_E_INVAL = -1
DKV_E_NOMEM = -2
DKV_E_RANGE = -3
DKV_E_TIMEOUT = -4
DKV_E_INTERNAL = -5
DKV_E_CUDA = -6
DKV_E_LENS = -7
DKV_PROFILE_KERNELS = 5
KERNEL_NAMES = ("k_prep", "k_classify", "k_scan", "k_pack", "k_commit")

_lib = None


class DkvError(RuntimeError):
    def __init__(self, code: int, what: str):
        detail = f" [{load().dkv_last_cuda_error().decode()}]" if code == DKV_E_CUDA else ""
        super().__init__(f"{what}: {status_string(code)} ({code}){detail}")
        self.code = code


class dkv_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32), ("max_len", ctypes.c_int32), ("T", ctypes.c_int64),
        ("unit_base", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("sig_sum", ctypes.c_void_p), ("sig_cnt", ctypes.c_void_p), ("lens", ctypes.c_void_p),
        ("classes", ctypes.c_void_p),
    ]


class dkv_params(ctypes.Structure):
    _fields_ = [("alpha_h", ctypes.c_float), ("alpha_l", ctypes.c_float), ("spin_limit", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("profiler", ctypes.c_void_p)]


class dkv_pool(ctypes.Structure):
    _fields_ = [
        ("F", ctypes.c_int64), ("P", ctypes.c_int32), ("scheme", ctypes.c_int32),
        ("free_list", ctypes.c_void_p), ("cursors", ctypes.c_void_p), ("rev_unit", ctypes.c_void_p),
        ("rev_idx", ctypes.c_void_p), ("page_cls", ctypes.c_void_p), ("pages", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


class dkv_tables(ctypes.Structure):
    _fields_ = [("fwd", ctypes.c_void_p), ("pmax", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("unit_hdr", ctypes.c_void_p)]


class dkv_decode_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32), ("cap", ctypes.c_int32), ("unit_base", ctypes.c_int64),
        ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("sig_sum", ctypes.c_void_p),
        ("sig_cnt", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
        ("classes", ctypes.c_void_p), ("slot_of", ctypes.c_void_p), ("window", ctypes.c_int32),
        ("mode", ctypes.c_int32),
    ]


class dkv_attn_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("layer0", ctypes.c_int32), ("n_layers", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p), ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("sig_sum", ctypes.c_void_p),
    ]


class dkv_prefill_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("max_len", ctypes.c_int32), ("reserved", ctypes.c_int32), ("T", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("lens", ctypes.c_void_p),
        ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("sig_sum", ctypes.c_void_p),
        ("sig_cnt", ctypes.c_void_p),
    ]


class dkv_extend_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("layer0", ctypes.c_int32), ("n_layers", ctypes.c_int32),
        ("max_new", ctypes.c_int32), ("T", ctypes.c_int64), ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p),
        ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


class dkv_fork_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("n", ctypes.c_int32), ("unit_base", ctypes.c_int64), ("src", ctypes.c_void_p),
        ("dst", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p), ("classes", ctypes.c_void_p),
        ("slot_of", ctypes.c_void_p), ("sig_sum", ctypes.c_void_p), ("sig_cnt", ctypes.c_void_p),
    ]


class dkv_release_batch(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("n", ctypes.c_int32),
                ("unit_base", ctypes.c_int64), ("reqs", ctypes.c_void_p)]


class dkv_chunk_pages(ctypes.Structure):
    _fields_ = [("F", ctypes.c_int64), ("B", ctypes.c_int32), ("tmax", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("table", ctypes.c_void_p)]


class dkv_chunk_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("layer0", ctypes.c_int32), ("n_layers", ctypes.c_int32),
        ("max_new", ctypes.c_int32), ("T", ctypes.c_int64), ("q_stride", ctypes.c_int64),
        ("kv_stride", ctypes.c_int64), ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p),
        ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


class dkv_evict_batch(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("R", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("sinks", ctypes.c_int32), ("window", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("unit_base", ctypes.c_int64), ("budgets", ctypes.c_void_p), ("ctx_lens", ctypes.c_void_p),
        ("sig_sum", ctypes.c_void_p), ("sig_cnt", ctypes.c_void_p), ("classes", ctypes.c_void_p),
        ("slot_of", ctypes.c_void_p),
    ]


def load():
    """Load libdkv.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sigs = {
        "dkv_version": ([], i32),
        "dkv_build_flags": ([], i32),
        "dkv_status_string": ([i32], ctypes.c_char_p),
        "dkv_last_cuda_error": ([], ctypes.c_char_p),
        "dkv_page_bytes": ([i32, i32, P(ctypes.c_int64)], i32),
        "dkv_workspace_size": ([P(dkv_batch), P(ctypes.c_size_t)], i32),
        "dkv_init_pool": ([P(dkv_pool), vp], i32),
        "dkv_compact": ([P(dkv_batch), P(dkv_params), P(dkv_pool), P(dkv_tables), vp, ctypes.c_size_t, vp], i32),
        "dkv_compact_noalloc": ([P(dkv_batch), P(dkv_params), P(dkv_pool), P(dkv_tables), vp], i32),
        "dkv_dequant_page": ([P(dkv_pool), i32, vp, vp, vp, vp], i32),
        "dkv_dequant_pages": ([P(dkv_pool), vp, i32, vp, vp, vp, vp], i32),
        "dkv_get_status": ([P(dkv_pool), vp], i32),
        "dkv_decode_workspace_size": ([P(dkv_decode_batch), P(ctypes.c_size_t)], i32),
        "dkv_decode_index": ([P(dkv_decode_batch), P(dkv_pool), P(dkv_tables), vp], i32),
        "dkv_decode_step": ([P(dkv_decode_batch), P(dkv_params), P(dkv_pool), P(dkv_tables), vp, ctypes.c_size_t,
                             vp], i32),
        "dkv_decode_attention": ([P(dkv_attn_batch), P(dkv_pool), P(dkv_tables), vp], i32),
        "dkv_prefill_attention": ([P(dkv_prefill_batch), P(dkv_pool), vp], i32),
        "dkv_extend_workspace_size": ([P(dkv_extend_batch), P(dkv_pool), P(dkv_tables), P(ctypes.c_size_t)], i32),
        "dkv_extend_attention": ([P(dkv_extend_batch), P(dkv_pool), P(dkv_tables), vp, ctypes.c_size_t, vp], i32),
        "dkv_extend_significance": ([P(dkv_extend_batch), vp, vp, P(dkv_pool), P(dkv_tables), vp], i32),
        "dkv_chunk_workspace_size": ([P(dkv_chunk_batch), P(dkv_chunk_pages), P(ctypes.c_size_t)], i32),
        "dkv_chunk_attention": ([P(dkv_chunk_batch), P(dkv_chunk_pages), P(dkv_pool), vp, ctypes.c_size_t, vp], i32),
        "dkv_chunk_significance": ([P(dkv_chunk_batch), P(dkv_chunk_pages), vp, P(dkv_pool), vp], i32),
        "dkv_evict_workspace_size": ([P(dkv_evict_batch), P(dkv_pool), P(dkv_tables), P(ctypes.c_size_t)], i32),
        "dkv_evict": ([P(dkv_evict_batch), P(dkv_pool), P(dkv_tables), vp, ctypes.c_size_t, vp], i32),
        "dkv_page_ops_workspace_size": ([P(dkv_pool), i64, P(ctypes.c_size_t)], i32),
        "dkv_fork": ([P(dkv_fork_batch), P(dkv_pool), P(dkv_tables), vp, ctypes.c_size_t, vp], i32),
        "dkv_release": ([P(dkv_release_batch), P(dkv_pool), P(dkv_tables), vp, ctypes.c_size_t, vp], i32),
        "dkv_defrag": ([P(dkv_pool), P(dkv_tables), i64, i64, vp, ctypes.c_size_t, vp], i32),
        "dkv_profiler_create": ([i32, P(vp)], i32),
        "dkv_profiler_read": ([vp, vp, i32], i32),
        "dkv_profiler_destroy": ([vp], i32),
    }
    for name, (args, res) in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def status_string(code: int) -> str:
    return load().dkv_status_string(int(code)).decode()


DKV_SCHEME_K8V4_K4V2 = 0
DKV_SCHEME_K8V2_K4V1 = 1
DKV_SCHEME_K4V8_K2V4 = 2


def dkv_page_bytes(scheme: int, P: int) -> int:
    n = ctypes.c_int64(0)
    rc = load().dkv_page_bytes(int(scheme), int(P), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_page_bytes")
    return int(n.value)


def _stream(stream=None) -> int:
    if stream is None:  # the handle alone: the Stream object costs 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _on_stream(stream, device):
    """Within it torch allocates and works on the stream of the call (None: the current one)."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):  # another library's
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return torch.cuda.stream(stream)


def _p(t) -> int | None:
    return None if t is None else t.data_ptr()


def _holding(batch, *tensors):
    """The batch with references to the tensors whose addresses it has: their memory is theirs as long as it lives."""
    batch.tensors = tensors
    return batch


class DevicePool:
    """Pool state in device memory (torch tensors owned by this object)."""

    def __init__(self, F: int, P: int, device="cuda", scheme: int = 0):
        self.F, self.P, self.scheme = int(F), int(P), int(scheme)
        d = torch.device(device)
        self.free_list = torch.empty(self.F, dtype=torch.int32, device=d)
        self.cursors = torch.zeros(2, dtype=torch.int64, device=d)   # uint64 bit patterns
        self.rev_unit = torch.empty(self.F, dtype=torch.int32, device=d)
        self.rev_idx = torch.empty(self.F, dtype=torch.int32, device=d)
        self.page_cls = torch.empty(self.F, dtype=torch.uint8, device=d)
        self.pages = torch.empty((self.F, dkv_page_bytes(self.scheme, self.P)), dtype=torch.uint8, device=d)
        self.status = torch.zeros(1, dtype=torch.int32, device=d)

    @classmethod
    def from_tensors(cls, P: int, scheme: int, free_list, cursors, rev_unit, rev_idx, page_cls, pages,
                     status) -> "DevicePool":
        """A pool over device tensors that the caller allocated and keeps in a
        valid state (F is the length of free_list)."""
        self = cls.__new__(cls)
        self.F, self.P, self.scheme = int(free_list.numel()), int(P), int(scheme)
        self.free_list, self.cursors, self.rev_unit, self.rev_idx = free_list, cursors, rev_unit, rev_idx
        self.page_cls, self.pages, self.status = page_cls, pages, status
        for name, dtype, n in (("free_list", torch.int32, self.F), ("cursors", torch.int64, 2),
                               ("rev_unit", torch.int32, self.F), ("rev_idx", torch.int32, self.F),
                               ("page_cls", torch.uint8, self.F),
                               ("pages", torch.uint8, self.F * dkv_page_bytes(self.scheme, self.P)),
                               ("status", torch.int32, 1)):
            t = getattr(self, name)
            if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous {dtype} tensor of {n} elements is wanted")
        return self

    def c(self) -> dkv_pool:
        return dkv_pool(self.F, self.P, self.scheme, _p(self.free_list), _p(self.cursors), _p(self.rev_unit),
                        _p(self.rev_idx), _p(self.page_cls), _p(self.pages), _p(self.status))


class DeviceTables:
    def __init__(self, U: int, pmax: int, device="cuda"):
        self.pmax = int(pmax)
        self.fwd = torch.empty((U, self.pmax), dtype=torch.int32, device=device)
        self.unit_hdr = torch.empty((U, 4), dtype=torch.int32, device=device)

    @classmethod
    def from_tensors(cls, fwd: torch.Tensor, unit_hdr: torch.Tensor) -> "DeviceTables":
        """Tables over the caller's int32 tensors fwd [U][pmax] and unit_hdr [U][4]."""
        if fwd.dtype != torch.int32 or unit_hdr.dtype != torch.int32 or fwd.dim() != 2 or \
                tuple(unit_hdr.shape) != (fwd.shape[0], 4) or not (fwd.is_contiguous() and unit_hdr.is_contiguous()):
            raise ValueError("fwd [U][pmax] and unit_hdr [U][4]: contiguous int32 tensors are wanted")
        self = cls.__new__(cls)
        self.pmax, self.fwd, self.unit_hdr = int(fwd.shape[1]), fwd, unit_hdr
        return self

    def units(self) -> int:
        return int(self.fwd.shape[0])

    def c(self) -> dkv_tables:
        return dkv_tables(_p(self.fwd), self.pmax, 0, _p(self.unit_hdr))


def make_batch(inp: dict, classes: torch.Tensor, max_len: int, unit_base: int = 0) -> dkv_batch:
    at = (inp["k"], inp["v"], inp["sig_sum"], inp["sig_cnt"], inp["lens"], classes)
    return _holding(dkv_batch(int(inp["L"]), int(inp["R"]), int(inp["Hq"]), int(inp["Hkv"]), 128, int(max_len),
                              int(inp["T"]), int(unit_base), *map(_p, at)), *at)


def dkv_workspace_size(batch: dkv_batch) -> int:
    n = ctypes.c_size_t(0)
    rc = load().dkv_workspace_size(ctypes.byref(batch), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_workspace_size")
    return int(n.value)


def dkv_init_pool(pool: DevicePool, stream=None) -> None:
    c = pool.c()
    rc = load().dkv_init_pool(ctypes.byref(c), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_init_pool")


def dkv_compact(batch: dkv_batch, alpha_h: float, alpha_l: float, pool: DevicePool, tables: DeviceTables,
                workspace: torch.Tensor, stream=None, spin_limit: int = -1, profiler=None) -> None:
    """Enqueue one compaction; device-side errors are read with dkv_get_status."""
    params = dkv_params(float(alpha_h), float(alpha_l), int(spin_limit), 0,
                        None if profiler is None else profiler.handle)
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_compact(ctypes.byref(batch), ctypes.byref(params), ctypes.byref(pc), ctypes.byref(tc),
                            _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_compact")


def dkv_compact_noalloc(batch: dkv_batch, alpha_h: float, alpha_l: float, pool: DevicePool,
                        tables: DeviceTables, stream=None, spin_limit: int = -1) -> None:
    """dkv_compact with the library's built-in scratch instead of a workspace."""
    params = dkv_params(float(alpha_h), float(alpha_l), int(spin_limit), 0, None)
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_compact_noalloc(ctypes.byref(batch), ctypes.byref(params), ctypes.byref(pc), ctypes.byref(tc),
                                    _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_compact_noalloc")


def dkv_get_status(pool: DevicePool, stream=None) -> int:
    c = pool.c()
    return int(load().dkv_get_status(ctypes.byref(c), _stream(stream)))


def dkv_dequant_page(pool: DevicePool, page_id: int, stream=None):
    P = pool.P
    dev = pool.pages.device
    with _on_stream(stream, dev):
        k = torch.empty((2 * P, 128), dtype=torch.float32, device=dev)
        v = torch.empty((2 * P, 128), dtype=torch.float32, device=dev)
        pos = torch.empty(2 * P, dtype=torch.int32, device=dev)
    c = pool.c()
    rc = load().dkv_dequant_page(ctypes.byref(c), int(page_id), _p(k), _p(v), _p(pos), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_dequant_page")
    return k, v, pos


def dkv_dequant_pages(pool: DevicePool, page_ids: torch.Tensor, stream=None):
    P = pool.P
    n = int(page_ids.numel())
    dev = pool.pages.device
    with _on_stream(stream, dev):
        ids = page_ids.to(device=dev, dtype=torch.int32).contiguous()
        k = torch.empty((n, 2 * P, 128), dtype=torch.float32, device=dev)
        v = torch.empty((n, 2 * P, 128), dtype=torch.float32, device=dev)
        pos = torch.empty((n, 2 * P), dtype=torch.int32, device=dev)
    c = pool.c()
    rc = load().dkv_dequant_pages(ctypes.byref(c), _p(ids), n, _p(k), _p(v), _p(pos), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_dequant_pages")
    return k, v, pos


class Profiler:
    """Per-kernel CUDA-event timing of dkv_compact calls (library-owned events)."""

    def __init__(self, max_calls: int):
        h = ctypes.c_void_p()
        rc = load().dkv_profiler_create(int(max_calls), ctypes.byref(h))
        if rc != DKV_OK:
            raise DkvError(rc, "dkv_profiler_create")
        self.handle = h.value
        self.max_calls = int(max_calls)

    def read(self):
        """[(ms per kernel) for each recorded call], then starts a new recording."""
        buf = (ctypes.c_float * (self.max_calls * DKV_PROFILE_KERNELS))()
        n = load().dkv_profiler_read(self.handle, buf, self.max_calls)
        if n < 0:
            raise DkvError(n, "dkv_profiler_read")
        return [list(buf[c * DKV_PROFILE_KERNELS:(c + 1) * DKV_PROFILE_KERNELS]) for c in range(n)]

    def close(self):
        if self.handle:
            load().dkv_profiler_destroy(self.handle)
            self.handle = None


class Compactor:
    """Convenience owner of pool, tables, classes and workspace for one shape."""

    def __init__(self, L: int, R: int, Hq: int, Hkv: int, T: int, max_len: int, P: int, F: int, device="cuda",
                 scheme: int = 0):
        self.L, self.R, self.Hq, self.Hkv, self.T, self.max_len = L, R, Hq, Hkv, T, max_len
        self.U = L * R * Hkv
        self.pmax = -(-max_len // P) + 1
        self.pool = DevicePool(F, P, device, scheme=scheme)
        self.tables = DeviceTables(self.U, self.pmax, device)
        self.classes = torch.empty(max(L * T * Hkv, 1), dtype=torch.uint8, device=device)
        probe = dkv_batch(L, R, Hq, Hkv, 128, max_len, T, 0, None, None, None, None, None, None)
        self.workspace = torch.empty(dkv_workspace_size(probe), dtype=torch.uint8, device=device)
        dkv_init_pool(self.pool)

    def batch(self, inp: dict, unit_base: int = 0) -> dkv_batch:
        return make_batch(inp, self.classes, self.max_len, unit_base)

    def compact(self, inp: dict, alpha_h: float, alpha_l: float, stream=None, spin_limit: int = -1,
                profiler=None, unit_base: int = 0) -> None:
        dkv_compact(self.batch(inp, unit_base), alpha_h, alpha_l, self.pool, self.tables, self.workspace,
                    stream=stream, spin_limit=spin_limit, profiler=profiler)


# ------------------------------------------------------------------ decode --

def dkv_decode_workspace_size(batch: dkv_decode_batch) -> int:
    n = ctypes.c_size_t(0)
    rc = load().dkv_decode_workspace_size(ctypes.byref(batch), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_decode_workspace_size")
    return int(n.value)


def dkv_decode_index(batch: dkv_decode_batch, pool: DevicePool, tables, stream=None) -> None:
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_decode_index(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_decode_index")


def dkv_decode_step(batch: dkv_decode_batch, alpha_h: float, alpha_l: float, pool: DevicePool, tables,
                    workspace: torch.Tensor, stream=None, spin_limit: int = -1, profiler=None) -> None:
    params = dkv_params(float(alpha_h), float(alpha_l), int(spin_limit), 0,
                        None if profiler is None else profiler.handle)
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_decode_step(ctypes.byref(batch), ctypes.byref(params), ctypes.byref(pc), ctypes.byref(tc),
                                _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_decode_step")


def dkv_decode_attention(batch: dkv_attn_batch, pool: DevicePool, tables, stream=None) -> None:
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_decode_attention(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_decode_attention")


def dkv_prefill_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lens: torch.Tensor, max_len: int,
                          scale: float, out: torch.Tensor, sig_sum: torch.Tensor, sig_cnt: torch.Tensor,
                          pool: DevicePool, stream=None) -> None:
    """dkv_prefill_attention: q [L][T][Hq][128], k / v [L][T][Hkv][128] bf16;
    out fp32 [L][T][Hq][128], sig_sum fp32 [L][T][Hq], sig_cnt int32 [T]."""
    L, T, Hq = int(q.shape[0]), int(q.shape[1]), int(q.shape[2])
    b = dkv_prefill_batch(L, int(lens.numel()), Hq, int(k.shape[2]), int(max_len), 0, T, _p(q), _p(k), _p(v),
                          _p(lens), float(scale), _p(out), _p(sig_sum), _p(sig_cnt))
    pc = pool.c()
    rc = load().dkv_prefill_attention(ctypes.byref(b), ctypes.byref(pc), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_prefill_attention")


# ------------------------------------- several tokens a request, page operations --

def make_extend_batch(L: int, Hkv: int, cap: int, q: torch.Tensor, new_lens: torch.Tensor, ctx_lens: torch.Tensor,
                      max_new: int, scale: float, k_new: torch.Tensor | None = None,
                      v_new: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, layer0: int = 0) -> dkv_extend_batch:
    """q, out bf16 [n_layers][T][Hq][128]; k_new, v_new bf16 [n_layers][T][Hkv][128]; lse fp32 [n_layers][T][Hq];
    new_lens, ctx_lens int32 [R]: of every request of the tables."""
    if ctx_lens.numel() != new_lens.numel():
        raise ValueError("new_lens and ctx_lens name the same requests")
    n_layers, T, Hq = int(q.shape[0]), int(q.shape[1]), int(q.shape[2])
    return _holding(dkv_extend_batch(int(L), int(new_lens.numel()), Hq, int(Hkv), int(cap), int(layer0), n_layers,
                                     int(max_new), T, _p(q), _p(k_new), _p(v_new), _p(new_lens), _p(ctx_lens),
                                     float(scale), _p(out), _p(lse)),
                    q, k_new, v_new, new_lens, ctx_lens, out, lse)


def dkv_extend_workspace_size(batch: dkv_extend_batch, pool: DevicePool, tables) -> int:
    n = ctypes.c_size_t(0)
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_extend_workspace_size(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_extend_workspace_size")
    return int(n.value)


def _workspace(w: torch.Tensor | None):
    return (None, 0) if w is None or w.numel() == 0 else (_p(w), w.numel() * w.element_size())


def dkv_extend_attention(batch: dkv_extend_batch, pool: DevicePool, tables, workspace: torch.Tensor | None,
                         stream=None) -> None:
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_extend_attention(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), *_workspace(workspace),
                                     _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_extend_attention")


def dkv_extend_significance(batch: dkv_extend_batch, acc_lens: torch.Tensor, sig_sum: torch.Tensor,
                            pool: DevicePool, tables, stream=None) -> None:
    if acc_lens.numel() != batch.R:
        raise ValueError("acc_lens and new_lens name the same requests")
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_extend_significance(ctypes.byref(batch), _p(acc_lens), _p(sig_sum), ctypes.byref(pc),
                                        ctypes.byref(tc), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_extend_significance")


def dkv_page_ops_workspace_size(pool: DevicePool, tables) -> int:
    n = ctypes.c_size_t(0)
    pc = pool.c()
    rc = load().dkv_page_ops_workspace_size(ctypes.byref(pc), int(tables.fwd.shape[0]), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_page_ops_workspace_size")
    return int(n.value)


def make_fork_batch(L: int, R: int, Hq: int, Hkv: int, cap: int, src: torch.Tensor, dst: torch.Tensor,
                    ctx_lens: torch.Tensor | None = None, classes: torch.Tensor | None = None,
                    slot_of: torch.Tensor | None = None, sig_sum: torch.Tensor | None = None,
                    sig_cnt: torch.Tensor | None = None, unit_base: int = 0) -> dkv_fork_batch:
    if src.numel() != dst.numel():
        raise ValueError("src and dst name the same number of requests")
    at = (src, dst, ctx_lens, classes, slot_of, sig_sum, sig_cnt)
    return _holding(dkv_fork_batch(int(L), int(R), int(Hq), int(Hkv), int(cap), int(src.numel()), int(unit_base),
                                   *map(_p, at)), *at)


def make_release_batch(L: int, R: int, Hkv: int, reqs: torch.Tensor, unit_base: int = 0) -> dkv_release_batch:
    return _holding(dkv_release_batch(int(L), int(R), int(Hkv), int(reqs.numel()), int(unit_base), _p(reqs)), reqs)


def dkv_fork(batch: dkv_fork_batch, pool: DevicePool, tables, workspace: torch.Tensor, stream=None) -> None:
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_fork(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), *_workspace(workspace),
                         _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_fork")


def dkv_release(batch: dkv_release_batch, pool: DevicePool, tables, workspace: torch.Tensor, stream=None) -> None:
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_release(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), *_workspace(workspace),
                            _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_release")


def dkv_defrag(pool: DevicePool, tables, workspace: torch.Tensor, unit_base: int = 0, stream=None) -> None:
    """Pack the pool; `tables` hold every unit that owns pages of it."""
    pc, tc = pool.c(), tables.c()
    rc = load().dkv_defrag(ctypes.byref(pc), ctypes.byref(tc), int(tables.fwd.shape[0]), int(unit_base),
                           *_workspace(workspace), _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_defrag")


# ------------------------------------------------- prompts in chunks, eviction --

def _want(t: torch.Tensor | None, name: str, dtype: torch.dtype, shape: tuple, like: torch.Tensor,
          contiguous: bool = True) -> None:
    """A tensor of this type and shape (a single number: so many elements) on the device of `like`."""
    if t is None:
        return
    fits = t.numel() == shape[0] if len(shape) == 1 else tuple(t.shape) == shape
    if t.dtype != dtype or not fits or t.device != like.device or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name}: a {'contiguous ' if contiguous else ''}{dtype} tensor of {list(shape)} on "
                         f"{like.device} is wanted")


def _on_device_of(batch, *others) -> None:
    """The batch's tensors (where it was made from tensors, which lie on one device then) are on the device of these."""
    at = others[0].device
    for t in (*getattr(batch, "tensors", ())[:1], *others[1:]):
        if t is not None and t.device != at:
            raise ValueError(f"tensors of one device are wanted, not of {at} and {t.device}")


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements from one token's rows [H][128] to the next of a view [n_layers][T][H][128]."""
    n, T, H = int(t.shape[0]), int(t.shape[1]), int(t.shape[2])
    s0, s1, s2, s3 = t.stride()
    s = s1 if T > 1 else (s0 if n > 1 else H * 128)  # a stride over one element says nothing
    if t.numel() and (s3 != 1 or (H > 1 and s2 != 128) or (n > 1 and s0 != T * s) or s < H * 128):
        raise ValueError(f"{name}: tokens may stand apart, their {H} rows of 128 and the layers may not")
    return int(s)


class ChunkPages:
    """bf16 pages [L][F][B][Hkv][128] of K and of V and the table [R][tmax] of the requests' pages (torch tensors
    owned by this object): what the chunks of a prompt have left until its compaction."""

    def __init__(self, L: int, R: int, Hkv: int, cap: int, B: int, F: int, device="cuda"):
        self.k = torch.zeros((L, F, B, Hkv, 128), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.table = torch.full((R, -(-cap // B)), -1, dtype=torch.int32, device=device)

    @classmethod
    def from_tensors(cls, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor) -> "ChunkPages":
        """Pages over the caller's bf16 tensors k, v [L][F][B][Hkv][128] and int32 table [R][tmax]."""
        if k.dim() != 5 or k.shape[4] != 128 or table.dim() != 2:
            raise ValueError("k and v [L][F][B][Hkv][128], table [R][tmax] are wanted")
        _want(k, "k", torch.bfloat16, tuple(k.shape), k)
        _want(v, "v", torch.bfloat16, tuple(k.shape), k)
        _want(table, "table", torch.int32, tuple(table.shape), k)
        self = cls.__new__(cls)
        self.k, self.v, self.table = k, v, table
        return self

    def c(self) -> dkv_chunk_pages:
        return dkv_chunk_pages(int(self.k.shape[1]), int(self.k.shape[2]), int(self.table.shape[1]), _p(self.k),
                               _p(self.v), _p(self.table))


def make_chunk_batch(Hkv: int, cap: int, q: torch.Tensor, new_lens: torch.Tensor, ctx_lens: torch.Tensor,
                     max_new: int, scale: float, k_new: torch.Tensor | None = None,
                     v_new: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, layer0: int = 0, L: int | None = None) -> dkv_chunk_batch:
    """q bf16 [n_layers][T][Hq][128]; k_new, v_new bf16 [n_layers][T][Hkv][128] (views of one projection's output are
    fine: rows of a token together, tokens at equal distances); out as q, contiguous; lse fp32 [n_layers][T][Hq];
    new_lens, ctx_lens int32 [R].  L: layers of the pages (layer0 + n_layers where not given)."""
    if q.dim() != 4 or q.shape[3] != 128:
        raise ValueError("q [n_layers][T][Hq][128] is wanted")
    n_layers, T, Hq = int(q.shape[0]), int(q.shape[1]), int(q.shape[2])
    R = int(new_lens.numel())
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new come together")
    _want(q, "q", torch.bfloat16, tuple(q.shape), q, contiguous=False)
    _want(k_new, "k_new", torch.bfloat16, (n_layers, T, int(Hkv), 128), q, contiguous=False)
    _want(v_new, "v_new", torch.bfloat16, (n_layers, T, int(Hkv), 128), q, contiguous=False)
    _want(out, "out", torch.bfloat16, tuple(q.shape), q)
    _want(lse, "lse", torch.float32, (n_layers, T, Hq), q)
    _want(new_lens, "new_lens", torch.int32, (R,), q)
    _want(ctx_lens, "ctx_lens", torch.int32, (R,), q)
    kv_stride = 0 if k_new is None else _token_stride(k_new, "k_new")
    if v_new is not None and _token_stride(v_new, "v_new") != kv_stride:
        raise ValueError("k_new and v_new: tokens at the same distances are wanted")
    return _holding(dkv_chunk_batch(int(L if L is not None else layer0 + n_layers), R, Hq, int(Hkv), int(cap),
                                    int(layer0), n_layers, int(max_new), T, _token_stride(q, "q"), kv_stride, _p(q),
                                    _p(k_new), _p(v_new), _p(new_lens), _p(ctx_lens), float(scale), _p(out), _p(lse)),
                    q, k_new, v_new, new_lens, ctx_lens, out, lse)


def _chunk_pages(batch: dkv_chunk_batch, pages: ChunkPages) -> dkv_chunk_pages:
    if pages.k.shape[0] != batch.L or pages.k.shape[3] != batch.Hkv or pages.table.shape[0] != batch.R:
        raise ValueError(f"pages of {batch.L} layers and {batch.Hkv} KV heads and a table of {batch.R} requests are "
                         f"wanted, not {pages.k.shape[0]}, {pages.k.shape[3]} and {pages.table.shape[0]}")
    return pages.c()


def _evict_tables(batch: dkv_evict_batch, tables) -> dkv_tables:
    units, there = batch.L * batch.R * batch.Hkv, tables.units()
    if there < units:
        raise ValueError(f"tables of {units} units are wanted, not of {there}")
    return tables.c()


def dkv_chunk_workspace_size(batch: dkv_chunk_batch, pages: ChunkPages) -> int:
    n = ctypes.c_size_t(0)
    pc = _chunk_pages(batch, pages)
    rc = load().dkv_chunk_workspace_size(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_chunk_workspace_size")
    return int(n.value)


def dkv_chunk_attention(batch: dkv_chunk_batch, pages: ChunkPages, pool: DevicePool, workspace: torch.Tensor | None,
                        stream=None) -> None:
    """Append the chunk to its pages and attend; of the pool the status word is used."""
    _on_device_of(batch, pages.k, pool.status, workspace)
    gc, pc = _chunk_pages(batch, pages), pool.c()
    rc = load().dkv_chunk_attention(ctypes.byref(batch), ctypes.byref(gc), ctypes.byref(pc), *_workspace(workspace),
                                    _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_chunk_attention")


def dkv_chunk_significance(batch: dkv_chunk_batch, pages: ChunkPages, sig_sum: torch.Tensor, pool: DevicePool,
                           stream=None) -> None:
    """sig_sum fp32 [L][R * cap][Hq]."""
    _want(sig_sum, "sig_sum", torch.float32, (batch.L * batch.R * batch.cap * batch.Hq,), pages.k)
    _on_device_of(batch, pages.k, pool.status)
    gc, pc = _chunk_pages(batch, pages), pool.c()
    rc = load().dkv_chunk_significance(ctypes.byref(batch), ctypes.byref(gc), _p(sig_sum), ctypes.byref(pc),
                                       _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_chunk_significance")


def make_evict_batch(L: int, R: int, Hq: int, Hkv: int, cap: int, budgets: torch.Tensor, ctx_lens: torch.Tensor,
                     sig_sum: torch.Tensor, classes: torch.Tensor, slot_of: torch.Tensor,
                     sig_cnt: torch.Tensor | None = None, sinks: int = 0, window: int = 0,
                     unit_base: int = 0) -> dkv_evict_batch:
    """budgets, ctx_lens int32 [R]; sig_sum fp32 [L][R * cap][Hq]; classes uint8 and slot_of int32
    [L][R * cap][Hkv]; sig_cnt int32 [R * cap], or None to compare the sums."""
    rows = int(L) * int(R) * int(cap)
    _want(budgets, "budgets", torch.int32, (int(R),), sig_sum)
    _want(ctx_lens, "ctx_lens", torch.int32, (int(R),), sig_sum)
    _want(sig_sum, "sig_sum", torch.float32, (rows * int(Hq),), sig_sum)
    _want(sig_cnt, "sig_cnt", torch.int32, (int(R) * int(cap),), sig_sum)
    _want(classes, "classes", torch.uint8, (rows * int(Hkv),), sig_sum)
    _want(slot_of, "slot_of", torch.int32, (rows * int(Hkv),), sig_sum)
    at = (budgets, ctx_lens, sig_sum, sig_cnt, classes, slot_of)
    return _holding(dkv_evict_batch(int(L), int(R), int(Hq), int(Hkv), int(cap), int(sinks), int(window), 0,
                                    int(unit_base), *map(_p, at)), *at)


def dkv_evict_workspace_size(batch: dkv_evict_batch, pool: DevicePool, tables) -> int:
    n = ctypes.c_size_t(0)
    pc, tc = pool.c(), _evict_tables(batch, tables)
    rc = load().dkv_evict_workspace_size(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), ctypes.byref(n))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_evict_workspace_size")
    return int(n.value)


def dkv_evict(batch: dkv_evict_batch, pool: DevicePool, tables, workspace: torch.Tensor, stream=None) -> None:
    _on_device_of(batch, pool.status, workspace)
    pc, tc = pool.c(), _evict_tables(batch, tables)
    rc = load().dkv_evict(ctypes.byref(batch), ctypes.byref(pc), ctypes.byref(tc), *_workspace(workspace),
                          _stream(stream))
    if rc != DKV_OK:
        raise DkvError(rc, "dkv_evict")


class _TableView:
    """Tables of a contiguous run of units (pointer offsets into DeviceTables)."""

    def __init__(self, t: DeviceTables, u0: int):
        self.t, self.u0 = t, int(u0)

    def units(self) -> int:
        return self.t.units() - self.u0

    def c(self) -> dkv_tables:
        return dkv_tables(_p(self.t.fwd) + 4 * self.u0 * self.t.pmax, self.t.pmax, 0,
                          _p(self.t.unit_hdr) + 16 * self.u0)


class Decoder:
    """Device state of a generation workload: pool, unit tables (pmax =
    ceil(cap / P) + 1), capacity-strided classes and slot index, workspace.
    prefill_layer() fills one layer's units with dkv_compact; index() derives
    classes and slot_of from the pages; step() runs dkv_decode_step."""

    def __init__(self, L: int, R: int, Hq: int, Hkv: int, cap: int, P: int, F: int, device="cuda",
                 window: int = 0, mode: int = 0, scheme: int = 0):
        self.L, self.R, self.Hq, self.Hkv, self.cap, self.P = L, R, Hq, Hkv, cap, P
        self.window, self.mode = int(window), int(mode)
        self.U = L * R * Hkv
        self.pmax = -(-cap // P) + 1
        self.device = torch.device(device)
        self.pool = DevicePool(F, P, device, scheme=scheme)
        self.tables = DeviceTables(self.U, self.pmax, device)
        rows = L * R * cap * Hkv
        self.classes = torch.zeros(rows, dtype=torch.uint8, device=device)
        self.slot_of = torch.full((rows,), -1, dtype=torch.int32, device=device)
        self.workspace = torch.empty(dkv_decode_workspace_size(self.batch({})), dtype=torch.uint8, device=device)
        dkv_init_pool(self.pool)
        self._pre_ws = self._ops_ws = self._evict_ws = None
        self._ext_ws: list[torch.Tensor] = []  # outgrown ones stay: a captured graph may use them

    def batch(self, d: dict) -> dkv_decode_batch:
        g = d.get
        at = (g("k_new"), g("v_new"), g("sig_sum"), g("sig_cnt"), g("ctx_lens"), g("new_lens"), self.classes, self.slot_of)
        return _holding(dkv_decode_batch(self.L, self.R, self.Hq, self.Hkv, 128, self.cap, 0, *map(_p, at), self.window,
                                         self.mode), *at)

    def prefill_layer(self, inp: dict, layer: int, max_len: int, alpha_h: float, alpha_l: float,
                      stream=None) -> None:
        """dkv_compact of one layer's prefill inputs (L = 1) into this pool,
        units of layer `layer` (unit_base and table rows offset)."""
        T = int(inp["T"])
        cls = self._scratch(max(T * self.Hkv, 1), stream)
        b = make_batch(inp, cls, max_len, unit_base=layer * self.R * self.Hkv)
        need = dkv_workspace_size(b)
        if self._pre_ws is None or self._pre_ws.numel() < need:
            self._pre_ws = self._scratch(need, stream)
        dkv_compact(b, alpha_h, alpha_l, self.pool, _TableView(self.tables, layer * self.R * self.Hkv),
                    self._pre_ws, stream=stream)

    def index(self, ctx_lens: torch.Tensor, stream=None) -> None:
        dkv_decode_index(self.batch({"ctx_lens": ctx_lens}), self.pool, self.tables, stream=stream)

    def step(self, d: dict, alpha_h: float, alpha_l: float, stream=None, spin_limit: int = -1,
             profiler=None) -> None:
        dkv_decode_step(self.batch(d), alpha_h, alpha_l, self.pool, self.tables, self.workspace, stream=stream,
                        spin_limit=spin_limit, profiler=profiler)

    def attend(self, q: torch.Tensor, ctx_lens: torch.Tensor, out: torch.Tensor, scale: float, layer0: int = 0,
               k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None,
               new_lens: torch.Tensor | None = None, sig_sum: torch.Tensor | None = None, stream=None) -> None:
        """dkv_decode_attention over layers [layer0, layer0 + q.shape[0])."""
        b = dkv_attn_batch(self.L, self.R, self.Hq, self.Hkv, self.cap, int(layer0), int(q.shape[0]), _p(q),
                           _p(k_new), _p(v_new), _p(new_lens), _p(ctx_lens), float(scale), _p(out), _p(sig_sum))
        dkv_decode_attention(b, self.pool, self.tables, stream=stream)

    def _extend_batch(self, q: torch.Tensor, new_lens: torch.Tensor, *args, **kw) -> dkv_extend_batch:
        if new_lens.numel() != self.R:  # the tables' units are numbered by all of them
            raise ValueError(f"new_lens: the {self.R} requests' lengths are wanted, 0 for those without new tokens")
        return make_extend_batch(self.L, self.Hkv, self.cap, q, new_lens, *args, **kw)

    def extend(self, q: torch.Tensor, new_lens: torch.Tensor, ctx_lens: torch.Tensor, max_new: int, out: torch.Tensor,
               scale: float, k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, layer0: int = 0, workspace: torch.Tensor | None = None,
               stream=None) -> None:
        """dkv_extend_attention of several new tokens a request over layers [layer0, layer0 + q.shape[0]).

        Calls (and replays of captured ones) that may run at the same time need a workspace each, of
        dkv_extend_workspace_size bytes; without one they share the decoder's and run in stream order."""
        b = self._extend_batch(q, new_lens, ctx_lens, max_new, scale, k_new=k_new, v_new=v_new, out=out, lse=lse,
                               layer0=layer0)
        if workspace is None:
            need = dkv_extend_workspace_size(b, self.pool, self.tables)
            if need and (not self._ext_ws or self._ext_ws[-1].numel() < need):
                self._ext_ws.append(self._scratch(need, stream))
            workspace = self._ext_ws[-1] if need else None
        dkv_extend_attention(b, self.pool, self.tables, workspace, stream=stream)

    def extend_significance(self, q: torch.Tensor, new_lens: torch.Tensor, acc_lens: torch.Tensor,
                            ctx_lens: torch.Tensor, max_new: int, scale: float, lse: torch.Tensor,
                            sig_sum: torch.Tensor, k_new: torch.Tensor | None = None,
                            v_new: torch.Tensor | None = None, layer0: int = 0, stream=None) -> None:
        """dkv_extend_significance of the first acc_lens[r] of those tokens."""
        b = self._extend_batch(q, new_lens, ctx_lens, max_new, scale, k_new=k_new, v_new=v_new, lse=lse, layer0=layer0)
        dkv_extend_significance(b, acc_lens, sig_sum, self.pool, self.tables, stream=stream)

    def _scratch(self, n: int, stream) -> torch.Tensor:
        # memory of the stream it is first used on: another stream's could still
        # be read or written by work that had it before
        with _on_stream(stream, self.device):
            return torch.empty(n, dtype=torch.uint8, device=self.device)

    def _page_ops_ws(self, stream) -> torch.Tensor:
        if self._ops_ws is None:
            self._ops_ws = self._scratch(dkv_page_ops_workspace_size(self.pool, self.tables), stream)
        return self._ops_ws

    def fork(self, src: torch.Tensor, dst: torch.Tensor, ctx_lens: torch.Tensor, sig_sum: torch.Tensor | None = None,
             sig_cnt: torch.Tensor | None = None, stream=None) -> None:
        """dkv_fork: request dst[k] becomes a copy of src[k] (pages, classes, slots and, where given, its
        significance rows and counts); the caller sets ctx_lens[dst] = ctx_lens[src]."""
        b = make_fork_batch(self.L, self.R, self.Hq, self.Hkv, self.cap, src, dst, ctx_lens, self.classes,
                            self.slot_of, sig_sum, sig_cnt)
        dkv_fork(b, self.pool, self.tables, self._page_ops_ws(stream), stream=stream)

    def release(self, reqs: torch.Tensor, stream=None) -> None:
        """dkv_release: the requests' pages go back to the free list; the caller sets their ctx_lens to 0."""
        dkv_release(make_release_batch(self.L, self.R, self.Hkv, reqs), self.pool, self.tables,
                    self._page_ops_ws(stream), stream=stream)

    def evict(self, budgets: torch.Tensor, ctx_lens: torch.Tensor, sig_sum: torch.Tensor,
              sig_cnt: torch.Tensor | None = None, sinks: int = 0, window: int | None = None, stream=None) -> None:
        """dkv_evict: each unit of a request keeps at most budgets[r] tokens (< 0: all), the most attended; the last
        `window` positions (the decoder's own where not given) and the first `sinks` stay."""
        b = make_evict_batch(self.L, self.R, self.Hq, self.Hkv, self.cap, budgets, ctx_lens, sig_sum, self.classes,
                             self.slot_of, sig_cnt, sinks, self.window if window is None else window)
        if self._evict_ws is None:
            self._evict_ws = self._scratch(dkv_evict_workspace_size(b, self.pool, self.tables), stream)
        dkv_evict(b, self.pool, self.tables, self._evict_ws, stream=stream)

    def defrag(self, stream=None) -> None:
        """dkv_defrag: the live pages move to the lowest ids."""
        dkv_defrag(self.pool, self.tables, self._page_ops_ws(stream), stream=stream)
