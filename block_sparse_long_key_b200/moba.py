"""Thin ctypes binding of libmoba.so (include/moba.h).

Argument marshalling only: tensors are checked for device, dtype and layout,
their device pointers and the current CUDA stream are handed to the C ABI,
and every step of the computation runs in the library's kernels.  There is
no CPU or PyTorch fallback: a missing library or a non-CUDA tensor raises.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoba.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "moba.h")

MOBA_OK, MOBA_EINVAL, MOBA_EALIGN, MOBA_EWORKSPACE, MOBA_ELAUNCH, MOBA_EDEVICE = 0, -1, -2, -3, -4, -5
STATUS_BAD_SEQLENS, STATUS_BAD_SEL_IDX, STATUS_INDEX_OVERFLOW, STATUS_TIMEOUT = 1, 2, 4, 8
STATUS_NO_PAGES, STATUS_BAD_TABLE, STATUS_NONFINITE = 16, 32, 64
PATH_ROUTE_TCGEN05, PATH_FWD_TCGEN05, PATH_BWD_TCGEN05, PATH_EXACT_ROWS = 1, 2, 4, 8


class Shape(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("h_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("topk", ctypes.c_int32),
    ]


class CacheStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n_pages", "max_blocks", "h_kv", "head_dim", "block_size", "kind",
                                              "conv_width", "set_back")] + \
               [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "cent", "tail_k", "tail_v", "hist",
                                               "block_table", "row_state", "free_pages", "ring")]


class PlanStruct(ctypes.Structure):
    _fields_ = [("total_new", ctypes.c_int32)] + \
               [(n, ctypes.c_void_p) for n in ("cu_new", "token_row", "token_pos", "slot_map")]


class MobaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (where, status_string(code), code))


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoba.so (built in-tree by ``block_sparse_long_key_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoba.so is not built (%s); run python -m block_sparse_long_key_b200.build"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, S, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(Shape)
        L.moba_fwd_workspace_size.argtypes = [F]
        L.moba_fwd_workspace_size.restype = S
        L.moba_bwd_workspace_size.argtypes = [F]
        L.moba_bwd_workspace_size.restype = S
        L.moba_key_conv_centroid.argtypes = [P, P, I, P, F, P, P, P, S, P]
        L.moba_key_conv_centroid.restype = I
        L.moba_forward.argtypes = [P, P, P, P, F, P, I, P, P, P, P, P, S, P]
        L.moba_forward.restype = I
        L.moba_build_index.argtypes = [P, P, F, P, P, P, S, P]
        L.moba_build_index.restype = I
        L.moba_backward.argtypes = [P, P, P, P, P, P, P, P, F, P, P, P, P, S, P, P]
        L.moba_backward.restype = I
        L.moba_key_conv_backward.argtypes = [P, P, I, P, F, P, P, P, P, S, P]
        L.moba_key_conv_backward.restype = I
        L.moba_set_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), I]
        L.moba_set_stage_events.restype = I
        L.moba_check_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
        L.moba_check_status.restype = I
        L.moba_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, P, S, P]
        L.moba_selftest_bounded_wait.restype = I
        L.moba_check_path.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
        L.moba_check_path.restype = I
        L.moba_status_string.argtypes = [I]
        C, N = ctypes.POINTER(CacheStruct), ctypes.POINTER(PlanStruct)
        L.moba_cache_workspace_size.argtypes = [C, I, I]
        L.moba_cache_workspace_size.restype = S
        L.moba_cache_reset.argtypes = [C, P]
        L.moba_cache_reset.restype = I
        L.moba_cache_tables.argtypes = [C, P, P, P, N, P, S, P]
        L.moba_cache_tables.restype = I
        L.moba_cache_append.argtypes = [C, N, P, P, P, P, S, P]
        L.moba_cache_append.restype = I
        L.moba_cache_route.argtypes = [C, N, P, I, I, P, P, S, P]
        L.moba_cache_route.restype = I
        L.moba_cache_attention.argtypes = [C, N, P, I, P, I, P, P, P, S, P]
        L.moba_cache_attention.restype = I
        L.moba_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def header_functions():
    """Names of the functions include/moba.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moba_[a-z_]+)\s*\(", text)))


def status_string(code: int) -> str:
    return lib().moba_status_string(int(code)).decode()


def make_shape(total_tokens, batch, h_q, h_kv, head_dim, block_size, topk) -> Shape:
    return Shape(int(total_tokens), int(batch), int(h_q), int(h_kv), int(head_dim), int(block_size), int(topk))


def fwd_workspace_size(shape: Shape) -> int:
    return int(lib().moba_fwd_workspace_size(ctypes.byref(shape)))


def bwd_workspace_size(shape: Shape) -> int:
    return int(lib().moba_bwd_workspace_size(ctypes.byref(shape)))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims" % (name, ndim))


def _check(rc: int, where: str):
    if rc != MOBA_OK:
        raise MobaError(rc, where)


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's allocator returns 512-byte aligned blocks; the ABI asks for 256.
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def shape_of(q: torch.Tensor, k: torch.Tensor, cu_seqlens: torch.Tensor, block_size: int, topk: int) -> Shape:
    T, hq, d = q.shape
    return make_shape(T, cu_seqlens.numel() - 1, hq, k.shape[1], d, block_size, topk)


def key_conv_centroid(k, cu_seqlens, block_size, conv_w=None, workspace=None, h_q=None):
    """Returns (k', centroid [h_kv, T//B + batch, d] fp32); k' is None without conv."""
    _need(k, torch.bfloat16, "k", 3)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    T, hkv, d = k.shape
    shape = make_shape(T, cu_seqlens.numel() - 1, h_q or hkv, hkv, d, block_size, 1)
    width = 0
    k_out = None
    if conv_w is not None:
        _need(conv_w, torch.float32, "conv_w", 3)
        width = conv_w.shape[2]
        k_out = torch.empty_like(k)
    nb = T // block_size + shape.batch
    cent = torch.empty((hkv, nb, d), dtype=torch.float32, device=k.device)
    ws = workspace if workspace is not None else alloc_workspace(fwd_workspace_size(shape), k.device)
    rc = lib().moba_key_conv_centroid(_ptr(k), _ptr(conv_w), width, _ptr(cu_seqlens), ctypes.byref(shape),
                                      _ptr(k_out), _ptr(cent), _ptr(ws), ws.numel(), _stream())
    _check(rc, "moba_key_conv_centroid")
    return k_out, cent


def forward(q, k, v, cu_seqlens, block_size: int, topk: int, conv_w=None, workspace=None,
            out=None, lse=None, sel_idx=None, k_conv=None):
    """MoBA forward.  Returns (out, lse, sel_idx, k_used) where k_used is k'
    when ``conv_w`` is given (pass it to ``backward``), else k."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n, 3)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    shape = shape_of(q, k, cu_seqlens, block_size, topk)
    T, hq, d = q.shape
    dev = q.device
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((T, hq), dtype=torch.float32, device=dev) if lse is None else lse
    sel_idx = torch.empty((T, hq, topk), dtype=torch.int32, device=dev) if sel_idx is None else sel_idx
    width = 0
    if conv_w is not None:
        _need(conv_w, torch.float32, "conv_w", 3)
        width = conv_w.shape[2]
        k_conv = torch.empty_like(k) if k_conv is None else k_conv
    else:
        k_conv = None
    ws = workspace if workspace is not None else alloc_workspace(fwd_workspace_size(shape), dev)
    rc = lib().moba_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), ctypes.byref(shape), _ptr(conv_w), width,
                            _ptr(k_conv), _ptr(out), _ptr(lse), _ptr(sel_idx), _ptr(ws), ws.numel(), _stream())
    _check(rc, "moba_forward")
    return out, lse, sel_idx, (k_conv if k_conv is not None else k)


def build_index(sel_idx, cu_seqlens, h_kv: int, block_size: int, workspace=None):
    """Returns (blk_ptr [h_kv * nblk + 1], blk_rows [T * h_q * topk]) int32."""
    _need(sel_idx, torch.int32, "sel_idx", 3)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    T, hq, topk = sel_idx.shape
    shape = make_shape(T, cu_seqlens.numel() - 1, hq, h_kv, 64, block_size, topk)
    nb = T // block_size + shape.batch
    dev = sel_idx.device
    ptr = torch.empty(h_kv * nb + 1, dtype=torch.int32, device=dev)
    rows = torch.empty(max(T * hq * topk, 1), dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else alloc_workspace(bwd_workspace_size(shape), dev)
    rc = lib().moba_build_index(_ptr(sel_idx), _ptr(cu_seqlens), ctypes.byref(shape), _ptr(ptr), _ptr(rows),
                                _ptr(ws), ws.numel(), _stream())
    _check(rc, "moba_build_index")
    return ptr, rows


def backward(q, k, v, out, lse, dout, sel_idx, cu_seqlens, block_size: int, workspace=None,
             dq=None, dk=None, dv=None, fwd_workspace=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """MoBA backward with the selection fixed.  Returns (dq, dk, dv).

    ``fwd_workspace``: the workspace of the forward call that produced
    ``sel_idx`` (untouched since); its block index is reused."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, n, 3)
    _need(lse, torch.float32, "lse", 2)
    _need(sel_idx, torch.int32, "sel_idx", 3)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    topk = sel_idx.shape[2]
    shape = shape_of(q, k, cu_seqlens, block_size, topk)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws = workspace if workspace is not None else alloc_workspace(bwd_workspace_size(shape), q.device)
    rc = lib().moba_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(sel_idx),
                             _ptr(cu_seqlens), ctypes.byref(shape), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(),
                             _ptr(fwd_workspace), _stream())
    _check(rc, "moba_backward")
    return dq, dk, dv


STAGES = ["fwd_plan", "fwd_centroid", "fwd_route", "fwd_index", "fwd_attn", "fwd_finalize",
          "bwd_plan", "bwd_index", "bwd_pre", "bwd_attn", "bwd_dq", "conv_bwd"]


class StageEvents:
    """Installs a per-stage CUDA event table on this thread (see
    moba_set_stage_events); ``ms()`` returns {stage: milliseconds}."""

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * len(STAGES))]
        for e in self.events:   # torch creates the CUDA event on its first record
            e.record()
        self._arr = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])

    def __enter__(self):
        _check(lib().moba_set_stage_events(self._arr, len(self.events)), "moba_set_stage_events")
        return self

    def __exit__(self, *exc):
        lib().moba_set_stage_events(None, 0)

    def ms(self):
        return {n: self.events[2 * i].elapsed_time(self.events[2 * i + 1]) for i, n in enumerate(STAGES)}


def key_conv_backward(k, conv_w, cu_seqlens, block_size: int, dk_conv, workspace=None, dk=None, dw=None, h_q=None):
    """Gradients of the key conv: (dK of the original keys, dW [h_kv, d, W])."""
    _need(k, torch.bfloat16, "k", 3)
    _need(dk_conv, torch.bfloat16, "dk_conv", 3)
    _need(conv_w, torch.float32, "conv_w", 3)
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    T, hkv, d = k.shape
    shape = make_shape(T, cu_seqlens.numel() - 1, h_q or hkv, hkv, d, block_size, 1)
    dk = torch.empty_like(k) if dk is None else dk
    dw = torch.empty_like(conv_w) if dw is None else dw
    ws = workspace if workspace is not None else alloc_workspace(bwd_workspace_size(shape), k.device)
    rc = lib().moba_key_conv_backward(_ptr(k), _ptr(conv_w), conv_w.shape[2], _ptr(cu_seqlens), ctypes.byref(shape),
                                      _ptr(dk_conv), _ptr(dk), _ptr(dw), _ptr(ws), ws.numel(), _stream())
    _check(rc, "moba_key_conv_backward")
    return dk, dw


def check_status(workspace: torch.Tensor) -> int:
    """Synchronises the current stream and returns the device status bits."""
    st = ctypes.c_int32(0)
    rc = lib().moba_check_status(_ptr(workspace), _stream(), ctypes.byref(st))
    if rc not in (MOBA_OK, MOBA_EDEVICE):
        raise MobaError(rc, "moba_check_status")
    return int(st.value)


def check_path(workspace: torch.Tensor) -> int:
    """Synchronises the current stream and returns the kernel-path bits
    (PATH_*) the last call on ``workspace`` set."""
    st = ctypes.c_int32(0)
    _check(lib().moba_check_path(_ptr(workspace), _stream(), ctypes.byref(st)), "moba_check_path")
    return int(st.value)


def selftest_bounded_wait(limit_ns: int, workspace: torch.Tensor) -> None:
    """Runs the bounded-wait self-test kernel (see moba_selftest_bounded_wait)
    on the current stream; read the outcome with ``check_status``."""
    _check(lib().moba_selftest_bounded_wait(int(limit_ns), _ptr(workspace), workspace.numel(), _stream()),
           "moba_selftest_bounded_wait")


# ---------------------------------------------------------------- paged 8-bit cache
CACHE_KINDS = {"e4m3": (0, torch.float8_e4m3fn), "int8": (1, torch.int8)}
_CACHE_HIST = 16


class CachePlan:
    """The new tokens of a step (see moba_cache_plan), packed row after row: cu_new int32 [rows + 1], token_row,
    token_pos, slot_map int32 [T].  Checked once; the tensors are fixed."""
    __slots__ = ("cu_new", "token_row", "token_pos", "slot_map", "total_new", "rows", "index", "struct", "_ref")

    def __init__(self, cu_new, token_row, token_pos, slot_map):
        _need(cu_new, torch.int32, "cu_new", 1)
        T = token_row.shape[0]
        for n, t in (("token_row", token_row), ("token_pos", token_pos), ("slot_map", slot_map)):
            _need_shape(t, torch.int32, n, (T,))
        if len({t.get_device() for t in (cu_new, token_row, token_pos, slot_map)}) != 1:
            raise ValueError("a plan's tensors must be on one device")
        self._set(cu_new, token_row, token_pos, slot_map, T)

    def _set(self, cu_new, token_row, token_pos, slot_map, T):
        self.cu_new, self.token_row, self.token_pos, self.slot_map = cu_new, token_row, token_pos, slot_map
        self.total_new, self.rows, self.index = T, cu_new.shape[0] - 1, cu_new.get_device()
        self.struct = PlanStruct(T, cu_new.data_ptr(), token_row.data_ptr(), token_pos.data_ptr(), slot_map.data_ptr())
        self._ref = ctypes.byref(self.struct)
        return self

    def __iter__(self):
        return iter((self.cu_new, self.token_row, self.token_pos, self.slot_map))


class Cache:
    """The buffers of a paged 8-bit cache (layouts: moba_cache in include/moba.h), checked once.

    ``alloc_cache`` makes an empty one.  Built from tensors of the caller, those
    that a call does not use may be None (bookkeeping alone needs block_table,
    row_state, free_pages and ring).  The tensors are fixed: write into them,
    do not rebind them.

    ``set_back`` (caches with a key conv): how many tokens a row's length may be
    set back by, as when only part of a step's drafts are accepted; 0 to
    17 - conv_width."""

    def __init__(self, *, rows: int, n_pages: int, max_blocks: int, h_kv: int, head_dim: int, block_size: int,
                 kind: str = "e4m3", conv_width: int = 0, k=None, v=None, k_scale=None, v_scale=None, cent=None,
                 tail_k=None, tail_v=None, hist=None, block_table=None, row_state=None, free_pages=None, ring=None,
                 set_back: int = 0):
        if kind not in CACHE_KINDS:
            raise ValueError("kind must be one of %s, got %r" % (sorted(CACHE_KINDS), kind))
        code, dt8 = CACHE_KINDS[kind]
        P, H, B, d = n_pages, h_kv, block_size, head_dim
        bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
        want = dict(k=(dt8, (P, H, B, d)), v=(dt8, (P, H, B, d)), k_scale=(f32, (P, H)), v_scale=(f32, (P, H)),
                    cent=(bf, (2, P, H, d)), tail_k=(bf, (rows, 2, H, B, d)), tail_v=(bf, (rows, 2, H, B, d)),
                    hist=(bf, (rows, _CACHE_HIST, H, d)), block_table=(i32, (rows, max_blocks)),
                    row_state=(i32, (rows, 2)), free_pages=(i32, (P,)), ring=(torch.int64, (2,)))
        given = dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, cent=cent, tail_k=tail_k, tail_v=tail_v, hist=hist,
                     block_table=block_table, row_state=row_state, free_pages=free_pages, ring=ring)
        devs = set()
        for n, x in given.items():
            if x is None:
                continue
            _need(x, want[n][0], n)
            if tuple(x.shape) != want[n][1]:
                raise ValueError("%s must have shape %s, got %s" % (n, want[n][1], tuple(x.shape)))
            devs.add(x.device)
        if len(devs) != 1:
            raise ValueError("the cache's tensors must be on one CUDA device")
        self.rows, self.n_pages, self.max_blocks, self.h_kv = int(rows), int(n_pages), int(max_blocks), int(h_kv)
        self.head_dim, self.block_size, self.kind, self.conv_width = int(d), int(B), kind, int(conv_width)
        self.set_back = int(set_back)
        self.device = devs.pop()
        self.index = self.device.index
        for n, x in given.items():
            setattr(self, n, x)
        self.struct = CacheStruct(self.rows, self.n_pages, self.max_blocks, self.h_kv, self.head_dim, self.block_size,
                                  code, self.conv_width, self.set_back,
                                  **{n: x.data_ptr() for n, x in given.items() if x is not None})
        self._ref = ctypes.byref(self.struct)

    def workspace_size(self, total_new: int, h_q: Optional[int] = None) -> int:
        """Bytes that a step of total_new tokens needs; a smaller step may need more (its rows are cut finer), so one
        workspace for many steps takes the largest of theirs."""
        return int(lib().moba_cache_workspace_size(self._ref, int(total_new), int(h_q or self.h_kv)))

    def alloc_workspace(self, total_new: int, h_q: Optional[int] = None) -> torch.Tensor:
        return alloc_workspace(self.workspace_size(total_new, h_q), self.device)

    def reset(self) -> None:
        """Empties the cache (moba_cache_reset)."""
        _launch(self, "moba_cache_reset")


# The current stream's handle: torch.cuda.current_stream builds a Stream object, which takes longer than the rest of a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _need_shape(t, dtype, name, shape):
    """A contiguous CUDA tensor of this type and shape (one look where all is well: these calls are short)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
        _need(t, dtype, name)
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _same_device(cache, **tensors):
    for n, t in tensors.items():
        if t is not None and t.get_device() != cache.index:
            raise ValueError("%s is on %s, the cache on %s" % (n, t.device, cache.device))


def _launch(cache, name, *args):
    """Calls moba_<name>(cache, *args, stream) on the cache's device and its current stream."""
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == cache.index:
        rc = fn(cache._ref, *args, _raw_stream(cache.index))
    else:
        with torch.cuda.device(cache.device):
            rc = fn(cache._ref, *args, _raw_stream(cache.index))
    if rc != MOBA_OK:
        raise MobaError(rc, name)


def _check_plan(cache, plan):
    if not isinstance(plan, CachePlan):
        raise TypeError("plan must be a CachePlan")
    if plan.rows != cache.rows or plan.index != cache.index:
        raise ValueError("the plan is for %d rows on device %d, the cache has %d on %d"
                         % (plan.rows, plan.index, cache.rows, cache.index))


def alloc_cache(rows: int, n_pages: int, max_blocks: int, h_kv: int, head_dim: int, block_size: int,
                kind: str = "e4m3", conv_width: int = 0, device=None, set_back: Optional[int] = None) -> Cache:
    """An empty cache on ``device`` (default: the current CUDA device).  With a key conv, lengths may be set back by
    ``set_back`` tokens (default: the most there can be, 17 - conv_width)."""
    if kind not in CACHE_KINDS:
        raise ValueError("kind must be one of %s, got %r" % (sorted(CACHE_KINDS), kind))
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if set_back is None:
        set_back = _CACHE_HIST + 1 - conv_width if conv_width > 1 else 0
    P, H, B, d = n_pages, h_kv, block_size, head_dim

    def new(dtype, *shape):
        return torch.empty(shape, dtype=dtype, device=dev)

    bf, f32, i32, dt8 = torch.bfloat16, torch.float32, torch.int32, CACHE_KINDS[kind][1]
    c = Cache(rows=rows, n_pages=P, max_blocks=max_blocks, h_kv=H, head_dim=d, block_size=B, kind=kind,
              conv_width=conv_width, k=new(dt8, P, H, B, d), v=new(dt8, P, H, B, d), k_scale=new(f32, P, H),
              v_scale=new(f32, P, H), cent=new(bf, 2, P, H, d), tail_k=new(bf, rows, 2, H, B, d),
              tail_v=new(bf, rows, 2, H, B, d), hist=new(bf, rows, _CACHE_HIST, H, d) if conv_width > 1 else None,
              block_table=new(i32, rows, max_blocks), row_state=new(i32, rows, 2), free_pages=new(i32, P),
              ring=new(torch.int64, 2), set_back=set_back)
    c.reset()
    return c


def cache_tables(cache: Cache, new_len: torch.Tensor, total_new: int, row_state_out=None, ring_out=None,
                 plan: Optional[CachePlan] = None, workspace=None) -> CachePlan:
    """Pages and slots for ``new_len`` (int32 [rows]; -1 releases a row) new tokens, at most ``total_new`` in all
    (moba_cache_tables).  Advances the cache's row_state and ring, or writes the state after the step to
    ``row_state_out`` / ``ring_out``.  Returns the plan the other calls take (written into ``plan`` if given)."""
    _need_shape(new_len, torch.int32, "new_len", (cache.rows,))
    T = int(total_new)
    if T < 0:
        raise ValueError("total_new must not be negative")
    if new_len.get_device() != cache.index:
        raise ValueError("new_len is on %s, the cache on %s" % (new_len.device, cache.device))
    if row_state_out is not None:
        _need_shape(row_state_out, torch.int32, "row_state_out", (cache.rows, 2))
    if ring_out is not None:
        _need_shape(ring_out, torch.int64, "ring_out", (2,))
    if plan is None:
        # one allocation, its parts 16-byte aligned (making a view takes longer than the kernel: no more than needed;
        # integers have no gradient that the plain split would look after)
        R, pad = cache.rows + 1, -T & 3
        buf = new_len.new_empty(3 * (T + pad) + R)
        if pad:
            row, _, pos, _, slot, _, cu = buf.unsafe_split_with_sizes((T, pad, T, pad, T, pad, R))
        else:
            row, pos, slot, cu = buf.unsafe_split_with_sizes((T, T, T, R))
        plan = CachePlan.__new__(CachePlan)._set(cu, row, pos, slot, T)
    else:
        _check_plan(cache, plan)
        if plan.total_new != T:
            raise ValueError("the plan has room for %d tokens, not total_new = %d" % (plan.total_new, T))
    ws = cache.alloc_workspace(0) if workspace is None else workspace
    _same_device(cache, row_state_out=row_state_out, ring_out=ring_out, workspace=ws)
    _launch(cache, "moba_cache_tables", new_len.data_ptr(), _addr(row_state_out), _addr(ring_out), plan._ref,
            ws.data_ptr(), ws.numel())
    return plan


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def cache_append(cache: Cache, plan: CachePlan, k: torch.Tensor, v: torch.Tensor, conv_w=None, workspace=None) -> None:
    """Writes the new keys and values [T, h_kv, d] bf16 into the cache, through the key conv when the cache has one
    (``conv_w`` fp32 [h_kv, d, conv_width]) (moba_cache_append)."""
    _check_plan(cache, plan)
    shape = (plan.total_new, cache.h_kv, cache.head_dim)
    _need_shape(k, torch.bfloat16, "k", shape)
    _need_shape(v, torch.bfloat16, "v", shape)
    if (conv_w is not None) != (cache.conv_width > 0):
        raise ValueError("conv_w must be given exactly when the cache has a key conv")
    if conv_w is not None:
        _need_shape(conv_w, torch.float32, "conv_w", (cache.h_kv, cache.head_dim, cache.conv_width))
    ws = alloc_workspace(256, cache.device) if workspace is None else workspace
    _same_device(cache, k=k, v=v, conv_w=conv_w, workspace=ws)
    _launch(cache, "moba_cache_append", plan._ref, k.data_ptr(), v.data_ptr(), _addr(conv_w), ws.data_ptr(), ws.numel())


def _check_q(cache, plan, q):
    _check_plan(cache, plan)
    _need(q, torch.bfloat16, "q", 3)
    T, h_q, d = q.shape
    if T != plan.total_new or d != cache.head_dim:
        raise ValueError("q must have shape (%d, h_q, %d), got %s" % (plan.total_new, cache.head_dim, tuple(q.shape)))
    return T, h_q


def cache_route(cache: Cache, plan: CachePlan, q: torch.Tensor, topk: int, workspace=None, sel_idx=None) -> torch.Tensor:
    """The blocks of every new query: sel_idx int32 [T, h_q, topk] (moba_cache_route)."""
    T, h_q = _check_q(cache, plan, q)
    topk = int(topk)
    if sel_idx is None:
        sel_idx = torch.empty((T, h_q, topk), dtype=torch.int32, device=cache.device)
    else:
        _need_shape(sel_idx, torch.int32, "sel_idx", (T, h_q, topk))
    ws = cache.alloc_workspace(T, h_q) if workspace is None else workspace
    _same_device(cache, q=q, sel_idx=sel_idx, workspace=ws)
    _launch(cache, "moba_cache_route", plan._ref, q.data_ptr(), h_q, topk, sel_idx.data_ptr(), ws.data_ptr(), ws.numel())
    return sel_idx


def cache_attention(cache: Cache, plan: CachePlan, q: torch.Tensor, sel_idx: Optional[torch.Tensor] = None,
                    workspace=None, out=None, lse=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the new queries over the blocks of ``sel_idx`` (cache_route's), or over all earlier tokens when it
    is None.  Returns (out bf16 [T, h_q, d], lse fp32 [T, h_q]) (moba_cache_attention)."""
    T, h_q = _check_q(cache, plan, q)
    topk = 1
    if sel_idx is not None:
        _need(sel_idx, torch.int32, "sel_idx", 3)
        topk = sel_idx.shape[2]
        _need_shape(sel_idx, torch.int32, "sel_idx", (T, h_q, topk))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_shape(out, torch.bfloat16, "out", q.shape)
    if lse is None:
        lse = torch.empty((T, h_q), dtype=torch.float32, device=cache.device)
    else:
        _need_shape(lse, torch.float32, "lse", (T, h_q))
    ws = cache.alloc_workspace(T, h_q) if workspace is None else workspace
    _same_device(cache, q=q, sel_idx=sel_idx, out=out, lse=lse, workspace=ws)
    _launch(cache, "moba_cache_attention", plan._ref, q.data_ptr(), h_q, _addr(sel_idx), topk, out.data_ptr(),
            lse.data_ptr(), ws.data_ptr(), ws.numel())
    return out, lse
