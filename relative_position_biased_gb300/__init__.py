"""GB300 relative-attention forward (Inkling-style relative position bias).

A thin ctypes binding over ``librelattn.so`` (C ABI in ``include/relattn.h``).
Functions named ``relattn_*`` mirror the C entry points one to one and only
marshal arguments; ``prefill`` / ``decode`` are conveniences that also allocate
``out`` / ``lse`` / workspace with torch (device memory is torch's job) before
calling the same entry points.  Every step of the computation runs in the CUDA
kernels; if the library is missing these functions raise -- there is no
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional, Tuple

from . import workloads  # noqa: F401  (seeded input generators)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librelattn.so")
# the same kernels with the relattn_test_* hooks (built beside the product library)
TEST_LIB_PATH = os.path.join(_HERE, "librelattn_test.so")

RELATTN_OK = 0
RELATTN_ERR_INVALID_ARG = 1
RELATTN_ERR_UNSUPPORTED = 2
RELATTN_ERR_TIMEOUT = 4
STATUS_NAMES = {
    0: "RELATTN_OK", 1: "RELATTN_ERR_INVALID_ARG", 2: "RELATTN_ERR_UNSUPPORTED",
    3: "RELATTN_ERR_CUDA", 4: "RELATTN_ERR_TIMEOUT", 5: "RELATTN_ERR_WORKSPACE",
    6: "RELATTN_ERR_DEVICE_ARGS",
}
EXPORTED = (
    "relattn_prefill", "relattn_decode", "relattn_decode_workspace_size",
    "relattn_decode_num_splits", "relattn_combine", "relattn_get_device_error",
    "relattn_status_string", "relattn_version", "relattn_decode_noalloc",
    "relattn_last_device_error_word",
    "relattn_prologue", "relattn_backward", "relattn_backward_workspace_size",
    "relattn_decode_paged", "relattn_decode_mxfp8", "relattn_quantize_mxfp8",
    "relattn_prologue_mxfp8",
    "relattn_store_nvfp4", "relattn_load_nvfp4", "relattn_decode_nvfp4",
    "relattn_decode_nvfp4_workspace_size", "relattn_key_weights",
    "relattn_key_weights_workspace_size", "relattn_evict", "relattn_evict_workspace_size",
    "relattn_extend", "relattn_extend_workspace_size", "relattn_prologue_paged",
    "relattn_backward_sinks", "relattn_backward_sinks_workspace_size",
)
# exported by the test build only
TEST_HOOKS = (
    "relattn_test_skip_k_tile", "relattn_test_band_ctas", "relattn_test_prologue_skip_tile",
    "relattn_test_backward_skip_step",
)
NOALLOC_SCRATCH_BYTES = 32 << 20   # RELATTN_NOALLOC_SCRATCH_BYTES
HEAD_DIM = workloads.HEAD_DIM


class RelattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class RelattnParams(ctypes.Structure):
    """Mirror of ``relattn_params`` (field order and types must match the header)."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("r", ctypes.c_void_p), ("P", ctypes.c_void_p),
        ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("batch", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
        ("max_seqlen_q", ctypes.c_int32), ("max_seqlen_k", ctypes.c_int32),
        ("num_heads_q", ctypes.c_int32), ("num_heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("r_dim", ctypes.c_int32), ("rel_extent", ctypes.c_int32),
        ("window", ctypes.c_int32), ("alpha", ctypes.c_float), ("log_scale_base", ctypes.c_float),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("num_splits", ctypes.c_int32),
    ]


class RelattnPagedKV(ctypes.Structure):
    """Mirror of ``relattn_paged_kv``."""
    _fields_ = [("block_table", ctypes.c_void_p), ("max_pages_per_seq", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


class RelattnKvMxfp8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class RelattnKvNvfp4(ctypes.Structure):
    """Mirror of ``relattn_kv_nvfp4``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_global", ctypes.c_void_p), ("v_global", ctypes.c_void_p),
                ("rows", ctypes.c_int64)]


class RelattnCacheRowsParams(ctypes.Structure):
    """Mirror of ``relattn_cache_rows_params``."""
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("batch", ctypes.c_int32), ("total_q", ctypes.c_int32),
        ("num_heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("cache", ctypes.POINTER(RelattnKvNvfp4)), ("pages", ctypes.POINTER(RelattnPagedKV)),
    ]


class RelattnPositions(ctypes.Structure):
    """Mirror of ``relattn_positions``."""
    _fields_ = [("key_pos", ctypes.c_void_p), ("q_pos", ctypes.c_void_p)]


class RelattnKeyWeightsParams(ctypes.Structure):
    """Mirror of ``relattn_key_weights_params``."""
    _fields_ = [
        ("fwd", RelattnParams), ("cache", ctypes.POINTER(RelattnKvNvfp4)),
        ("positions", ctypes.POINTER(RelattnPositions)), ("pages", ctypes.POINTER(RelattnPagedKV)),
        ("weights_in", ctypes.c_void_p), ("weights_out", ctypes.c_void_p), ("decay", ctypes.c_float),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


MAX_PLANES = 8   # RELATTN_MAX_PLANES


class RelattnPlane(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("bytes", ctypes.c_int32)]


class RelattnEvictParams(ctypes.Structure):
    """Mirror of ``relattn_evict_params``."""
    _fields_ = [
        ("weights", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("cu_seqlens_keep", ctypes.c_void_p), ("key_pos", ctypes.c_void_p),
        ("batch", ctypes.c_int32), ("total_k", ctypes.c_int32), ("total_keep", ctypes.c_int32),
        ("max_seqlen_k", ctypes.c_int32), ("num_heads_kv", ctypes.c_int32),
        ("sink", ctypes.c_int32), ("recent", ctypes.c_int32),
        ("rows", ctypes.c_int64), ("rows_keep", ctypes.c_int64),
        ("pages", ctypes.POINTER(RelattnPagedKV)), ("pages_keep", ctypes.POINTER(RelattnPagedKV)),
        ("num_planes", ctypes.c_int32), ("planes", RelattnPlane * MAX_PLANES),
        ("weights_out", ctypes.c_void_p), ("key_pos_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("clear_out", ctypes.c_int32),
    ]


class RelattnBwdParams(ctypes.Structure):
    """Mirror of ``relattn_bwd_params`` (field order and types must match the header)."""
    _fields_ = [
        ("fwd", RelattnParams), ("dout", ctypes.c_void_p), ("dq", ctypes.c_void_p),
        ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p), ("dr", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class RelattnPrologueParams(ctypes.Structure):
    """Mirror of ``relattn_prologue_params`` (field order and types must match the header)."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("conv_k", ctypes.c_void_p), ("conv_v", ctypes.c_void_p),
        ("norm_q", ctypes.c_void_p), ("norm_k", ctypes.c_void_p), ("eps", ctypes.c_float),
        ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("batch", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
        ("num_heads_q", ctypes.c_int32), ("num_heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("q_out", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("conv_state_in_k", ctypes.c_void_p), ("conv_state_in_v", ctypes.c_void_p),
        ("conv_state_out_k", ctypes.c_void_p), ("conv_state_out_v", ctypes.c_void_p),
    ]


_lock = threading.RLock()
_lib = None
_libs = {}    # path -> configured handle


def build(force: bool = False) -> str:
    from .buildlib import build as _build
    return _build(force=force)


def _open(path: str):
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with relative_position_biased_gb300.build()")
    return ctypes.CDLL(path)


def load_library(path: Optional[str] = None):
    """Load ``librelattn.so`` (raises if it has not been built).  Inside
    ``test_library()`` this is the test build instead."""
    global _lib
    with _lock:
        if path is not None:
            return _configure(path)
        if _lib is None:
            _lib = _configure(LIB_PATH)
        return _lib


def load_test_library():
    """Load ``librelattn_test.so``: the same kernels plus the relattn_test_* hooks."""
    with _lock:
        lib = _configure(TEST_LIB_PATH)
        for name in TEST_HOOKS:
            getattr(lib, name).restype = ctypes.c_int
        lib.relattn_test_skip_k_tile.argtypes = [ctypes.c_int32]
        lib.relattn_test_prologue_skip_tile.argtypes = [ctypes.c_int32]
        lib.relattn_test_backward_skip_step.argtypes = [ctypes.c_int32, ctypes.c_int32]
        lib.relattn_test_band_ctas.argtypes = [ctypes.c_int32]
        return lib


@contextlib.contextmanager
def test_library():
    """Route every call of this module to the test build for the duration of
    the block (tests that set a hook run their calls inside one).  The device
    error word and the hooks belong to the test build's own copy."""
    global _lib
    with _lock:
        prev = load_library()
        _lib = load_test_library()
    try:
        yield _lib
    finally:
        with _lock:
            _lib = prev


def _configure(path: str):
    with _lock:
        if path in _libs:
            return _libs[path]
        lib = _open(path)
        P, vp = ctypes.POINTER(RelattnParams), ctypes.c_void_p
        for name in ("relattn_prefill", "relattn_decode", "relattn_decode_noalloc"):
            f = getattr(lib, name)
            f.argtypes, f.restype = [P, vp], ctypes.c_int
        lib.relattn_decode_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.relattn_decode_workspace_size.restype = ctypes.c_int
        lib.relattn_decode_num_splits.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        lib.relattn_decode_num_splits.restype = ctypes.c_int
        lib.relattn_combine.argtypes = [vp, vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                        vp, vp, vp]
        lib.relattn_combine.restype = ctypes.c_int
        lib.relattn_get_device_error.argtypes = [vp]
        lib.relattn_get_device_error.restype = ctypes.c_int
        lib.relattn_status_string.argtypes = [ctypes.c_int]
        lib.relattn_status_string.restype = ctypes.c_char_p
        lib.relattn_last_device_error_word.argtypes = []
        lib.relattn_last_device_error_word.restype = ctypes.c_int32
        lib.relattn_decode_paged.argtypes = [P, ctypes.POINTER(RelattnPagedKV), vp]
        lib.relattn_decode_paged.restype = ctypes.c_int
        lib.relattn_decode_mxfp8.argtypes = [P, ctypes.POINTER(RelattnKvMxfp8), vp]
        lib.relattn_decode_mxfp8.restype = ctypes.c_int
        lib.relattn_quantize_mxfp8.argtypes = [vp, ctypes.c_int64, vp, vp, vp]
        lib.relattn_quantize_mxfp8.restype = ctypes.c_int
        BP = ctypes.POINTER(RelattnBwdParams)
        lib.relattn_backward.argtypes = [BP, vp]
        lib.relattn_backward.restype = ctypes.c_int
        lib.relattn_backward_workspace_size.argtypes = [BP, ctypes.POINTER(ctypes.c_size_t)]
        lib.relattn_backward_workspace_size.restype = ctypes.c_int
        lib.relattn_prologue.argtypes = [ctypes.POINTER(RelattnPrologueParams), vp]
        lib.relattn_prologue.restype = ctypes.c_int
        lib.relattn_prologue_mxfp8.argtypes = [ctypes.POINTER(RelattnPrologueParams),
                                               ctypes.POINTER(RelattnKvMxfp8), vp]
        lib.relattn_prologue_mxfp8.restype = ctypes.c_int
        KV, PG, POS = (ctypes.POINTER(RelattnKvNvfp4), ctypes.POINTER(RelattnPagedKV),
                       ctypes.POINTER(RelattnPositions))
        SZ = ctypes.POINTER(ctypes.c_size_t)
        for name, args in (
                ("relattn_store_nvfp4", [ctypes.POINTER(RelattnCacheRowsParams), vp]),
                ("relattn_load_nvfp4", [ctypes.POINTER(RelattnCacheRowsParams), vp]),
                ("relattn_decode_nvfp4", [P, KV, POS, PG, vp]),
                ("relattn_decode_nvfp4_workspace_size", [P, POS, SZ]),
                ("relattn_key_weights", [ctypes.POINTER(RelattnKeyWeightsParams), vp]),
                ("relattn_key_weights_workspace_size", [ctypes.POINTER(RelattnKeyWeightsParams), SZ]),
                ("relattn_extend", [P, PG, ctypes.c_int32, vp]),
                ("relattn_extend_workspace_size", [P, PG, ctypes.c_int32, SZ]),
                ("relattn_prologue_paged", [ctypes.POINTER(RelattnPrologueParams), PG, vp]),
                ("relattn_backward_sinks", [BP, ctypes.c_int32, vp]),
                ("relattn_backward_sinks_workspace_size", [BP, ctypes.c_int32, SZ]),
                ("relattn_evict", [ctypes.POINTER(RelattnEvictParams), vp]),
                ("relattn_evict_workspace_size", [ctypes.POINTER(RelattnEvictParams), SZ])):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        lib.relattn_version.argtypes = []
        lib.relattn_version.restype = ctypes.c_char_p
        _libs[path] = lib
        return lib


def _check(status: int, where: str) -> None:
    if status != RELATTN_OK:
        raise RelattnError(status, where)


# ------------------------------------------------------------------ C mirrors

def relattn_prefill(params: RelattnParams, stream: int = 0) -> int:
    return load_library().relattn_prefill(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_decode(params: RelattnParams, stream: int = 0) -> int:
    return load_library().relattn_decode(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_decode_noalloc(params: RelattnParams, stream: int = 0) -> int:
    """Decode with the library's fixed scratch array; params.workspace is ignored."""
    return load_library().relattn_decode_noalloc(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_decode_workspace_size(params: RelattnParams) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_decode_workspace_size(ctypes.byref(params), ctypes.byref(n))
    return st, int(n.value)


def relattn_decode_num_splits(params: RelattnParams) -> Tuple[int, int]:
    n = ctypes.c_int32(0)
    st = load_library().relattn_decode_num_splits(ctypes.byref(params), ctypes.byref(n))
    return st, int(n.value)


def relattn_combine(o_part: int, lse_part: int, num_splits: int, total_q: int, num_heads: int,
                    out: int, lse: int, stream: int = 0) -> int:
    return load_library().relattn_combine(o_part, lse_part, num_splits, total_q, num_heads,
                                          out, lse, ctypes.c_void_p(stream))


def relattn_get_device_error(stream: int = 0) -> int:
    return load_library().relattn_get_device_error(ctypes.c_void_p(stream))


def relattn_last_device_error_word() -> int:
    return int(load_library().relattn_last_device_error_word())


def relattn_test_skip_k_tile(tile: int) -> int:
    """Test build: later tensor-core launches never load key tile ``tile`` (-1: off)."""
    return int(load_test_library().relattn_test_skip_k_tile(int(tile)))


def relattn_test_prologue_skip_tile(tile: int) -> int:
    """Test build: the staged prologue never copies token tile ``tile`` (-1: off)."""
    return int(load_test_library().relattn_test_prologue_skip_tile(int(tile)))


def relattn_test_backward_skip_step(kernel: int, step: int) -> int:
    """Test build: the tcgen05 backward producer of ``kernel`` (0: dk / dv, 1:
    dq) never loads its step ``step`` (-1: off)."""
    return int(load_test_library().relattn_test_backward_skip_step(int(kernel), int(step)))


def relattn_test_band_ctas(n: int) -> int:
    """Test build: at most ``n`` CTAs for the persistent / walking launches (0: one per SM)."""
    return int(load_test_library().relattn_test_band_ctas(int(n)))


def relattn_status_string(status: int) -> str:
    return load_library().relattn_status_string(status).decode()


def relattn_decode_paged(params: RelattnParams, kv: RelattnPagedKV, stream: int = 0) -> int:
    return load_library().relattn_decode_paged(ctypes.byref(params), ctypes.byref(kv),
                                               ctypes.c_void_p(stream))


def relattn_backward(params: RelattnBwdParams, stream: int = 0) -> int:
    return load_library().relattn_backward(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_backward_workspace_size(params: RelattnBwdParams) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_backward_workspace_size(ctypes.byref(params), ctypes.byref(n))
    return st, int(n.value)


def relattn_prologue(params: RelattnPrologueParams, stream: int = 0) -> int:
    return load_library().relattn_prologue(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_version() -> str:
    return load_library().relattn_version().decode()


# ------------------------------------------------------------------ torch conveniences

def _placed(call):
    """Runs a call with its first tensor's device current and, where a stream is
    given, that stream too: what it allocates (a workspace that it gives back on
    return among it) then belongs to the stream that it launches on."""
    name = call.__code__.co_varnames[0]

    @functools.wraps(call)
    def placed(*args, stream: Optional[int] = None, **kw):
        device = (args[0] if args else kw[name]).device
        if _stream_here(device, stream) is not None:
            return call(*args, **kw)
        with _switched(device, stream):
            return call(*args, **kw)
    return placed


def make_params(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int,
                max_seqlen_k: int, alpha: float, window: int = 0, log_scale_base: float = 0.0,
                out=None, lse=None, workspace=None, num_splits: int = 0,
                total_q: Optional[int] = None, total_k: Optional[int] = None) -> RelattnParams:
    """Fill a RelattnParams from torch tensors (pointers and sizes only)."""
    def ptr(t):
        return None if t is None else t.data_ptr()
    r_dim = int(r.shape[-1]) if r is not None and r.dim() == 3 else 0
    E = int(P.shape[-1]) if P is not None and P.dim() == 2 else 0
    return RelattnParams(
        q=ptr(q), k=ptr(k), v=ptr(v), r=ptr(r), P=ptr(P),
        cu_seqlens_q=ptr(cu_seqlens_q), cu_seqlens_k=ptr(cu_seqlens_k),
        batch=int(cu_seqlens_q.numel()) - 1,
        total_q=int(q.shape[0]) if total_q is None else int(total_q),
        total_k=int(k.shape[0]) if total_k is None else int(total_k),
        max_seqlen_q=int(max_seqlen_q), max_seqlen_k=int(max_seqlen_k),
        num_heads_q=int(q.shape[1]), num_heads_kv=int(k.shape[1]), head_dim=int(q.shape[2]),
        r_dim=r_dim, rel_extent=E, window=int(window), alpha=float(alpha),
        log_scale_base=float(log_scale_base), out=ptr(out), lse=ptr(lse),
        workspace=ptr(workspace),
        workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size(),
        num_splits=int(num_splits))


def _current_stream() -> int:
    import torch
    return torch.cuda.current_stream().cuda_stream


def _outputs(q, out, lse):
    import torch
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=q.device)
    return out, lse


@_placed
def prefill(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int, max_seqlen_k: int,
            alpha: float, window: int = 0, log_scale_base: float = 0.0, out=None, lse=None,
            stream: Optional[int] = None):
    """Relative-attention prefill on device tensors; returns (out, lse[Hq, Tq])."""
    out, lse = _outputs(q, out, lse)
    prm = make_params(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                      max_seqlen_k=max_seqlen_k, alpha=alpha, window=window,
                      log_scale_base=log_scale_base, out=out, lse=lse)
    _check(relattn_prefill(prm, _current_stream() if stream is None else stream), "relattn_prefill")
    return out, lse


def decode_workspace(params: RelattnParams, device):
    import torch
    st, nbytes = relattn_decode_workspace_size(params)
    _check(st, "relattn_decode_workspace_size")
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 3) // 4, dtype=torch.float32, device=device)


@_placed
def decode(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int, max_seqlen_k: int,
           alpha: float, window: int = 0, log_scale_base: float = 0.0, num_splits: int = 0,
           out=None, lse=None, workspace=None, stream: Optional[int] = None):
    """Split-KV decode (<= 16 query rows per sequence); returns (out, lse[Hq, Tq])."""
    out, lse = _outputs(q, out, lse)
    prm = make_params(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                      max_seqlen_k=max_seqlen_k, alpha=alpha, window=window,
                      log_scale_base=log_scale_base, out=out, lse=lse, num_splits=num_splits)
    if workspace is None:
        workspace = decode_workspace(prm, q.device)
    if workspace is not None:
        prm.workspace = workspace.data_ptr()
        prm.workspace_bytes = workspace.numel() * workspace.element_size()
    _check(relattn_decode(prm, _current_stream() if stream is None else stream), "relattn_decode")
    return out, lse


@_placed
def prologue(q, k, v, conv_k, conv_v, norm_q, norm_k, cu_seqlens_q, cu_seqlens_k, k_cache,
             v_cache, *, eps: float = 1e-6, q_out=None, conv_state_in=None,
             conv_state_out=None, total_k: Optional[int] = None, mxfp8=None, block_table=None,
             page_size: int = 0, stream: Optional[int] = None):
    """ShortConv + Q/K RMSNorm + KV-cache write for one chunk, on device tensors.

    ``conv_state_in`` / ``conv_state_out`` are ``(k_state, v_state)`` pairs of
    bf16 [batch, 3, Hkv*128] tensors, or None.  Writes ``k_cache`` / ``v_cache``
    rows in place and returns ``q_out`` (a new tensor unless given; pass
    ``q_out=q`` to normalise in place).  With ``mxfp8=(k8, v8, k_scale,
    v_scale)`` (uint8 [total_k, Hkv, 128] codes and [total_k, Hkv, 4] scales)
    the cache rows are also written as MXFP8 (relattn_prologue_mxfp8); the bf16
    caches may then be None.  With ``block_table`` int32 [batch,
    max_pages_per_seq] the caches are pools of pages of ``page_size`` keys
    (relattn_prologue_paged; bf16 only).
    """
    import torch
    if block_table is not None:
        return _prologue_paged(q, k, v, conv_k, conv_v, norm_q, norm_k, cu_seqlens_q, cu_seqlens_k, k_cache, v_cache,
                               eps, q_out, conv_state_in, conv_state_out, mxfp8, block_table, page_size, stream)
    if q_out is None:
        q_out = torch.empty_like(q)

    def ptr(t):
        return None if t is None else t.data_ptr()
    sin = conv_state_in if conv_state_in is not None else (None, None)
    sout = conv_state_out if conv_state_out is not None else (None, None)
    prm = RelattnPrologueParams(
        q=ptr(q), k=ptr(k), v=ptr(v), conv_k=ptr(conv_k), conv_v=ptr(conv_v),
        norm_q=ptr(norm_q), norm_k=ptr(norm_k), eps=float(eps),
        cu_seqlens_q=ptr(cu_seqlens_q), cu_seqlens_k=ptr(cu_seqlens_k),
        batch=int(cu_seqlens_q.numel()) - 1, total_q=int(q.shape[0]),
        total_k=int((k_cache if k_cache is not None else mxfp8[0]).shape[0]) if total_k is None else int(total_k),
        num_heads_q=int(q.shape[1]), num_heads_kv=int(k.shape[1]), head_dim=int(q.shape[2]),
        q_out=ptr(q_out), k_cache=ptr(k_cache), v_cache=ptr(v_cache),
        conv_state_in_k=ptr(sin[0]), conv_state_in_v=ptr(sin[1]),
        conv_state_out_k=ptr(sout[0]), conv_state_out_v=ptr(sout[1]))
    st = _current_stream() if stream is None else stream
    if mxfp8 is None:
        _check(relattn_prologue(prm, st), "relattn_prologue")
    else:
        mx = RelattnKvMxfp8(k=ptr(mxfp8[0]), v=ptr(mxfp8[1]), k_scale=ptr(mxfp8[2]), v_scale=ptr(mxfp8[3]))
        _check(load_library().relattn_prologue_mxfp8(ctypes.byref(prm), ctypes.byref(mx), st),
               "relattn_prologue_mxfp8")
    return q_out


def relattn_decode_mxfp8(params: RelattnParams, kv: RelattnKvMxfp8, stream: int = 0) -> int:
    return load_library().relattn_decode_mxfp8(ctypes.byref(params), ctypes.byref(kv), stream)


def relattn_quantize_mxfp8(x: int, n_blocks: int, codes: int, scales: int, stream: int = 0) -> int:
    return load_library().relattn_quantize_mxfp8(x, n_blocks, codes, scales, stream)


@_placed
def quantize_mxfp8(x, stream: Optional[int] = None):
    """MXFP8 of a contiguous bf16 CUDA tensor whose last dimension is a multiple
    of 32: (codes uint8 with x's shape, scales uint8 with the last dimension
    divided by 32)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_contiguous() or x.shape[-1] % 32:
        raise ValueError("x must be a contiguous bf16 tensor with a last dimension divisible by 32")
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty(*x.shape[:-1], x.shape[-1] // 32, dtype=torch.uint8, device=x.device)
    _check(relattn_quantize_mxfp8(x.data_ptr(), x.numel() // 32, codes.data_ptr(), scales.data_ptr(),
                                  _current_stream() if stream is None else stream),
           "relattn_quantize_mxfp8")
    return codes, scales


@_placed
def decode_mxfp8(q, k8, v8, k_scale, v_scale, r, P, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int,
                 max_seqlen_k: int, alpha: float, window: int = 0, log_scale_base: float = 0.0,
                 num_splits: int = 0, out=None, lse=None, workspace=None, stream: Optional[int] = None):
    """Split-KV decode against an MXFP8 K / V cache: k8 / v8 uint8 E4M3 codes
    [total_k, Hkv, 128], k_scale / v_scale uint8 E8M0 [total_k, Hkv, 4].
    Returns (out, lse)."""
    out, lse = _outputs(q, out, lse)
    prm = make_params(q, k8, v8, r, P, cu_seqlens_q, cu_seqlens_k,
                      max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k, alpha=alpha,
                      window=window, log_scale_base=log_scale_base, out=out, lse=lse,
                      num_splits=num_splits)
    if workspace is None:
        workspace = decode_workspace(prm, q.device)
    if workspace is not None:
        prm.workspace = workspace.data_ptr()
        prm.workspace_bytes = workspace.numel() * workspace.element_size()
    kv = RelattnKvMxfp8(k=k8.data_ptr(), v=v8.data_ptr(), k_scale=k_scale.data_ptr(),
                        v_scale=v_scale.data_ptr())
    _check(relattn_decode_mxfp8(prm, kv, _current_stream() if stream is None else stream),
           "relattn_decode_mxfp8")
    return out, lse


@_placed
def decode_paged(q, k_pool, v_pool, r, P, cu_seqlens_q, cu_seqlens_k, block_table, *,
                 page_size: int, max_seqlen_q: int, max_seqlen_k: int, alpha: float,
                 window: int = 0, log_scale_base: float = 0.0, num_splits: int = 0,
                 total_k: Optional[int] = None, out=None, lse=None, workspace=None,
                 stream: Optional[int] = None):
    """Split-KV decode against a paged KV cache: k_pool / v_pool [num_pages *
    page_size, Hkv, 128], block_table int32 [batch, max_pages_per_seq] on the
    device; cu_seqlens_k holds cumulative key counts.  ``total_k`` (their
    sum) sizes the split plan; when it is not given it is read back from
    cu_seqlens_k, which waits for the stream.  Returns (out, lse)."""
    out, lse = _outputs(q, out, lse)
    if total_k is None:
        total_k = int(cu_seqlens_k[-1].item())
    prm = make_params(q, k_pool, v_pool, r, P, cu_seqlens_q, cu_seqlens_k,
                      max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k, alpha=alpha,
                      window=window, log_scale_base=log_scale_base, out=out, lse=lse,
                      num_splits=num_splits, total_k=total_k)
    if workspace is None:
        workspace = decode_workspace(prm, q.device)
    if workspace is not None:
        prm.workspace = workspace.data_ptr()
        prm.workspace_bytes = workspace.numel() * workspace.element_size()
    kv = RelattnPagedKV(block_table=block_table.data_ptr(),
                        max_pages_per_seq=int(block_table.shape[1]), page_size=int(page_size),
                        num_pages=int(k_pool.shape[0]) // int(page_size))
    _check(relattn_decode_paged(prm, kv, _current_stream() if stream is None else stream),
           "relattn_decode_paged")
    return out, lse


def backward(q, k, v, r, P, out, lse, dout, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int,
             max_seqlen_k: int, alpha: float, window: int = 0, log_scale_base: float = 0.0,
             dq=None, dk=None, dv=None, dr=None, workspace=None, stream: Optional[int] = None, sink: int = 0):
    """Gradients of sum(dout * out) w.r.t. q, k, v and r (P frozen), from the
    forward's inputs and its saved out / lse.  Returns (dq, dk, dv, dr); dr is
    None when r has no channels.  ``sink``: the window keeps the first keys, as
    in ``extend``, which gave out and lse (relattn_backward_sinks)."""
    import torch
    _fit(sink)
    here = _stream_here(q.device, stream)
    if here is None:
        with _switched(q.device, stream):
            return backward(q, k, v, r, P, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                            max_seqlen_k=max_seqlen_k, alpha=alpha, window=window, log_scale_base=log_scale_base, dq=dq,
                            dk=dk, dv=dv, dr=dr, workspace=workspace, sink=sink)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    r_dim = int(r.shape[-1]) if r is not None and r.dim() == 3 else 0
    if dr is None and r_dim > 0:
        dr = torch.empty_like(r)
    prm = RelattnBwdParams(
        fwd=make_params(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                        max_seqlen_k=max_seqlen_k, alpha=alpha, window=window,
                        log_scale_base=log_scale_base, out=out, lse=lse),
        dout=dout.data_ptr(), dq=dq.data_ptr(), dk=dk.data_ptr(), dv=dv.data_ptr(),
        dr=None if dr is None else dr.data_ptr())
    if workspace is None:
        st, nbytes = relattn_backward_sinks_workspace_size(prm, sink) if sink else relattn_backward_workspace_size(prm)
        _check(st, "relattn_backward_workspace_size")
        workspace = torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=q.device)
    prm.workspace = workspace.data_ptr()
    prm.workspace_bytes = workspace.numel() * workspace.element_size()
    if sink:
        _check(relattn_backward_sinks(prm, sink, here), "relattn_backward_sinks")
    else:
        _check(relattn_backward(prm, here), "relattn_backward")
    return dq, dk, dv, dr


def relattn_backward_sinks(params: RelattnBwdParams, sink: int, stream: int = 0) -> int:
    return load_library().relattn_backward_sinks(ctypes.byref(params), sink, ctypes.c_void_p(stream))


def relattn_backward_sinks_workspace_size(params: RelattnBwdParams, sink: int) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_backward_sinks_workspace_size(ctypes.byref(params), sink, ctypes.byref(n))
    return st, int(n.value)


# ------------------------------------------------------------------ 4-bit cache, key weights, eviction

def relattn_store_nvfp4(params: RelattnCacheRowsParams, stream: int = 0) -> int:
    return load_library().relattn_store_nvfp4(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_load_nvfp4(params: RelattnCacheRowsParams, stream: int = 0) -> int:
    return load_library().relattn_load_nvfp4(ctypes.byref(params), ctypes.c_void_p(stream))


def _ref(x):
    return None if x is None else ctypes.byref(x)


def relattn_decode_nvfp4(params: RelattnParams, cache: RelattnKvNvfp4,
                         positions: Optional[RelattnPositions] = None,
                         pages: Optional[RelattnPagedKV] = None, stream: int = 0) -> int:
    return load_library().relattn_decode_nvfp4(ctypes.byref(params), ctypes.byref(cache),
                                               _ref(positions), _ref(pages), ctypes.c_void_p(stream))


def relattn_decode_nvfp4_workspace_size(params: RelattnParams,
                                        positions: Optional[RelattnPositions] = None) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_decode_nvfp4_workspace_size(ctypes.byref(params), _ref(positions),
                                                            ctypes.byref(n))
    return st, int(n.value)


def relattn_key_weights(params: RelattnKeyWeightsParams, stream: int = 0) -> int:
    return load_library().relattn_key_weights(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_key_weights_workspace_size(params: RelattnKeyWeightsParams) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_key_weights_workspace_size(ctypes.byref(params), ctypes.byref(n))
    return st, int(n.value)


def relattn_evict(params: RelattnEvictParams, stream: int = 0) -> int:
    return load_library().relattn_evict(ctypes.byref(params), ctypes.c_void_p(stream))


def relattn_evict_workspace_size(params: RelattnEvictParams) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_evict_workspace_size(ctypes.byref(params), ctypes.byref(n))
    return st, int(n.value)


class _KvTensors(NamedTuple):
    k: "torch.Tensor"            # noqa: F821
    v: "torch.Tensor"            # noqa: F821
    k_scale: "torch.Tensor"      # noqa: F821
    v_scale: "torch.Tensor"      # noqa: F821
    k_global: Optional["torch.Tensor"] = None   # noqa: F821
    v_global: Optional["torch.Tensor"] = None   # noqa: F821


class KvNvfp4(_KvTensors):
    """A 4-bit (NVFP4) K / V cache: code bytes k / v uint8 [rows, Hkv, 64], E4M3
    scale bytes k_scale / v_scale uint8 [rows, Hkv, 8], and optional fp32 [Hkv]
    factors (None: 1).  The tensors are checked here, and again by a call that
    finds one of them at another address (``t.data = ...``, ``t.set_(...)``)."""

    def __new__(cls, k, v, k_scale, v_scale, k_global=None, v_global=None):
        self = super().__new__(cls, k, v, k_scale, v_scale, k_global, v_global)
        self.c_struct = RelattnKvNvfp4()
        self.c_pointer = ctypes.pointer(self.c_struct)
        self._bind()
        return self

    def _bind(self) -> None:
        import torch
        k, dev = self.k, self.k.device
        _need(k.dim() == 3, "cache.k must have three dimensions")
        rows, H = (int(x) for x in k.shape[:2])
        ptr = [_tensor(t, f"cache.{n}", torch.uint8, (rows, H, w), dev)
               for n, t, w in zip(self._fields, self, (64, 64, 8, 8))]
        ptr += [None if t is None else _tensor(t, f"cache.{n}", torch.float32, (H,), dev)
                for n, t in zip(self._fields[4:], self[4:])]
        self.rows, self.num_heads_kv, self.device = rows, H, dev
        self.c_struct.__init__(*ptr, rows)
        self.data_ptrs, self.addresses = [t.data_ptr for t in self if t is not None], [x for x in ptr if x is not None]

    @classmethod
    def _make(cls, tensors):                 # (_replace makes its result through it)
        return cls(*tensors)

    def __reduce__(self):                    # copies and pickles too
        return type(self), tuple(self)


def empty_nvfp4(rows: int, num_heads_kv: int, device, k_global=None, v_global=None) -> KvNvfp4:
    """A cache of ``rows`` rows, zeroed (every value reads 0 until it is stored)."""
    import torch
    codes = [torch.zeros(rows, num_heads_kv, 64, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros(rows, num_heads_kv, 8, dtype=torch.uint8, device=device) for _ in range(2)]
    return KvNvfp4(*codes, *scales, k_global, v_global)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _fit(*sizes) -> None:
    """(ctypes would cut a larger number to its low 32 bits)"""
    if max(sizes) > 0x7fffffff or min(sizes) < -0x80000000:
        raise ValueError(f"sizes and counts must fit 32 bits: one of {sizes} does not")


def _tensor(t, name: str, dtype, shape, device) -> int:
    """Address of a contiguous tensor of this type and shape on `device`."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    _need(t.dtype == dtype, f"{name} must be {dtype}, not {t.dtype}")
    _need(t.shape == shape, f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, not {device}")


def _address(t, name: str, dtype, device) -> int:
    """Address of a contiguous tensor of this type on `device` whose shape has
    been looked at.  (These checks are most of a short call's host time: they
    format nothing and look at nothing twice.)"""
    if t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    return _tensor(t, name, dtype, t.shape, device)


def _shape(t, name: str, n: int, *want):
    """t's shape, of n dimensions whose last ones are `want`."""
    s = t.shape
    if len(s) != n or (want and s[n - len(want):] != want):
        raise ValueError(f"{name} must have {n} dimensions{f' ending in {want}' if want else ''}, not shape {tuple(s)}")
    return s


def _lengths(cu_q, cu_k, name_q: str, name_k: str, device):
    """(batch, addresses) of two cu_seqlens tensors."""
    import torch
    n, int32 = cu_q.numel(), torch.int32
    if n < 1:
        raise ValueError(f"{name_q} needs at least one entry")
    if cu_q.dim() == 1 and cu_k.dim() == 1 and cu_k.numel() == n:
        return n - 1, _address(cu_q, name_q, int32, device), _address(cu_k, name_k, int32, device)
    return n - 1, _tensor(cu_q, name_q, int32, (n,), device), _tensor(cu_k, name_k, int32, (n,), device)


def _cache(cache: KvNvfp4, device) -> None:
    if not isinstance(cache, KvNvfp4):
        raise ValueError("cache must be a KvNvfp4")
    if [f() for f in cache.data_ptrs] != cache.addresses:
        cache._bind()
    if cache.device != device:
        raise ValueError(f"the cache is on {cache.device}, not {device}")


def _pages(block_table, page_size: int, rows: int, device, batch: int) -> Optional[RelattnPagedKV]:
    import torch
    if block_table is None:
        return None
    _need(page_size > 0 and rows % page_size == 0, "rows must be a multiple of page_size")
    seqs, slots = _shape(block_table, "block_table", 2)
    if seqs != batch:
        _tensor(block_table, "block_table", torch.int32, (batch, slots), device)
    return RelattnPagedKV(_address(block_table, "block_table", torch.int32, device), slots, page_size,
                          rows // page_size)


def _positions(key_pos, q_pos, num_heads_kv: int, rows: int, batch: int, device) -> Optional[RelattnPositions]:
    import torch
    if key_pos is None and q_pos is None:
        return None
    _need(key_pos is not None and q_pos is not None, "key_pos and q_pos go together")
    return RelattnPositions(_tensor(key_pos, "key_pos", torch.int32, (num_heads_kv, rows), device),
                            _tensor(q_pos, "q_pos", torch.int32, (batch,), device))


def _stream_here(device, stream: Optional[int]) -> Optional[int]:
    """The current stream of `device` when a call may launch on it as things
    are: no stream given and the device current.  Else None (see _switched)."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {device}")
    index = device.index                     # (a tensor on it: CUDA is initialised)
    if stream is not None or index != torch._C._cuda_getDevice():
        return None
    return torch._C._cuda_getCurrentRawStream(index)


@contextlib.contextmanager
def _switched(device, stream: Optional[int]):
    """With the tensors' device current and, where a stream is given, that stream
    too, so that what the block allocates belongs to the stream it launches on."""
    import torch
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream
                                   else torch.cuda.default_stream(device)):
                yield


def _queries(q, r, P, num_heads_kv: int, device):
    """(total_q, Hq, r_dim, E) and addresses of q [Tq, Hq, 128], r [Tq, Hq,
    r_dim], P [r_dim, E]."""
    import torch
    bf16 = torch.bfloat16
    Tq, Hq, _ = _shape(q, "q", 3, HEAD_DIM)
    if num_heads_kv <= 0 or Hq % num_heads_kv:
        raise ValueError(f"num_heads_q = {Hq} must be a multiple of num_heads_kv = {num_heads_kv}")
    qp = _address(q, "q", bf16, device)
    if r is None or P is None:
        _need(r is None and P is None, "r and P go together")
        return Tq, Hq, 0, 0, qp, None, None
    rs, Ps = r.shape, P.shape
    if len(rs) == 3 and len(Ps) == 2 and rs[0] == Tq and rs[1] == Hq and Ps[0] == rs[2]:
        return Tq, Hq, rs[2], Ps[1], qp, _address(r, "r", bf16, device), _address(P, "P", bf16, device)
    rd, E = _shape(r, "r", 3)[2], _shape(P, "P", 2)[1]
    _tensor(r, "r", bf16, (Tq, Hq, rd), device)
    _tensor(P, "P", bf16, (rd, E), device)
    raise AssertionError("one of them was refused")


def _cache_rows(k, v, cu_q, cu_k, cache, block_table, page_size):
    import torch
    dev, bf16 = k.device, torch.bfloat16
    _cache(cache, dev)
    H = cache.num_heads_kv
    batch, cq, ck = _lengths(cu_q, cu_k, "cu_seqlens_q", "cu_seqlens_k", dev)
    pages = _pages(block_table, page_size, cache.rows, dev, batch)
    shape = (k.shape[0], H, HEAD_DIM)
    return RelattnCacheRowsParams(
        _tensor(k, "k", bf16, shape, dev), _tensor(v, "v", bf16, shape, dev), cq, ck, batch,
        shape[0], H, HEAD_DIM, cache.c_pointer, None if pages is None else ctypes.pointer(pages))


def store_nvfp4(k, v, cu_seqlens_q, cu_seqlens_k, cache: KvNvfp4, *, block_table=None, page_size: int = 0,
                stream: Optional[int] = None) -> None:
    """Quantises the chunk's rows k / v bf16 [total_q, Hkv, 128] (the last rows
    of every sequence) into the 4-bit cache; with ``block_table`` int32 [batch,
    max_pages_per_seq] the cache's rows are pages of ``page_size`` keys."""
    prm = _cache_rows(k, v, cu_seqlens_q, cu_seqlens_k, cache, block_table, page_size)
    st = _stream_here(k.device, stream)
    if st is None:
        with _switched(k.device, stream):
            return store_nvfp4(k, v, cu_seqlens_q, cu_seqlens_k, cache, block_table=block_table, page_size=page_size)
    _check((_lib or load_library()).relattn_store_nvfp4(ctypes.byref(prm), st), "relattn_store_nvfp4")


def load_nvfp4(cache: KvNvfp4, cu_seqlens_q, cu_seqlens_k, *, total_q: int, block_table=None, page_size: int = 0,
               k=None, v=None, stream: Optional[int] = None):
    """The last cu_seqlens_q rows of every sequence as bf16 (k, v) [total_q, Hkv,
    128] (pass cu_seqlens_k twice for all of them)."""
    import torch
    if not isinstance(cache, KvNvfp4):
        raise ValueError("cache must be a KvNvfp4")
    st = _stream_here(cache.device, stream)
    if st is None:
        with _switched(cache.device, stream):
            return load_nvfp4(cache, cu_seqlens_q, cu_seqlens_k, total_q=total_q, block_table=block_table,
                              page_size=page_size, k=k, v=v)
    shape = (int(total_q), cache.num_heads_kv, HEAD_DIM)
    k = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if v is None else v
    _need(k.shape[0] == total_q, "k must have total_q rows")
    prm = _cache_rows(k, v, cu_seqlens_q, cu_seqlens_k, cache, block_table, page_size)
    _check((_lib or load_library()).relattn_load_nvfp4(ctypes.byref(prm), st), "relattn_load_nvfp4")
    return k, v


def _total_k(total_k: Optional[int], block_table, cu_k, rows: int) -> int:
    if total_k is not None:
        return int(total_k)
    return int(cu_k[-1].item()) if block_table is not None else rows


def _workspace(nbytes: int, workspace, device):
    """(tensor kept alive, pointer, bytes) of a workspace of at least nbytes."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        import torch
        words = (nbytes + 3) // 4
        workspace = torch.empty(words, dtype=torch.float32, device=device)
        return workspace, workspace.data_ptr(), 4 * words
    _need(workspace.device == device, "workspace is on another device")
    _need(workspace.is_contiguous(), "workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def decode_nvfp4(q, cache: KvNvfp4, r, P, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int, max_seqlen_k: int,
                 alpha: float, window: int = 0, log_scale_base: float = 0.0, key_pos=None, q_pos=None,
                 block_table=None, page_size: int = 0, total_k: Optional[int] = None, num_splits: int = 0,
                 out=None, lse=None, workspace=None, stream: Optional[int] = None):
    """Split-KV decode against the 4-bit cache (contiguous, or paged with
    ``block_table``); ``key_pos`` int32 [Hkv, rows] and ``q_pos`` int32 [batch]
    give positions that are not the row indices.  ``total_k`` (the sum of the
    key counts) sizes the split plan; without it a paged call reads it back
    from cu_seqlens_k, which waits for the stream.  Returns (out, lse)."""
    import torch
    dev = q.device
    st = _stream_here(dev, stream)
    if st is None:
        with _switched(dev, stream):
            return decode_nvfp4(q, cache, r, P, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                                max_seqlen_k=max_seqlen_k, alpha=alpha, window=window, log_scale_base=log_scale_base,
                                key_pos=key_pos, q_pos=q_pos, block_table=block_table, page_size=page_size,
                                total_k=total_k, num_splits=num_splits, out=out, lse=lse, workspace=workspace)
    _cache(cache, dev)
    H, rows = cache.num_heads_kv, cache.rows
    Tq, Hq, rd, E, qp, rp, Pp = _queries(q, r, P, H, dev)
    batch, cq, ck = _lengths(cu_seqlens_q, cu_seqlens_k, "cu_seqlens_q", "cu_seqlens_k", dev)
    pages = _pages(block_table, page_size, rows, dev, batch)
    pos = _positions(key_pos, q_pos, H, rows, batch, dev)
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _tensor(out, "out", torch.bfloat16, (Tq, Hq, HEAD_DIM), dev)
    if lse is None:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _tensor(lse, "lse", torch.float32, (Hq, Tq), dev)
    total_k = _total_k(total_k, block_table, cu_seqlens_k, rows)
    _fit(total_k, max_seqlen_q, max_seqlen_k, window, num_splits)
    prm = RelattnParams(
        qp, None, None, rp, Pp, cq, ck, batch, Tq, total_k,
        max_seqlen_q, max_seqlen_k, Hq, H, HEAD_DIM, rd, E, window, alpha, log_scale_base, op, lp, None, 0, num_splits)
    lib, need = _lib or load_library(), ctypes.c_size_t()
    ref, pos = ctypes.byref(prm), _ref(pos)
    _check(lib.relattn_decode_nvfp4_workspace_size(ref, pos, ctypes.byref(need)), "relattn_decode_nvfp4_workspace_size")
    keep, prm.workspace, prm.workspace_bytes = _workspace(need.value, workspace, dev)
    _check(lib.relattn_decode_nvfp4(ref, cache.c_pointer, pos, _ref(pages), st), "relattn_decode_nvfp4")
    return out, lse


def key_weights(q, k, r, P, lse, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int, max_seqlen_k: int, alpha: float,
                window: int = 0, log_scale_base: float = 0.0, weights_in=None, decay: float = 1.0, key_pos=None,
                q_pos=None, block_table=None, page_size: int = 0, total_k: Optional[int] = None, out=None,
                workspace=None, stream: Optional[int] = None):
    """The attention weight each cached key receives from the rows of q, whose
    lse [Hq, total_q] the forward or decode returned: fp32 [Hkv, rows],
    decay * weights_in + the rows' weights (the newest rows' keys start from
    0).  ``k`` is a bf16 tensor [rows, Hkv, 128] or a KvNvfp4 cache.  ``out`` may be
    ``weights_in``; a new one is zeroed first, since rows that hold no key are
    not written."""
    import torch
    dev = q.device
    st = _stream_here(dev, stream)
    if st is None:
        with _switched(dev, stream):
            return key_weights(q, k, r, P, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                               max_seqlen_k=max_seqlen_k, alpha=alpha, window=window, log_scale_base=log_scale_base,
                               weights_in=weights_in, decay=decay, key_pos=key_pos, q_pos=q_pos,
                               block_table=block_table, page_size=page_size, total_k=total_k, out=out,
                               workspace=workspace)
    fp4 = isinstance(k, KvNvfp4)
    if fp4:
        _cache(k, dev)
        rows, H = k.rows, k.num_heads_kv
    else:
        rows, H, _ = _shape(k, "k", 3, HEAD_DIM)
        kp = _address(k, "k", torch.bfloat16, dev)
    Tq, Hq, rd, E, qp, rp, Pp = _queries(q, r, P, H, dev)
    batch, cq, ck = _lengths(cu_seqlens_q, cu_seqlens_k, "cu_seqlens_q", "cu_seqlens_k", dev)
    pages = _pages(block_table, page_size, rows, dev, batch)
    pos = _positions(key_pos, q_pos, H, rows, batch, dev)
    w_in = None if weights_in is None else _tensor(weights_in, "weights_in", torch.float32, (H, rows), dev)
    if out is None:
        out = torch.zeros(H, rows, dtype=torch.float32, device=dev)
    w_out = w_in if out is weights_in else _tensor(out, "out", torch.float32, (H, rows), dev)
    total_k = _total_k(total_k, block_table, cu_seqlens_k, rows)
    _fit(total_k, max_seqlen_q, max_seqlen_k, window)
    if not fp4 and block_table is None:
        _need(total_k == rows, "a contiguous k has total_k rows")
    fwd = RelattnParams(
        qp, None if fp4 else kp, None, rp, Pp, cq, ck, batch, Tq, total_k, max_seqlen_q, max_seqlen_k, Hq, H,
        HEAD_DIM, rd, E, window, alpha, log_scale_base, None,
        _tensor(lse, "lse", torch.float32, (Hq, Tq), dev), None, 0, 0)
    prm = RelattnKeyWeightsParams(
        fwd, k.c_pointer if fp4 else None, None if pos is None else ctypes.pointer(pos),
        None if pages is None else ctypes.pointer(pages), w_in, w_out, decay)
    lib, need, ref = _lib or load_library(), ctypes.c_size_t(), ctypes.byref(prm)
    _check(lib.relattn_key_weights_workspace_size(ref, ctypes.byref(need)), "relattn_key_weights_workspace_size")
    keep, prm.workspace, prm.workspace_bytes = _workspace(need.value, workspace, dev)
    _check(lib.relattn_key_weights(ref, st), "relattn_key_weights")
    return out


_NO_PLANES = RelattnPlane * MAX_PLANES


def evict(planes, dst_planes, weights, cu_seqlens_k, cu_seqlens_keep, *, max_seqlen_k: int, recent: int, sink: int = 0,
          total_keep: int, total_k: Optional[int] = None, key_pos=None, block_table=None, page_size: int = 0,
          block_table_keep=None, page_size_keep: int = 0, key_pos_out=None, weights_out=None, workspace=None,
          rows_keep: Optional[int] = None, stream: Optional[int] = None):
    """Keeps, per sequence and kv head, the newest ``recent`` keys, the first
    ``sink`` and the heaviest of the rest (``weights`` fp32 [Hkv, rows]) -- in
    all cu_seqlens_keep[b+1] - cu_seqlens_keep[b] of sequence b -- and copies
    their rows of every plane [rows, Hkv, ...] into ``dst_planes``, in order of
    index.  Returns (key_pos [Hkv, rows_keep] int32, weights [Hkv, rows_keep])
    of the new cache.  ``rows_keep``, the rows of the new cache, is that of
    ``dst_planes``; without planes it may be given (a paged destination needs
    it) and is else ``total_keep``."""
    import torch
    dev = weights.device
    st = _stream_here(dev, stream)
    if st is None:
        with _switched(dev, stream):
            return evict(planes, dst_planes, weights, cu_seqlens_k, cu_seqlens_keep, max_seqlen_k=max_seqlen_k,
                         recent=recent, sink=sink, total_keep=total_keep, total_k=total_k, key_pos=key_pos,
                         block_table=block_table, page_size=page_size, block_table_keep=block_table_keep,
                         page_size_keep=page_size_keep, key_pos_out=key_pos_out, weights_out=weights_out,
                         workspace=workspace, rows_keep=rows_keep)
    n = len(planes)
    if not n == len(dst_planes) <= MAX_PLANES:
        raise ValueError(f"as many dst_planes as planes, at most {MAX_PLANES}")
    H, rows = _shape(weights, "weights", 2)
    batch, ck, ckeep = _lengths(cu_seqlens_k, cu_seqlens_keep, "cu_seqlens_k", "cu_seqlens_keep", dev)
    if n:
        _need(rows_keep is None or rows_keep == dst_planes[0].shape[0], "rows_keep is not that of dst_planes")
        rows_keep = dst_planes[0].shape[0]
    else:
        rows_keep = int(total_keep if rows_keep is None else rows_keep)
    wp = _tensor(weights, "weights", torch.float32, (H, rows), dev)
    table = _NO_PLANES()
    for i in range(n):
        a, b = planes[i], dst_planes[i]
        sa, sb = a.shape, b.shape
        if len(sa) < 2 or sa[0] != rows or sa[1] != H or len(sb) < 2 or sb[0] != rows_keep or sb[1:] != sa[1:]:
            raise ValueError(f"plane {i} must be [rows, Hkv, ...] and its destination [rows_keep, Hkv, ...]")
        dtype = a.dtype
        if not (b.dtype is dtype and a.device == dev and b.device == dev and a.is_contiguous() and b.is_contiguous()):
            _tensor(a, f"plane {i}", dtype, sa, dev)
            _tensor(b, f"destination {i}", dtype, sb, dev)
        table[i] = (a.data_ptr(), b.data_ptr(), a.element_size() * sa[2:].numel())
    pages = _pages(block_table, page_size, rows, dev, batch)
    pages_keep = _pages(block_table_keep, page_size_keep, rows_keep, dev, batch)
    new_pos, new_w = key_pos_out is None, weights_out is None
    if new_pos:                                  # (both new: cleared by the call)
        key_pos_out = (torch.empty(H, rows_keep, dtype=torch.int32, device=dev) if new_w
                       else torch.full((H, rows_keep), -1, dtype=torch.int32, device=dev))
    if new_w:
        weights_out = (torch.empty if new_pos else torch.zeros)(H, rows_keep, dtype=torch.float32, device=dev)
    total_k = _total_k(total_k, block_table, cu_seqlens_k, rows)
    recent, sink = min(recent, 0x7fffffff), min(sink, 0x7fffffff)      # (no sequence has more keys)
    _fit(total_k, total_keep, max_seqlen_k, recent, sink)
    prm = RelattnEvictParams(
        wp, ck, ckeep, None if key_pos is None else _tensor(key_pos, "key_pos", torch.int32, (H, rows), dev), batch,
        total_k, total_keep, max_seqlen_k, H, sink, recent, rows, rows_keep,
        None if pages is None else ctypes.pointer(pages), None if pages_keep is None else ctypes.pointer(pages_keep),
        n, table, weights_out.data_ptr() if new_w else _tensor(weights_out, "weights_out", torch.float32, (H, rows_keep), dev),
        key_pos_out.data_ptr() if new_pos else _tensor(key_pos_out, "key_pos_out", torch.int32, (H, rows_keep), dev),
        None, 0, new_pos and new_w)
    lib, need, ref = _lib or load_library(), ctypes.c_size_t(), ctypes.byref(prm)
    _check(lib.relattn_evict_workspace_size(ref, ctypes.byref(need)), "relattn_evict_workspace_size")
    keep, prm.workspace, prm.workspace_bytes = _workspace(need.value, workspace, dev)
    _check(lib.relattn_evict(ref, st), "relattn_evict")
    return key_pos_out, weights_out


# ------------------------------------------------------------------ new tokens over a cache, windows with sinks

def relattn_extend(params: RelattnParams, pages: Optional[RelattnPagedKV] = None, sink: int = 0, stream: int = 0) -> int:
    return load_library().relattn_extend(ctypes.byref(params), _ref(pages), sink, ctypes.c_void_p(stream))


def relattn_extend_workspace_size(params: RelattnParams, pages: Optional[RelattnPagedKV] = None,
                                  sink: int = 0) -> Tuple[int, int]:
    n = ctypes.c_size_t(0)
    st = load_library().relattn_extend_workspace_size(ctypes.byref(params), _ref(pages), sink, ctypes.byref(n))
    return st, int(n.value)


def relattn_prologue_paged(params: RelattnPrologueParams, pages: RelattnPagedKV, stream: int = 0) -> int:
    return load_library().relattn_prologue_paged(ctypes.byref(params), ctypes.byref(pages), ctypes.c_void_p(stream))


def extend(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, *, max_seqlen_q: int, max_seqlen_k: int, alpha: float,
           window: int = 0, sink: int = 0, log_scale_base: float = 0.0, block_table=None, page_size: int = 0,
           total_k: Optional[int] = None, num_splits: int = 0, out=None, lse=None, workspace=None,
           stream: Optional[int] = None):
    """Attention of new tokens -- one, a chunk, a whole prompt -- over the cache
    that holds them: k / v bf16 [rows, Hkv, 128], contiguous, or with
    ``block_table`` int32 [batch, max_pages_per_seq] a pool of pages of
    ``page_size`` keys (a multiple of 16).  A ``window`` keeps the first
    ``sink`` keys.  ``total_k`` (the sum of the key counts) sizes the work
    split; without it a paged call reads it back from cu_seqlens_k, which waits
    for the stream.  ``num_splits``: 0 chooses; n > 0 cuts a row's keys into at
    most n partials.  Returns (out, lse)."""
    import torch
    dev = q.device
    st = _stream_here(dev, stream)
    if st is None:
        with _switched(dev, stream):
            return extend(q, k, v, r, P, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                          max_seqlen_k=max_seqlen_k, alpha=alpha, window=window, sink=sink, log_scale_base=log_scale_base,
                          block_table=block_table, page_size=page_size, total_k=total_k, num_splits=num_splits, out=out,
                          lse=lse, workspace=workspace)
    rows, H, _ = _shape(k, "k", 3, HEAD_DIM)
    kp, vp = _address(k, "k", torch.bfloat16, dev), _tensor(v, "v", torch.bfloat16, k.shape, dev)
    Tq, Hq, rd, E, qp, rp, Pp = _queries(q, r, P, H, dev)
    batch, cq, ck = _lengths(cu_seqlens_q, cu_seqlens_k, "cu_seqlens_q", "cu_seqlens_k", dev)
    pages = _pages(block_table, page_size, rows, dev, batch)
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _tensor(out, "out", torch.bfloat16, (Tq, Hq, HEAD_DIM), dev)
    if lse is None:
        lse = torch.empty(Hq, Tq, dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _tensor(lse, "lse", torch.float32, (Hq, Tq), dev)
    if block_table is None:
        _need(total_k is None or total_k == rows, "a contiguous k has total_k rows")
    total_k = _total_k(total_k, block_table, cu_seqlens_k, rows)
    _fit(total_k, max_seqlen_q, max_seqlen_k, window, sink, num_splits)
    prm = RelattnParams(
        qp, kp, vp, rp, Pp, cq, ck, batch, Tq, total_k, max_seqlen_q, max_seqlen_k, Hq, H, HEAD_DIM, rd, E, window,
        alpha, log_scale_base, op, lp, None, 0, num_splits)
    lib, need = _lib or load_library(), ctypes.c_size_t()
    ref, pages = ctypes.byref(prm), _ref(pages)
    _check(lib.relattn_extend_workspace_size(ref, pages, sink, ctypes.byref(need)), "relattn_extend_workspace_size")
    keep, prm.workspace, prm.workspace_bytes = _workspace(need.value, workspace, dev)
    _check(lib.relattn_extend(ref, pages, sink, st), "relattn_extend")
    return out, lse


def _prologue_paged(q, k, v, conv_k, conv_v, norm_q, norm_k, cu_seqlens_q, cu_seqlens_k, k_pool, v_pool, eps, q_out,
                    conv_state_in, conv_state_out, mxfp8, block_table, page_size, stream):
    import torch
    _need(mxfp8 is None, "a paged cache is bf16 only")
    dev, bf16, f32 = q.device, torch.bfloat16, torch.float32
    st = _stream_here(dev, stream)
    if st is None:
        with _switched(dev, stream):
            return _prologue_paged(q, k, v, conv_k, conv_v, norm_q, norm_k, cu_seqlens_q, cu_seqlens_k, k_pool, v_pool, eps,
                                   q_out, conv_state_in, conv_state_out, mxfp8, block_table, page_size, None)
    Tq, Hq, _ = _shape(q, "q", 3, HEAD_DIM)
    rows, H, _ = pool = _shape(k_pool, "k_cache", 3, HEAD_DIM)
    C = H * HEAD_DIM
    new, taps, gain = (Tq, H, HEAD_DIM), (C, 4), (HEAD_DIM,)
    batch, cq, ck = _lengths(cu_seqlens_q, cu_seqlens_k, "cu_seqlens_q", "cu_seqlens_k", dev)
    pages = _pages(block_table, page_size, rows, dev, batch)
    qp = _address(q, "q", bf16, dev)
    if q_out is None:
        q_out = torch.empty_like(q)
        op = q_out.data_ptr()
    else:
        op = _tensor(q_out, "q_out", bf16, (Tq, Hq, HEAD_DIM), dev)

    def state(pair, name):
        if pair is None:
            return None, None
        a, b = pair
        s = (batch, 3, C)
        return None if a is None else _tensor(a, name, bf16, s, dev), None if b is None else _tensor(b, name, bf16, s, dev)
    prm = RelattnPrologueParams(
        qp, _tensor(k, "k", bf16, new, dev), _tensor(v, "v", bf16, new, dev), _tensor(conv_k, "conv_k", f32, taps, dev),
        _tensor(conv_v, "conv_v", f32, taps, dev), _tensor(norm_q, "norm_q", f32, gain, dev),
        _tensor(norm_k, "norm_k", f32, gain, dev), eps, cq, ck, batch, Tq, 0, Hq, H, HEAD_DIM, op,
        _address(k_pool, "k_cache", bf16, dev), _tensor(v_pool, "v_cache", bf16, pool, dev),
        *state(conv_state_in, "conv_state_in"), *state(conv_state_out, "conv_state_out"))
    _check((_lib or load_library()).relattn_prologue_paged(ctypes.byref(prm), ctypes.byref(pages), st),
           "relattn_prologue_paged")
    return q_out
