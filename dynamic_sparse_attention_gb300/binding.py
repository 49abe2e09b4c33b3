"""ctypes binding of libdsa.so: argument marshalling only.

Every step of the hot path runs in the CUDA kernels behind the C ABI
(``include/dsa.h``).  This module turns torch CUDA tensors into device
pointers, allocates the scratch workspace the library asks for (unless the
caller passes one) and forwards the current torch stream.  There is no CPU
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

from . import _build

MAX_STAGES = 8
BF16, F32, BF16_FP8KV = 0, 1, 2   # dsa_dtype

_c_int = ctypes.c_int
_vp = ctypes.c_void_p


class DecodeShape(ctypes.Structure):
    _fields_ = [("B", _c_int), ("T_max", _c_int), ("T_q", _c_int), ("H_q", _c_int),
                ("H_kv", _c_int), ("D", _c_int), ("dtype", _c_int)]


class HipCfg(ctypes.Structure):
    _fields_ = [("n_stages", _c_int), ("chunk", _c_int * MAX_STAGES),
                ("keep", _c_int * MAX_STAGES), ("n_sink", _c_int), ("n_stream", _c_int)]


class HipDebug(ctypes.Structure):
    _fields_ = [("stage_idx", _vp * MAX_STAGES), ("stage_cnt", _vp * MAX_STAGES),
                ("chunk_score", _vp * MAX_STAGES), ("rep", _vp * MAX_STAGES),
                ("rep_score", _vp * MAX_STAGES)]


class PrefillShape(ctypes.Structure):
    _fields_ = [("B", _c_int), ("S", _c_int), ("H_q", _c_int), ("H_kv", _c_int), ("D", _c_int)]


class VsCfg(ctypes.Structure):
    _fields_ = [("last_q", _c_int), ("n_vertical", _c_int), ("n_slash", _c_int), ("block", _c_int)]


class VsDebug(ctypes.Structure):
    _fields_ = [("vsum", _vp), ("ssum", _vp)]


class MixedCfg(ctypes.Structure):
    _fields_ = [("head_pattern", _vp), ("vs", VsCfg), ("n_global", _c_int), ("n_local", _c_int),
                ("k_b", _c_int)]


PATTERN_VERTICAL_SLASH, PATTERN_A_SHAPE, PATTERN_BLOCK_SPARSE = 0, 1, 2
_PATTERN_NAMES = {"vertical_slash": 0, "vs": 0, "a_shape": 1, "block_sparse": 2}


class BsDebug(ctypes.Structure):
    _fields_ = [("q_pool", _vp), ("k_pool", _vp), ("scores", _vp)]


class PagedShape(ctypes.Structure):
    _fields_ = [("B", _c_int), ("n_tok", _c_int), ("max_pages", _c_int), ("n_pages", _c_int),
                ("page_size", _c_int), ("H_q", _c_int), ("H_kv", _c_int), ("D", _c_int),
                ("dtype", _c_int)]


class RopeCfg(ctypes.Structure):
    _fields_ = [("q_weight", _vp), ("k_weight", _vp), ("weight_f32", _c_int), ("eps", ctypes.c_float),
                ("inv_freq", _vp), ("rot", _c_int), ("interleaved", _c_int), ("rope_scale", ctypes.c_float)]


class PageSelectCfg(ctypes.Structure):
    _fields_ = [("keep", _c_int), ("n_sink", _c_int), ("n_local", _c_int), ("q_block", _c_int)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", _c_int), ("total_ms", ctypes.c_double)]


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


_lib = None

# name -> (restype, argtypes)
_SIGNATURES = {
    "dsa_version": (_c_int, []),
    "dsa_last_error": (ctypes.c_char_p, []),
    "dsa_strerror": (ctypes.c_char_p, [_c_int]),
    "dsa_hip_max_chunks": (_c_int, [_vp, _vp, _c_int, ctypes.POINTER(_c_int)]),
    "hip_select_workspace": (_c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_size_t)]),
    "hip_select": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "hip_select_cached": (_c_int, [_vp, _vp, _vp, _vp, _vp, ctypes.c_uint32, _vp, _vp, _vp, _vp,
                                   ctypes.c_size_t, _vp]),
    "sparse_attn_decode_workspace": (_c_int, [_vp, _c_int, _c_int, _c_int,
                                              ctypes.POINTER(ctypes.c_size_t)]),
    "sparse_attn_decode": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                    ctypes.c_float, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "vs_index_build_workspace": (_c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_size_t)]),
    "vs_index_build": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                ctypes.c_size_t, _vp]),
    "ashape_index_build": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp]),
    "block_sparse_index_build_workspace": (_c_int, [_vp, _c_int, ctypes.POINTER(ctypes.c_size_t)]),
    "block_sparse_index_build": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                          _vp, _vp, ctypes.c_size_t, _vp]),
    "mixed_index_build_workspace": (_c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_size_t)]),
    "mixed_index_build": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                   _vp]),
    "dsa_hip_prefill_max_chunks": (_c_int, [_vp, _vp, _c_int, ctypes.POINTER(_c_int)]),
    "hip_prefill_select_workspace": (_c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_size_t)]),
    "hip_prefill_select": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "hip_prefill_lists": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp]),
    "sparse_attn_prefill": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                     _vp, ctypes.c_float, _vp, _vp, _vp]),
    "sparse_attn_decode_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                            ctypes.c_float, _vp, _vp, _vp, _vp]),
    "kv_cache_write": (_c_int, [_vp, _vp, ctypes.c_longlong, ctypes.c_longlong, _vp, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp, _vp]),
    "kv_cache_read": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp]),
    "paged_attn_workspace": (_c_int, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    "paged_attn": (_c_int, [_vp, ctypes.c_longlong, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int,
                            _c_int, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "paged_attn_lists": (_c_int, [_vp, ctypes.c_longlong, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int,
                                  _c_int, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "kv_cache_write_rope": (_c_int, [_vp, ctypes.c_longlong, _vp, ctypes.c_longlong, _vp, ctypes.c_longlong,
                                     _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_longlong, _vp, _vp, _vp, _vp, _vp]),
    "page_digest_update": (_c_int, [_vp] * 9),
    "page_select_sizes": (_c_int, [_vp, _vp, ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "page_select": (_c_int, [_vp, ctypes.c_longlong] + [_vp] * 12),
    "kv_pages_copy": (_c_int, [_vp, _vp, _c_int] + [_vp] * 8),
    "dsa_device_error": (_c_int, [ctypes.POINTER(_c_int)]),
    "dsa_set_wait_limit": (_c_int, [ctypes.c_ulonglong]),
    "dsa_profile_enable": (_c_int, [_c_int]),
    "dsa_profile_collect": (_c_int, [_vp, _c_int, ctypes.POINTER(_c_int)]),
}


def device_error() -> int:
    """Read and clear the library's device error words: 0 = none; bit 0 / bit 1: a
    prefill-attention / vertical-slash-estimate CTA gave up a wait; bit 2 (checked
    build): a kernel met out-of-range device-side input; bit 3 / bit 4: a paged-attention /
    page-selection CTA gave up a wait."""
    lib = load()
    c = _c_int()
    st = lib.dsa_device_error(ctypes.byref(c))
    if st == -6:   # DSA_ERR_DEVICE_CHECK: the code says what was met
        return c.value
    _check("dsa_device_error", st)
    return c.value


def set_wait_limit(ns: int = 0) -> None:
    """Limit of the tensor-core kernels' bounded waits in nanoseconds (0: the default)."""
    lib = load()
    _check("dsa_set_wait_limit", lib.dsa_set_wait_limit(ctypes.c_ulonglong(ns)))


def profile_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with CUDA events on its stream."""
    load().dsa_profile_enable(1 if on else 0)


def profile_collect() -> dict:
    """Wait for the recorded events; {kernel name: (launches, total ms)}, then clear."""
    lib = load()
    buf = (KernelStat * 64)()
    n = _c_int()
    _check("dsa_profile_collect", lib.dsa_profile_collect(buf, 64, ctypes.byref(n)))
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(min(n.value, 64))}


def library_path() -> str:
    """Path of the library this process loads (the checked build with DSA_CHECKED=1)."""
    return _build.LIB_CHECKED if os.environ.get("DSA_CHECKED") == "1" else _build.LIB


def load(build_if_missing: bool = False):
    """Load libdsa.so (building it first if asked and absent).  With DSA_CHECKED=1 in
    the environment at the first call, the checked build libdsa_checked.so instead (the
    same kernels with device-side input checks compiled in)."""
    global _lib
    if _lib is not None:
        return _lib
    checked = os.environ.get("DSA_CHECKED") == "1"
    path = _build.LIB_CHECKED if checked else _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise ImportError(f"{os.path.basename(path)} not built ({path}); run __graft_entry__.build()")
        _build.build(checked=checked)
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name, None)
        if fn is None:
            continue  # reported by exported_symbols(); calling it raises AttributeError
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def exported_symbols() -> dict:
    """Which C entry points of the binding the loaded library exports."""
    lib = load()
    return {name: hasattr(lib, name) for name in _SIGNATURES}


def _check(fn: str, status: int):
    if status != 0:
        msg = _lib.dsa_last_error().decode(errors="replace")
        raise DsaError(fn, status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _workspace(nbytes: int, device, ws):
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace too small: {nbytes} bytes needed")
        return ws
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------------------- decode

@dataclass
class HipConfig:
    chunk: tuple
    keep: tuple
    n_sink: int
    n_stream: int

    def c(self) -> HipCfg:
        cfg = HipCfg()
        cfg.n_stages = len(self.chunk)
        for i, (c, k) in enumerate(zip(self.chunk, self.keep)):
            cfg.chunk[i] = int(c)
            cfg.keep[i] = int(k)
        cfg.n_sink = int(self.n_sink)
        cfg.n_stream = int(self.n_stream)
        return cfg


def _is_fp8(t: torch.Tensor) -> bool:
    return t.dtype == torch.uint8 or t.dtype == getattr(torch, "float8_e4m3fn", None)


def decode_shape(q: torch.Tensor, k: torch.Tensor) -> DecodeShape:
    """q bf16 / fp32 with k of the same type, or q bf16 with k FP8 E4M3 (a uint8 or
    float8_e4m3fn tensor of codes)."""
    B, T_q, H_q, D = q.shape
    T_max, H_kv = k.shape[1], k.shape[2]
    if _is_fp8(k):
        if q.dtype != torch.bfloat16:
            raise TypeError("FP8 keys and values need a bfloat16 query")
        return DecodeShape(B, T_max, T_q, H_q, H_kv, D, BF16_FP8KV)
    if k.dtype != q.dtype:
        raise TypeError(f"k ({k.dtype}) must have the type of q ({q.dtype})")
    return DecodeShape(B, T_max, T_q, H_q, H_kv, D, _dtype_code(q))


def hip_select_workspace_bytes(q, k, cfg: HipConfig) -> int:
    lib = load()
    n = ctypes.c_size_t()
    shape, c = decode_shape(q, k), cfg.c()
    _check("hip_select_workspace", lib.hip_select_workspace(ctypes.byref(shape), ctypes.byref(c),
                                                             ctypes.byref(n)))
    return n.value


def hip_max_chunks(q, k, cfg: HipConfig, stage: int) -> int:
    lib = load()
    n = _c_int()
    shape, c = decode_shape(q, k), cfg.c()
    _check("dsa_hip_max_chunks", lib.dsa_hip_max_chunks(ctypes.byref(shape), ctypes.byref(c),
                                                         stage, ctypes.byref(n)))
    return n.value


def hip_select(q, k, kv_len, cfg: HipConfig, *, debug: bool = False, out=None, workspace=None,
               stream=None):
    """Run all pruning stages; returns (sel_idx [B, keep[-1]], sel_cnt [B][, debug dict])."""
    return _hip_select(q, k, kv_len, cfg, None, debug, out, workspace, stream)


def hip_select_cached(q, k, kv_len, cfg: HipConfig, refresh: int, *, out, workspace,
                      debug: bool = False, stream=None):
    """Recompute only the pruning stages whose bit is set in `refresh` (InfiniteHiP,
    section 3.4 "Sparse Attention Mask Caching"); the others keep the lists they left in
    `workspace` / `out` on an earlier call, so both must persist between calls.
    Returns like hip_select (debug tensors of skipped stages stay at their fill)."""
    if out is None or workspace is None:
        raise ValueError("hip_select_cached needs the persistent out buffers and workspace")
    return _hip_select(q, k, kv_len, cfg, int(refresh), debug, out, workspace, stream)


def refresh_mask(step: int, n_refresh) -> int:
    """Stages to recompute at decoding step `step` (counted from 0) when stage i is
    refreshed every n_refresh[i] steps (InfiniteHiP, section 3.4): bit i is set iff
    step % n_refresh[i] == 0, so step 0 recomputes every stage."""
    m = 0
    for i, r in enumerate(n_refresh):
        if int(r) <= 0:
            raise ValueError("refresh intervals must be positive")
        if step % int(r) == 0:
            m |= 1 << i
    return m


class HipSelectCache:
    """Decoding-loop helper for mask caching: owns the workspace and the selection
    buffers, keeps the step counter and recomputes, on each call, the stages whose
    refresh interval divides it.  Shapes and config are fixed at construction."""

    def __init__(self, q, k, cfg: HipConfig, n_refresh):
        if len(n_refresh) != len(cfg.chunk):
            raise ValueError("one refresh interval per pruning stage")
        refresh_mask(0, n_refresh)
        self.cfg = cfg
        self.n_refresh = tuple(int(r) for r in n_refresh)
        B = q.shape[0]
        self.sel_idx = torch.empty(B, cfg.keep[-1], dtype=torch.int32, device=q.device)
        self.sel_cnt = torch.empty(B, dtype=torch.int32, device=q.device)
        self.workspace = _workspace(hip_select_workspace_bytes(q, k, cfg), q.device, None)
        self.step = 0

    def mask(self, step=None) -> int:
        return refresh_mask(self.step if step is None else step, self.n_refresh)

    def __call__(self, q, k, kv_len, *, debug: bool = False, stream=None):
        m = self.mask()
        self.step += 1
        return hip_select_cached(q, k, kv_len, self.cfg, m, out=(self.sel_idx, self.sel_cnt),
                                 workspace=self.workspace, debug=debug, stream=stream)


def _hip_select(q, k, kv_len, cfg, refresh, debug, out, workspace, stream):
    lib = load()
    _need_cuda(q, k, kv_len)
    shape, c = decode_shape(q, k), cfg.c()
    B = shape.B
    dev = q.device
    if out is None:
        sel_idx = torch.empty(B, cfg.keep[-1], dtype=torch.int32, device=dev)
        sel_cnt = torch.empty(B, dtype=torch.int32, device=dev)
    else:
        sel_idx, sel_cnt = out
    dbg = None
    dbg_t = None
    if debug:
        dbg = HipDebug()
        dbg_t = {"stage_idx": [], "stage_cnt": [], "chunk_score": [], "rep": [], "rep_score": []}
        for i in range(len(cfg.chunk)):
            mc = hip_max_chunks(q, k, cfg, i)
            t = {
                "stage_idx": torch.full((B, cfg.keep[i]), -7, dtype=torch.int32, device=dev),
                "stage_cnt": torch.full((B,), -7, dtype=torch.int32, device=dev),
                "chunk_score": torch.full((B, max(mc, 1)), float("nan"), device=dev),
                "rep": torch.full((B, shape.H_q, max(mc, 1)), -7, dtype=torch.int32, device=dev),
                "rep_score": torch.full((B, shape.H_q, max(mc, 1)), float("nan"), device=dev),
            }
            for key, v in t.items():
                dbg_t[key].append(v)
                getattr(dbg, key)[i] = v.data_ptr()
    nbytes = hip_select_workspace_bytes(q, k, cfg)
    ws = _workspace(nbytes, dev, workspace)
    dbg_p = ctypes.byref(dbg) if dbg else None
    if refresh is None:
        st = lib.hip_select(_ptr(q), _ptr(k), _ptr(kv_len), ctypes.byref(shape), ctypes.byref(c),
                            _ptr(sel_idx), _ptr(sel_cnt), dbg_p, _ptr(ws),
                            ctypes.c_size_t(ws.numel()), _stream(stream))
    else:
        st = lib.hip_select_cached(_ptr(q), _ptr(k), _ptr(kv_len), ctypes.byref(shape),
                                   ctypes.byref(c), refresh, _ptr(sel_idx), _ptr(sel_cnt),
                                   dbg_p, _ptr(ws), ctypes.c_size_t(ws.numel()), _stream(stream))
    _check("hip_select" if refresh is None else "hip_select_cached", st)
    if debug:
        return sel_idx, sel_cnt, dbg_t
    return sel_idx, sel_cnt


def sparse_attn_decode_workspace_bytes(q, k, max_sel: int, n_sink: int, n_stream: int) -> int:
    lib = load()
    n = ctypes.c_size_t()
    shape = decode_shape(q, k)
    _check("sparse_attn_decode_workspace",
           lib.sparse_attn_decode_workspace(ctypes.byref(shape), max_sel, n_sink, n_stream,
                                            ctypes.byref(n)))
    return n.value


def sparse_attn_decode(q, k, v, kv_len, sel_idx, sel_cnt, *, n_sink: int, n_stream: int,
                       scale: float | None = None, out=None, lse=None, want_lse: bool = True,
                       workspace=None, stream=None):
    """Attention over sink + selected + window keys; returns (out, lse or None)."""
    lib = load()
    _need_cuda(q, k, v, kv_len, sel_idx, sel_cnt)
    shape = decode_shape(q, k)
    max_sel = sel_idx.shape[1] if sel_idx is not None else 0
    if scale is None:
        scale = shape.D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(shape.B, shape.T_q, shape.H_q, dtype=torch.float32, device=q.device)
    nbytes = sparse_attn_decode_workspace_bytes(q, k, max_sel, n_sink, n_stream)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib.sparse_attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_len), _ptr(sel_idx),
                                _ptr(sel_cnt), max_sel, n_sink, n_stream, ctypes.c_float(scale),
                                ctypes.byref(shape), _ptr(out), _ptr(lse), _ptr(ws),
                                ctypes.c_size_t(ws.numel()), _stream(stream))
    _check("sparse_attn_decode", st)
    return out, lse


def sparse_attn_decode_noalloc(q, k, v, kv_len, sel_idx, sel_cnt, *, n_sink: int, n_stream: int,
                               scale: float | None = None, out=None, lse=None,
                               want_lse: bool = True, stream=None):
    """sparse_attn_decode whose split-K scratch is the library's built-in device array.

    For callers that must not allocate device memory when they call: nothing is
    allocated here either when `out` (and `lse`, or want_lse=False) are given.
    Calls that overlap on the GPU share the one array and must be serialised.
    """
    lib = load()
    _need_cuda(q, k, v, kv_len, sel_idx, sel_cnt)
    shape = decode_shape(q, k)
    max_sel = sel_idx.shape[1] if sel_idx is not None else 0
    if scale is None:
        scale = shape.D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(shape.B, shape.T_q, shape.H_q, dtype=torch.float32, device=q.device)
    st = lib.sparse_attn_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_len), _ptr(sel_idx),
                                        _ptr(sel_cnt), max_sel, n_sink, n_stream,
                                        ctypes.c_float(scale), ctypes.byref(shape), _ptr(out),
                                        _ptr(lse), _stream(stream))
    _check("sparse_attn_decode_noalloc", st)
    return out, lse


# ----------------------------------------------------------------------------- prefill

def prefill_shape(q: torch.Tensor, k: torch.Tensor) -> PrefillShape:
    B, S, H_q, D = q.shape
    return PrefillShape(B, S, H_q, k.shape[2], D)


def vs_index_build_workspace_bytes(q, k, last_q, n_vertical, n_slash, block=64) -> int:
    lib = load()
    n = ctypes.c_size_t()
    shape = prefill_shape(q, k)
    cfg = VsCfg(last_q, n_vertical, n_slash, block)
    _check("vs_index_build_workspace",
           lib.vs_index_build_workspace(ctypes.byref(shape), ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def vs_index_build(q, k, *, last_q: int = 64, n_vertical: int, n_slash: int, block: int = 64,
                   debug: bool = False, out: dict | None = None, workspace=None, stream=None):
    """Vertical-slash index and its tile/column lists; returns a dict of tensors."""
    lib = load()
    _need_cuda(q, k)
    shape = prefill_shape(q, k)
    B, S, H_q = shape.B, shape.S, shape.H_q
    nq = (S + block - 1) // block
    dev = q.device
    if out is None:
        out = {
            "vertical": torch.empty(B, H_q, n_vertical, dtype=torch.int32, device=dev),
            "slash": torch.empty(B, H_q, n_slash, dtype=torch.int32, device=dev),
            "blk_cnt": torch.empty(B, H_q, nq, dtype=torch.int32, device=dev),
            "blk_idx": torch.empty(B, H_q, nq, nq, dtype=torch.int32, device=dev),
            "col_cnt": torch.empty(B, H_q, nq, dtype=torch.int32, device=dev),
            "col_idx": torch.empty(B, H_q, nq, max(n_vertical, 1), dtype=torch.int32, device=dev),
        }
    dbg = None
    if debug:
        out["vsum"] = torch.empty(B, H_q, S, dtype=torch.float32, device=dev)
        out["ssum"] = torch.empty(B, H_q, S, dtype=torch.float32, device=dev)
        dbg = VsDebug(out["vsum"].data_ptr(), out["ssum"].data_ptr())
    cfg = VsCfg(last_q, n_vertical, n_slash, block)
    ws = _workspace(vs_index_build_workspace_bytes(q, k, last_q, n_vertical, n_slash, block),
                    dev, workspace)
    st = lib.vs_index_build(_ptr(q), _ptr(k), ctypes.byref(shape), ctypes.byref(cfg),
                            _ptr(out["vertical"]), _ptr(out["slash"]), _ptr(out["blk_cnt"]),
                            _ptr(out["blk_idx"]), _ptr(out["col_cnt"]), _ptr(out["col_idx"]),
                            ctypes.byref(dbg) if dbg else None, _ptr(ws),
                            ctypes.c_size_t(ws.numel()), _stream(stream))
    _check("vs_index_build", st)
    return out


def _block_lists(B, H_q, nq, max_blk, dev, out):
    if out is None:
        out = {
            "blk_cnt": torch.empty(B, H_q, nq, dtype=torch.int32, device=dev),
            "blk_idx": torch.empty(B, H_q, nq, max(max_blk, 1), dtype=torch.int32, device=dev),
            "col_cnt": torch.empty(B, H_q, nq, dtype=torch.int32, device=dev),
        }
    out.setdefault("col_idx", None)
    return out


def ashape_index_build(q, k, *, n_global: int, n_local: int, block: int = 64, max_blk=None,
                       out: dict | None = None, stream=None):
    """A-shape lists (initial blocks + a band ending at the diagonal); q and k give the
    shape only.  Returns a dict with blk_cnt, blk_idx, col_cnt (all 0), col_idx None."""
    lib = load()
    shape = prefill_shape(q, k)
    nq = (shape.S + block - 1) // block
    if max_blk is None:
        max_blk = min(nq, n_global // block + n_local // block)
    out = _block_lists(shape.B, shape.H_q, nq, max_blk, q.device, out)
    _need_cuda(out["blk_cnt"], out["blk_idx"], out["col_cnt"])
    st = lib.ashape_index_build(ctypes.byref(shape), block, n_global, n_local,
                                out["blk_idx"].shape[-1], _ptr(out["blk_cnt"]),
                                _ptr(out["blk_idx"]), _ptr(out["col_cnt"]), _stream(stream))
    _check("ashape_index_build", st)
    return out


def block_sparse_index_build_workspace_bytes(q, k, block: int = 64) -> int:
    lib = load()
    n = ctypes.c_size_t()
    shape = prefill_shape(q, k)
    _check("block_sparse_index_build_workspace",
           lib.block_sparse_index_build_workspace(ctypes.byref(shape), block, ctypes.byref(n)))
    return n.value


def block_sparse_index_build(q, k, *, k_b: int, block: int = 64, max_blk=None,
                             debug: bool = False, out: dict | None = None, workspace=None,
                             stream=None):
    """Block-Sparse lists (mean-pooled block attention, top-k_b key blocks per query
    block).  Returns a dict with blk_cnt, blk_idx, col_cnt (all 0), col_idx None and,
    with debug, the pooled blocks and the block logits."""
    lib = load()
    _need_cuda(q, k)
    shape = prefill_shape(q, k)
    B, S, H_q = shape.B, shape.S, shape.H_q
    nq = (S + block - 1) // block
    if max_blk is None:
        max_blk = min(k_b, nq)
    out = _block_lists(B, H_q, nq, max_blk, q.device, out)
    dbg = None
    if debug:
        dev = q.device
        out["q_pool"] = torch.empty(B, H_q, nq, shape.D, dtype=torch.float32, device=dev)
        out["k_pool"] = torch.empty(B, shape.H_kv, nq, shape.D, dtype=torch.float32, device=dev)
        out["scores"] = torch.full((B, H_q, nq, nq), float("nan"), dtype=torch.float32, device=dev)
        dbg = BsDebug(out["q_pool"].data_ptr(), out["k_pool"].data_ptr(),
                      out["scores"].data_ptr())
    ws = _workspace(block_sparse_index_build_workspace_bytes(q, k, block), q.device, workspace)
    st = lib.block_sparse_index_build(_ptr(q), _ptr(k), ctypes.byref(shape), block, k_b,
                                      out["blk_idx"].shape[-1], _ptr(out["blk_cnt"]),
                                      _ptr(out["blk_idx"]), _ptr(out["col_cnt"]),
                                      ctypes.byref(dbg) if dbg else None, _ptr(ws),
                                      ctypes.c_size_t(ws.numel()), _stream(stream))
    _check("block_sparse_index_build", st)
    return out


def _mixed_cfg(H_q, head_pattern, last_q, n_vertical, n_slash, n_global, n_local, k_b, block):
    pats = [(_PATTERN_NAMES[p] if isinstance(p, str) else int(p)) for p in head_pattern]
    if len(pats) != H_q:
        raise ValueError(f"head_pattern needs {H_q} entries, got {len(pats)}")
    arr = (ctypes.c_uint8 * H_q)(*pats)
    cfg = MixedCfg(ctypes.cast(arr, _vp), VsCfg(last_q, n_vertical, n_slash, block), n_global,
                   n_local, k_b)
    return cfg, arr, pats


def mixed_index_build(q, k, *, head_pattern, last_q: int = 64, n_vertical: int = 1000,
                      n_slash: int = 6096, n_global: int = 1024, n_local: int = 4096,
                      k_b: int = 100, block: int = 64, out: dict | None = None, workspace=None,
                      stream=None):
    """Per-head patterns (head_pattern: one of "vertical_slash", "a_shape",
    "block_sparse" or 0/1/2 per query head) into one set of tile/column lists."""
    lib = load()
    _need_cuda(q, k)
    shape = prefill_shape(q, k)
    B, S, H_q = shape.B, shape.S, shape.H_q
    cfg, arr, pats = _mixed_cfg(H_q, head_pattern, last_q, n_vertical, n_slash, n_global,
                                n_local, k_b, block)
    nq = (S + block - 1) // block
    dev = q.device
    if out is None:
        out = {
            "blk_cnt": torch.empty(B, H_q, nq, dtype=torch.int32, device=dev),
            "blk_idx": torch.empty(B, H_q, nq, nq, dtype=torch.int32, device=dev),
            "col_cnt": torch.empty(B, H_q, nq, dtype=torch.int32, device=dev),
            "col_idx": torch.empty(B, H_q, nq, max(n_vertical, 1), dtype=torch.int32, device=dev),
        }
    n = ctypes.c_size_t()
    _check("mixed_index_build_workspace",
           lib.mixed_index_build_workspace(ctypes.byref(shape), ctypes.byref(cfg), ctypes.byref(n)))
    ws = _workspace(n.value, dev, workspace)
    st = lib.mixed_index_build(_ptr(q), _ptr(k), ctypes.byref(shape), ctypes.byref(cfg),
                               _ptr(out["blk_cnt"]), _ptr(out["blk_idx"]), _ptr(out["col_cnt"]),
                               _ptr(out["col_idx"]), _ptr(ws), ctypes.c_size_t(ws.numel()),
                               _stream(stream))
    del arr
    _check("mixed_index_build", st)
    return out


def mixed_index_build_workspace_bytes(q, k, *, head_pattern, last_q: int = 64,
                                      n_vertical: int = 1000, n_slash: int = 6096,
                                      n_global: int = 1024, n_local: int = 4096, k_b: int = 100,
                                      block: int = 64) -> int:
    lib = load()
    shape = prefill_shape(q, k)
    cfg, arr, _ = _mixed_cfg(shape.H_q, head_pattern, last_q, n_vertical, n_slash, n_global,
                             n_local, k_b, block)
    n = ctypes.c_size_t()
    _check("mixed_index_build_workspace",
           lib.mixed_index_build_workspace(ctypes.byref(shape), ctypes.byref(cfg), ctypes.byref(n)))
    del arr
    return n.value


def hip_prefill_max_chunks(q, k, cfg: HipConfig, stage: int) -> int:
    lib = load()
    n = _c_int()
    shape, c = prefill_shape(q, k), cfg.c()
    _check("dsa_hip_prefill_max_chunks",
           lib.dsa_hip_prefill_max_chunks(ctypes.byref(shape), ctypes.byref(c), stage, ctypes.byref(n)))
    return n.value


def hip_prefill_select_workspace_bytes(q, k, cfg: HipConfig) -> int:
    lib = load()
    n = ctypes.c_size_t()
    shape, c = prefill_shape(q, k), cfg.c()
    _check("hip_prefill_select_workspace",
           lib.hip_prefill_select_workspace(ctypes.byref(shape), ctypes.byref(c), ctypes.byref(n)))
    return n.value


def hip_prefill_select(q, k, cfg: HipConfig, *, debug: bool = False, out=None, workspace=None,
                       stream=None):
    """InfiniteHiP pruning for every 64-row query block of a causal prefill; returns
    (sel_idx [B * n_qblk, keep[-1]], sel_cnt [B * n_qblk][, debug dict]), rows ordered
    b * n_qblk + m."""
    lib = load()
    _need_cuda(q, k)
    shape, c = prefill_shape(q, k), cfg.c()
    R = shape.B * ((shape.S + 63) // 64)
    dev = q.device
    if out is None:
        sel_idx = torch.empty(R, cfg.keep[-1], dtype=torch.int32, device=dev)
        sel_cnt = torch.empty(R, dtype=torch.int32, device=dev)
    else:
        sel_idx, sel_cnt = out
    dbg = dbg_t = None
    if debug:
        dbg = HipDebug()
        dbg_t = {"stage_idx": [], "stage_cnt": [], "chunk_score": [], "rep": [], "rep_score": []}
        for i in range(len(cfg.chunk)):
            mc = max(hip_prefill_max_chunks(q, k, cfg, i), 1)
            t = {
                "stage_idx": torch.full((R, cfg.keep[i]), -7, dtype=torch.int32, device=dev),
                "stage_cnt": torch.full((R,), -7, dtype=torch.int32, device=dev),
                "chunk_score": torch.full((R, mc), float("nan"), device=dev),
                "rep": torch.full((R, shape.H_q, mc), -7, dtype=torch.int32, device=dev),
                "rep_score": torch.full((R, shape.H_q, mc), float("nan"), device=dev),
            }
            for key, v in t.items():
                dbg_t[key].append(v)
                getattr(dbg, key)[i] = v.data_ptr()
    ws = _workspace(hip_prefill_select_workspace_bytes(q, k, cfg), dev, workspace)
    st = lib.hip_prefill_select(_ptr(q), _ptr(k), ctypes.byref(shape), ctypes.byref(c),
                                _ptr(sel_idx), _ptr(sel_cnt), ctypes.byref(dbg) if dbg else None,
                                _ptr(ws), ctypes.c_size_t(ws.numel()), _stream(stream))
    _check("hip_prefill_select", st)
    if debug:
        return sel_idx, sel_cnt, dbg_t
    return sel_idx, sel_cnt


def hip_prefill_lists(q, k, cfg: HipConfig, sel_idx, sel_cnt, *, out: dict | None = None,
                      stream=None):
    """Each query block's sink + selection + window as sparse_attn_prefill lists (the
    same for every head); returns a dict with blk_cnt, blk_idx, col_cnt, col_idx."""
    lib = load()
    _need_cuda(sel_idx, sel_cnt)
    shape, c = prefill_shape(q, k), cfg.c()
    nq = (shape.S + 63) // 64
    max_blk = -(-cfg.n_sink // 64) + -(-cfg.n_stream // 64) + 2
    max_col = cfg.keep[-1] + 126
    dev = sel_idx.device
    if out is None:
        out = {
            "blk_cnt": torch.empty(shape.B, shape.H_q, nq, dtype=torch.int32, device=dev),
            "blk_idx": torch.empty(shape.B, shape.H_q, nq, max_blk, dtype=torch.int32, device=dev),
            "col_cnt": torch.empty(shape.B, shape.H_q, nq, dtype=torch.int32, device=dev),
            "col_idx": torch.empty(shape.B, shape.H_q, nq, max_col, dtype=torch.int32, device=dev),
        }
    st = lib.hip_prefill_lists(ctypes.byref(shape), ctypes.byref(c), _ptr(sel_idx), _ptr(sel_cnt),
                               out["blk_idx"].shape[-1], out["col_idx"].shape[-1],
                               _ptr(out["blk_cnt"]), _ptr(out["blk_idx"]), _ptr(out["col_cnt"]),
                               _ptr(out["col_idx"]), _stream(stream))
    _check("hip_prefill_lists", st)
    return out


def sparse_attn_prefill(q, k, v, blk_cnt, blk_idx, col_cnt, col_idx, *, scale=None,
                        block: int = 64, out=None, lse=None, want_lse: bool = True, stream=None):
    """Causal attention over the listed tiles and columns (col_idx None: no columns);
    returns (out, lse or None)."""
    lib = load()
    _need_cuda(q, k, v, blk_cnt, blk_idx, col_cnt, col_idx)
    shape = prefill_shape(q, k)
    if scale is None:
        scale = shape.D ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(shape.B, shape.H_q, shape.S, dtype=torch.float32, device=q.device)
    st = lib.sparse_attn_prefill(_ptr(q), _ptr(k), _ptr(v), ctypes.byref(shape), block,
                                 blk_idx.shape[-1], 0 if col_idx is None else col_idx.shape[-1],
                                 _ptr(blk_cnt),
                                 _ptr(blk_idx), _ptr(col_cnt), _ptr(col_idx),
                                 ctypes.c_float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check("sparse_attn_prefill", st)
    return out, lse


# ----------------------------------------------------------------------------- paged cache

@dataclass
class PagedKVCache:
    """Keys and values in pages [n_pages, page_size, H_kv, D]: bf16, or FP8 E4M3 codes (a
    uint8 or float8_e4m3fn tensor) with one scale byte per token and head in k_scale /
    v_scale [n_pages, page_size, H_kv] (uint8; a row's values are code * 2**(byte - 127)).
    The tensors are the caller's; `empty` allocates a cache."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    @classmethod
    def empty(cls, n_pages: int, page_size: int, H_kv: int, D: int, *, fp8: bool = False,
              device="cuda") -> "PagedKVCache":
        shape = (n_pages, page_size, H_kv, D)
        if not fp8:
            return cls(*(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        return cls(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)))

    @property
    def fp8(self) -> bool:
        return _is_fp8(self.k)


_MAX_KEYS = 1 << 30   # of a sequence: larger windows see no more
_FP8_TYPES = (torch.uint8, torch.float8_e4m3fn)

# Every decode step makes these calls, and a small one is over on the GPU in a few
# microseconds: the checks below read each property of a tensor once, numbers that follow from
# the shape alone are kept (_paged_shape), and the device and stream are only switched when
# the call needs another one than the current.

def _shape_struct(*sizes):
    """PagedShape of B, n_tok, max_pages, n_pages, page_size, H_q, H_kv, D, dtype."""
    for (name, _), x in zip(PagedShape._fields_, sizes):
        if not -2 ** 31 <= x < 2 ** 31:                 # (ctypes would cut it to 32 bits)
            raise ValueError(f"{name}={x} does not fit in 32 bits")
    return PagedShape(*sizes)


@functools.lru_cache(maxsize=1024)
def _paged_shape(*sizes):
    """(ctypes shape, workspace bytes of paged_attn) of B, n_tok, max_pages, n_pages,
    page_size, H_q, H_kv, D, dtype."""
    shape, n = _shape_struct(*sizes), ctypes.c_size_t()
    _check("paged_attn_workspace", load().paged_attn_workspace(ctypes.byref(shape), ctypes.byref(n)))
    return ctypes.byref(shape), n.value


def _index(t, name, dims, dev):
    """Pointer of a contiguous int32 tensor of `dims` dimensions on device `dev`."""
    if t.dtype != torch.int32 or t.dim() != dims:
        raise TypeError(f"{name} must be a {dims}-dimensional int32 tensor")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on the cache's device")
    return t.data_ptr()


def _cache_args(cache: PagedKVCache):
    """(pointers of k, v, k_scale, v_scale, shape of k, dsa_dtype, device index), checked."""
    k, v, ks, vs = cache.k, cache.v, cache.k_scale, cache.v_scale
    dev, shape, dtype = k.get_device(), k.shape, k.dtype
    if dev < 0:
        raise ValueError("tensors must be contiguous CUDA tensors")
    if len(shape) != 4 or v.shape != shape or v.dtype != dtype:
        raise ValueError("k and v must be [n_pages, page_size, H_kv, D] tensors of one type")
    if v.get_device() != dev or not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("k and v must be contiguous CUDA tensors on one device")
    if dtype == torch.bfloat16:
        if ks is not None or vs is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return k.data_ptr(), v.data_ptr(), None, None, shape, BF16, dev
    if dtype not in _FP8_TYPES:
        raise TypeError(f"unsupported cache type {dtype}; use bfloat16 or FP8 E4M3 codes")
    for t in (ks, vs):
        if t is None or t.dtype != torch.uint8 or t.shape != shape[:3]:
            raise ValueError("an FP8 cache needs uint8 scales of [n_pages, page_size, H_kv]")
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError("the scales must be contiguous and on the cache's device")
    return k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), shape, BF16_FP8KV, dev


def _table_args(page_table, kv_len, q_start, dev, heads=0):
    """(pointers of page_table, kv_len, q_start, B, max_pages), checked; with `heads` the table is
    [B, heads, max_pages]."""
    if heads:
        table = _index(page_table, "page_table", 3, dev)
        B, h, max_pages = page_table.shape
        if h != heads:
            raise ValueError(f"a page table for each KV head must be [B, {heads}, max_pages]")
    else:
        B, max_pages = page_table.shape if page_table.dim() == 2 else (-1, -1)
        table = _index(page_table, "page_table", 2, dev)
    lens = _index(kv_len, "kv_len", 1, dev)
    if kv_len.shape[0] != B:
        raise ValueError("kv_len must be [B], page_table [B, max_pages]")
    if q_start is None:
        return table, lens, None, B, max_pages
    start = _index(q_start, "q_start", 1, dev)
    if q_start.shape[0] != B + 1:
        raise ValueError("q_start must be [B + 1]")
    return table, lens, start, B, max_pages


def _token_rows(t, name, heads, D, dev):
    """(rows, token stride) of a bf16 [n_tok, heads, D] tensor; only tokens may be strided."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or t.dtype != torch.bfloat16 or (heads and shape[1] != heads):
        raise ValueError(f"{name} must be a bfloat16 [n_tok, {heads or 'H_q'}, {D}] tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the cache's device")
    s = t.stride()
    if s[2] != 1 or (s[1] != D and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous (only tokens may be strided)")
    return shape[0], s[0] if shape[0] > 1 else shape[1] * D


def _current_stream(dev):
    """Raw current stream of device `dev` if that is the current device, else None."""
    return torch._C._cuda_getCurrentRawStream(dev) if torch._C._cuda_getDevice() == dev else None


def _call_stream(dev, stream):
    """Raw stream of a call on device `dev`, None if the device or the stream has to be switched
    first (_on).  Handles say nothing about the device: every default stream's is 0."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream is on device {stream.device_index}, the cache on device {dev}")
    st = _current_stream(dev)
    return st if stream is None or stream.cuda_stream == st else None


class _on:
    """Device `dev` as the current one and `stream` (None: its current stream) as the stream
    that outputs and workspaces are allocated and a call is enqueued on."""

    def __init__(self, dev, stream):
        _call_stream(dev, stream)   # refuses another device's
        self.device_ctx = torch.cuda.device(dev)
        self.stream = stream

    def __enter__(self):
        self.device_ctx.__enter__()
        self.stream_ctx = torch.cuda.stream(self.stream)   # None: nothing changes
        self.stream_ctx.__enter__()
        return torch.cuda.current_stream()

    def __exit__(self, *exc):
        self.stream_ctx.__exit__(*exc)
        self.device_ctx.__exit__(*exc)


def kv_cache_write(cache: PagedKVCache, k_new, v_new, q_start, kv_len, page_table, *, stream=None) -> None:
    """Write the chunks' keys and values (bf16 [n_tok, H_kv, D], tokens may be strided) into
    their pages, quantised if the cache is FP8.  Sequence b's chunk is rows q_start[b] ..
    q_start[b + 1] - 1 and holds its last positions; kv_len counts the chunk."""
    lib = _lib or load()
    k, v, ks, vs, (n_pages, page_size, H_kv, D), dtype, dev = _cache_args(cache)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return kv_cache_write(cache, k_new, v_new, q_start, kv_len, page_table)
    table, lens, start, B, max_pages = _table_args(page_table, kv_len, q_start, dev)
    n_tok, k_stride = _token_rows(k_new, "k_new", H_kv, D, dev)
    n_v, v_stride = _token_rows(v_new, "v_new", H_kv, D, dev)
    if n_v != n_tok:
        raise ValueError("k_new and v_new must have the same tokens")
    shape, _ = _paged_shape(B, n_tok, max_pages, n_pages, page_size, H_kv, H_kv, D, dtype)
    status = lib.kv_cache_write(k_new.data_ptr(), v_new.data_ptr(), k_stride, v_stride, start, lens,
                                table, shape, k, v, ks, vs, st)
    if status:
        _check("kv_cache_write", status)


def kv_cache_read(cache: PagedKVCache, kv_len, page_table, *, T_max: int | None = None, out=None,
                  stream=None):
    """The sequences' rows as contiguous bf16 (k, v) [B, T_max, H_kv, D], the layout that
    hip_select, sparse_attn_decode and the index builders read.  `out`: (k, v) to write into
    (rows behind a sequence's end stay as they are); else new tensors, zero there, of T_max
    (default: max_pages * page_size) rows, whose zeroes take more time than the rows: 131,072 FP8
    tokens of 8 heads of 128 in 263 us, with `out` in 122."""
    lib = _lib or load()
    k, v, ks, vs, (n_pages, page_size, H_kv, D), dtype, dev = _cache_args(cache)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return kv_cache_read(cache, kv_len, page_table, T_max=T_max, out=out)
    table, lens, _, B, max_pages = _table_args(page_table, kv_len, None, dev)
    shape, _ = _paged_shape(B, 0, max_pages, n_pages, page_size, H_kv, H_kv, D, dtype)
    if out is None:
        rows = max_pages * page_size if T_max is None else int(T_max)
        out = tuple(torch.zeros(B, rows, H_kv, D, dtype=torch.bfloat16, device=cache.k.device)
                    for _ in range(2))
    k_out, v_out = out
    rows = k_out.shape[1] if T_max is None else int(T_max)
    for t in out:
        if t.shape != (B, rows, H_kv, D) or t.dtype != torch.bfloat16:
            raise ValueError("out must be two bfloat16 [B, T_max, H_kv, D] tensors")
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError("out must be contiguous and on the cache's device")
    status = lib.kv_cache_read(k, v, ks, vs, lens, table, shape, rows, k_out.data_ptr(), v_out.data_ptr(), st)
    if status:
        _check("kv_cache_read", status)
    return k_out, v_out


def paged_attn_workspace_bytes(q, cache: PagedKVCache, page_table) -> int:
    n_pages, page_size, H_kv, D = cache.k.shape
    return _paged_shape(page_table.shape[0], q.shape[0], page_table.shape[-1], n_pages, page_size,
                        q.shape[1], H_kv, D, BF16_FP8KV if cache.fp8 else BF16)[1]


def paged_attn(q, cache: PagedKVCache, q_start, kv_len, page_table, *, n_sink: int = 0,
               n_stream: int | None = None, scale: float | None = None, out=None, lse=None,
               want_lse: bool = True, workspace=None, stream=None):
    """Causal attention of the chunks q (bf16 [n_tok, H_q, D], tokens may be strided) over the
    cache, which holds their own keys already (kv_cache_write).  A row at position p attends
    every key j <= p, or with n_stream the n_stream newest of them (its own included) beside
    the first n_sink.  page_table [B, max_pages], or [B, H_kv, max_pages] with a list of pages for each
    KV head (page_select's), whose places are then the positions.  Returns (out [n_tok, H_q, D], lse [n_tok, H_q] or None)."""
    lib = _lib or load()
    k, v, ks, vs, (n_pages, page_size, H_kv, D), dtype, dev = _cache_args(cache)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return paged_attn(q, cache, q_start, kv_len, page_table, n_sink=n_sink, n_stream=n_stream,
                              scale=scale, out=out, lse=lse, want_lse=want_lse, workspace=workspace)
    lists = page_table.dim() == 3
    table, lens, start, B, max_pages = _table_args(page_table, kv_len, q_start, dev, H_kv if lists else 0)
    n_tok, q_stride = _token_rows(q, "q", 0, D, dev)
    H_q = q.shape[1]
    if n_sink < 0:                                      # (ctypes would cut a large negative one to 32 bits)
        raise ValueError("n_sink must be >= 0")
    if n_stream is None:
        n_stream = -1
    elif n_stream < 0:
        raise ValueError("n_stream must be >= 0, or None for every key")
    if n_sink > _MAX_KEYS or n_stream > _MAX_KEYS:
        n_sink, n_stream = min(n_sink, _MAX_KEYS), min(n_stream, _MAX_KEYS)
    shape, nbytes = _paged_shape(B, n_tok, max_pages, n_pages, page_size, H_q, H_kv, D, dtype)
    device = q.device
    if out is None:
        out = torch.empty((n_tok, H_q, D), dtype=torch.bfloat16, device=device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor of q's shape on its device")
    if lse is None:
        if want_lse:
            lse = torch.empty((n_tok, H_q), dtype=torch.float32, device=device)
    elif lse.shape != (n_tok, H_q) or lse.dtype != torch.float32 or lse.get_device() != dev or \
            not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [n_tok, H_q] tensor on q's device")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the cache's device")
    call = lib.paged_attn_lists if lists else lib.paged_attn
    status = call(q.data_ptr(), q_stride, k, v, ks, vs, start, lens, table, shape, n_sink, n_stream,
                  D ** -0.5 if scale is None else scale, out.data_ptr(),
                  None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                  workspace.numel() * workspace.element_size(), st)
    if status:
        _check("paged_attn_lists" if lists else "paged_attn", status)
    return out, lse


# ----------------------------------------------------------------------------- the pages' sparse path

def kv_cache_write_rope(cache: PagedKVCache, q, k_new, v_new, q_start, kv_len, page_table, inv_freq, *,
                        interleaved: bool = False, rope_scale: float = 1.0, q_weight=None, k_weight=None,
                        eps: float = 1e-6, q_out=None, stream=None):
    """kv_cache_write with each head's norm and the rotation by position in the same pass, for
    the queries too; returns the rotated queries [n_tok, H_q, D] (`q_out`, which may be q itself, else a
    new tensor).  q, k_new, v_new: bf16 [n_tok, heads, D], tokens may be strided (slices of a
    fused projection).  q_weight, k_weight [D] (bf16 or fp32, both alike): the rows are divided by their
    root mean square (eps added to the square) and multiplied by it; None: no norm.  inv_freq: float64
    [rot / 2] on the device, radians per position of the pairs (i, i + rot / 2), or (2 i, 2 i + 1) when
    interleaved, of the first `rot` dimensions (a multiple of 16); None: no rotation."""
    lib = _lib or load()
    k, v, ks, vs, (n_pages, page_size, H_kv, D), dtype, dev = _cache_args(cache)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return kv_cache_write_rope(cache, q, k_new, v_new, q_start, kv_len, page_table, inv_freq,
                                       interleaved=interleaved, rope_scale=rope_scale, q_weight=q_weight,
                                       k_weight=k_weight, eps=eps, q_out=q_out)
    table, lens, start, B, max_pages = _table_args(page_table, kv_len, q_start, dev)
    n_tok, q_stride = _token_rows(q, "q", 0, D, dev)
    n_k, k_stride = _token_rows(k_new, "k_new", H_kv, D, dev)
    n_v, v_stride = _token_rows(v_new, "v_new", H_kv, D, dev)
    if n_k != n_tok or n_v != n_tok:
        raise ValueError("q, k_new and v_new must have the same tokens")
    H_q = q.shape[1]
    wtype = None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if w.dtype not in (torch.bfloat16, torch.float32) or (wtype or w.dtype) != w.dtype or w.shape != (D,):
            raise ValueError(f"{name} must be a [{D}] tensor, bfloat16 or float32 and both alike")
        if w.get_device() != dev or not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous and on the cache's device")
        wtype = w.dtype
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be a 1-dimensional float64 tensor")
        if inv_freq.get_device() != dev or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be contiguous and on the cache's device")
        rot = 2 * inv_freq.shape[0]
    if q_out is None:
        q_out = torch.empty((n_tok, H_q, D), dtype=torch.bfloat16, device=q.device)
    elif q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    n_o, o_stride = _token_rows(q_out, "q_out", H_q, D, dev)
    shape, _ = _paged_shape(B, n_tok, max_pages, n_pages, page_size, H_q, H_kv, D, dtype)
    cfg = RopeCfg(None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
                  wtype == torch.float32, eps, inv_freq.data_ptr() if rot else None, rot, bool(interleaved), rope_scale)
    status = lib.kv_cache_write_rope(q.data_ptr(), q_stride, k_new.data_ptr(), k_stride, v_new.data_ptr(), v_stride,
                                     start, lens, table, shape, ctypes.byref(cfg), q_out.data_ptr(), o_stride,
                                     k, v, ks, vs, st)
    if status:
        _check("kv_cache_write_rope", status)
    return q_out


@dataclass
class PageDigest:
    """8-bit bounds of the keys of a cache's pages: bounds int8 [n_pages, H_kv, 2, D] (smallest,
    largest of each channel, rounded outwards) times 2**exp, exp int8 [n_pages, H_kv].  The
    tensors are the caller's; `empty` allocates them for a cache."""
    bounds: torch.Tensor
    exp: torch.Tensor
    page_size: int

    @classmethod
    def empty(cls, cache: PagedKVCache) -> "PageDigest":
        n_pages, page_size, H_kv, D = cache.k.shape
        return cls(torch.zeros(n_pages, H_kv, 2, D, dtype=torch.int8, device=cache.k.device),
                   torch.zeros(n_pages, H_kv, dtype=torch.int8, device=cache.k.device), page_size)


def _digest_args(digest: PageDigest):
    """(pointers of bounds and exp, n_pages, H_kv, D, device index), checked."""
    bounds, exp = digest.bounds, digest.exp
    dev, shape = bounds.get_device(), bounds.shape
    if dev < 0:
        raise ValueError("tensors must be contiguous CUDA tensors")
    if len(shape) != 4 or shape[2] != 2 or exp.shape != shape[:2]:
        raise ValueError("bounds must be [n_pages, H_kv, 2, D] and exp [n_pages, H_kv]")
    if bounds.dtype != torch.int8 or exp.dtype != torch.int8:
        raise TypeError("bounds and exp must be int8")
    if exp.get_device() != dev or not bounds.is_contiguous() or not exp.is_contiguous():
        raise ValueError("bounds and exp must be contiguous CUDA tensors on one device")
    return bounds.data_ptr(), exp.data_ptr(), shape[0], shape[1], shape[3], dev


def _digest_of_cache(digest, n_pages, page_size, H_kv, D, dev):
    """Pointers of a digest that has to belong to a cache."""
    bounds, exp, n, h, d, ddev = _digest_args(digest)
    if (n, h, d, digest.page_size) != (n_pages, H_kv, D, page_size):
        raise ValueError("the digest is of another cache's shape")
    if ddev != dev:
        raise ValueError("the digest must be on the cache's device")
    return bounds, exp


def page_digest_update(cache: PagedKVCache, digest: PageDigest, n_tok: int, q_start, kv_len, page_table, *,
                       stream=None) -> None:
    """Digest again the pages that the chunks touch, over all of their keys below kv_len: after every
    write of new tokens.  n_tok: rows of the chunks' token tensors (at least q_start[-1])."""
    lib = _lib or load()
    k, _, ks, _, (n_pages, page_size, H_kv, D), dtype, dev = _cache_args(cache)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return page_digest_update(cache, digest, n_tok, q_start, kv_len, page_table)
    bounds, exp = _digest_of_cache(digest, n_pages, page_size, H_kv, D, dev)
    table, lens, start, B, max_pages = _table_args(page_table, kv_len, q_start, dev)
    shape, _ = _paged_shape(B, int(n_tok), max_pages, n_pages, page_size, H_kv, H_kv, D, dtype)
    status = lib.page_digest_update(k, ks, start, lens, table, shape, bounds, exp, st)
    if status:
        _check("page_digest_update", status)


@dataclass
class PageSelection:
    """Lists of pages for blocks of queries, as paged_attn takes them: rows q_start[j] ..
    q_start[j + 1] - 1 of the queries attend kv_len[j] keys in the pages page_table[j, h] (-1
    behind the end).  index: the same lists as places in the sequences' tables, if asked for."""
    q_start: torch.Tensor
    kv_len: torch.Tensor
    page_table: torch.Tensor
    index: torch.Tensor | None = None


@functools.lru_cache(maxsize=1024)
def _select_sizes(keep, n_sink, n_local, q_block, *sizes):
    """(ctypes shape, ctypes cfg, n_blocks, max_list) of a page_select call."""
    shape, cfg = _shape_struct(*sizes), PageSelectCfg(keep, n_sink, n_local, q_block)
    n, m = _c_int(), _c_int()
    _check("page_select_sizes", load().page_select_sizes(ctypes.byref(shape), ctypes.byref(cfg), ctypes.byref(n),
                                                         ctypes.byref(m)))
    return ctypes.byref(shape), ctypes.byref(cfg), n.value, m.value


def page_select(q, digest: PageDigest, q_start, kv_len, page_table, *, keep: int, n_sink: int = 1,
                n_local: int = 1, q_block: int = 1, want_index: bool = False, out: PageSelection | None = None,
                stream=None) -> PageSelection:
    """Which pages each block of q_block queries (bf16 [n_tok, H_q, D], tokens may be strided) attends, for
    each KV head: the first n_sink, the `keep` with the largest bound on a score (from the digest), the
    n_local before the block's own ones, and those.  The result goes to paged_attn:
        sel = page_select(q, digest, q_start, kv_len, page_table, keep=60)
        out, lse = paged_attn(q, cache, sel.q_start, sel.kv_len, sel.page_table)
    `out`: a PageSelection to write into (its index, if it has one, as well)."""
    lib = _lib or load()
    bounds, exp, n_pages, H_kv, D, dev = _digest_args(digest)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return page_select(q, digest, q_start, kv_len, page_table, keep=keep, n_sink=n_sink, n_local=n_local,
                               q_block=q_block, want_index=want_index, out=out)
    for name, x in (("keep", keep), ("n_sink", n_sink), ("n_local", n_local), ("q_block", q_block)):
        if not 0 <= x <= _MAX_KEYS:                     # (ctypes would cut a larger one to 32 bits)
            raise ValueError(f"{name}={x} must be in [0, 2^30]")
    table, lens, start, B, max_pages = _table_args(page_table, kv_len, q_start, dev)
    n_tok, q_stride = _token_rows(q, "q", 0, D, dev)
    shape, cfg, n_blocks, max_list = _select_sizes(keep, n_sink, n_local, q_block, B, n_tok, max_pages, n_pages,
                                                   digest.page_size, q.shape[1], H_kv, D, BF16)
    dims = (n_blocks, H_kv, max_list)
    if out is None:
        def new(*size):
            return torch.empty(size, dtype=torch.int32, device=q.device)
        out = PageSelection(new(n_blocks + 1), new(n_blocks), new(*dims), new(*dims) if want_index else None)
    else:
        for name, t, size in (("q_start", out.q_start, (n_blocks + 1,)), ("kv_len", out.kv_len, (n_blocks,)),
                              ("page_table", out.page_table, dims), ("index", out.index, dims)):
            if t is None and name == "index":
                continue
            if _index(t, "out." + name, len(size), dev) and tuple(t.shape) != size:
                raise ValueError(f"out.{name} must be {list(size)}")
    status = lib.page_select(q.data_ptr(), q_stride, bounds, exp, start, lens, table, shape, cfg,
                             out.q_start.data_ptr(), out.kv_len.data_ptr(), out.page_table.data_ptr(),
                             None if out.index is None else out.index.data_ptr(), st)
    if status:
        _check("page_select", status)
    return out


def kv_pages_copy(cache: PagedKVCache, src, dst, *, digest: PageDigest | None = None, stream=None) -> None:
    """Page dst[i] becomes a copy of page src[i] (int32 [n] on the device): keys, values, scales, and
    the digest if given.  A fork copies the partly filled last page of a sequence and shares the others in
    its table; a compaction moves pages and rewrites the tables.  Each page stands in dst at most once, and
    none of them in src; entries outside the cache are skipped."""
    lib = _lib or load()
    k, v, ks, vs, (n_pages, page_size, H_kv, D), dtype, dev = _cache_args(cache)
    st = _call_stream(dev, stream)
    if st is None:
        with _on(dev, stream):
            return kv_pages_copy(cache, src, dst, digest=digest)
    bounds = exp = None
    if digest is not None:
        bounds, exp = _digest_of_cache(digest, n_pages, page_size, H_kv, D, dev)
    s, d = _index(src, "src", 1, dev), _index(dst, "dst", 1, dev)
    n = src.shape[0]
    if dst.shape[0] != n:
        raise ValueError("src and dst must have the same length")
    shape, _ = _paged_shape(1, 0, 1, n_pages, page_size, H_kv, H_kv, D, dtype)
    status = lib.kv_pages_copy(s, d, n, shape, k, v, ks, vs, bounds, exp, st)
    if status:
        _check("kv_pages_copy", status)
