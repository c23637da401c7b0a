"""Thin Python binding of libsparsepr.so (the C ABI in include/sparsepr.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. torch is used for device memory and streams. Importing this module
loads the in-tree library and raises if it has not been built.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsparsepr.so")
MAX_HEADS = 256

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_NUMERIC = range(7)
ERR_CAPACITY = 7
BF16, F32 = 0, 1
# sparsepr_params.partition; the parameter dicts name the mode as the oracle does
PARTITION_MODES = dict(response=0, semantic=1, coclustering=2)

EXPORTED = ("sparsepr_workspace_bytes", "sparsepr_status_string", "sparsepr_partition",
            "sparsepr_permute", "sparsepr_route", "sparsepr_route_width",
            "sparsepr_block_sparse_attn", "sparsepr_probe_correct", "sparsepr_read_stats",
            "sparsepr_reset_stats", "sparsepr_check_wait_limit", "sparsepr_route_noalloc",
            "sparsepr_workspace_region", "sparsepr_probe_diagnostics",
            "sparsepr_support_expansion", "sparsepr_density_profile", "sparsepr_attention",
            "sparsepr_check_reciprocal", "sparsepr_window_workspace_bytes",
            "sparsepr_window_attention", "sparsepr_cache_workspace_bytes",
            "sparsepr_cache_reserve", "sparsepr_cache_append", "sparsepr_cache_attention",
            "sparsepr_cache_fork", "sparsepr_cache_free", "sparsepr_cache_evict",
            "sparsepr_cache_compact")


class Params(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("n_text", ctypes.c_int32), ("Ck", ctypes.c_int32), ("Cq", ctypes.c_int32),
                ("Ms", ctypes.c_int32), ("n_eig", ctypes.c_int32),
                ("kmeans_iters", ctypes.c_int32), ("M", ctypes.c_int32), ("r", ctypes.c_int32),
                ("partition", ctypes.c_int32), ("lam", ctypes.c_double), ("scale", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("keep", ctypes.POINTER(ctypes.c_double))]


class CallBuffers(ctypes.Structure):
    """sparsepr_call_buffers: device pointers of every output of one call."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "label_q", "label_k", "perm_q", "perm_k", "off_q", "off_k", "qp", "kp", "vp", "csr",
        "k_per_head", "o_sparse", "pairs_sparse", "probes", "pairs_exec", "fit")]


class Stats(ctypes.Structure):
    _fields_ = [("status", ctypes.c_uint32), ("H", ctypes.c_int32),
                ("key_passes", ctypes.c_int32 * MAX_HEADS),
                ("query_passes", ctypes.c_int32 * MAX_HEADS),
                ("pairs_sparse", ctypes.c_int64 * MAX_HEADS),
                ("pairs_exec", ctypes.c_int64 * MAX_HEADS),
                ("recheck_rows", ctypes.c_int64 * 2),
                ("eig_sweeps", ctypes.c_int32 * 2), ("near_ties", ctypes.c_int64 * 2)]


class Visibility(ctypes.Structure):
    """sparsepr_visibility: which keys a query sees, by frames."""
    _fields_ = [(n, ctypes.c_int32) for n in ("frame", "window", "sinks", "causal")]


class WindowParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d")] + [
        ("see", Visibility), ("scale", ctypes.c_double)]


class CacheParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hkv", "d", "page", "n_pages", "max_pages")]


class CachePointers(ctypes.Structure):
    """sparsepr_cache: device pointers of a cache."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k8", "v8", "k_scale", "v_scale", "table", "len",
                                               "ref")]


class CacheAttentionParams(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("Nq", ctypes.c_int32), ("see", Visibility),
                ("scale", ctypes.c_double)]


class SparsePRError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s: %s (status %d)" % (where, status_string(code), code))
        self.code = code


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError("libsparsepr.so is not built; run "
                          "`python -m free_block_sparse_eigenbasis_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, V, I32P, I64P = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    PP = ctypes.POINTER(Params)
    st = ctypes.c_int
    sz = ctypes.c_size_t
    lib.sparsepr_workspace_bytes.argtypes = [PP]
    lib.sparsepr_workspace_bytes.restype = sz
    lib.sparsepr_status_string.argtypes = [st]
    lib.sparsepr_status_string.restype = ctypes.c_char_p
    lib.sparsepr_route_width.argtypes = [PP]
    lib.sparsepr_route_width.restype = ctypes.c_int32
    lib.sparsepr_partition.argtypes = [P, P, st, PP, I32P, I32P, V, sz, V]
    lib.sparsepr_permute.argtypes = [P, P, P, st, PP, I32P, I32P, I32P, I32P, I32P, I32P, P, P, P,
                                     V, sz, V]
    lib.sparsepr_route.argtypes = [P, P, st, PP, I32P, I32P, I32P, I32P, V, sz, V]
    lib.sparsepr_block_sparse_attn.argtypes = [P, P, P, st, PP, I32P, I32P, I32P, I32P, P, I64P,
                                               V, sz, V]
    lib.sparsepr_probe_correct.argtypes = [P, P, P, st, PP, I32P, I32P, P, I64P, P, I32P, I64P, P,
                                           V, sz, V]
    lib.sparsepr_route_noalloc.argtypes = [P, P, st, PP, I32P, I32P, I32P, I32P, V]
    lib.sparsepr_route_noalloc.restype = st
    lib.sparsepr_workspace_region.argtypes = [PP, ctypes.c_char_p, ctypes.POINTER(sz),
                                              ctypes.POINTER(sz)]
    lib.sparsepr_workspace_region.restype = st
    lib.sparsepr_probe_diagnostics.argtypes = [PP, I32P, P, P, P, V, sz, V]
    lib.sparsepr_probe_diagnostics.restype = st
    lib.sparsepr_support_expansion.argtypes = [P, P, st, PP, I32P, I32P, ctypes.c_double,
                                               ctypes.c_int32, P, P, V, sz, V]
    lib.sparsepr_support_expansion.restype = st
    lib.sparsepr_density_profile.argtypes = [P, P, st, PP, ctypes.c_double, ctypes.c_int32, P, V,
                                             sz, V]
    lib.sparsepr_density_profile.restype = st
    lib.sparsepr_attention.argtypes = [P, P, P, st, PP, ctypes.POINTER(CallBuffers), P, V, sz, V]
    lib.sparsepr_attention.restype = st
    lib.sparsepr_read_stats.argtypes = [V, ctypes.POINTER(Stats)]
    lib.sparsepr_reset_stats.argtypes = [V, V]
    lib.sparsepr_check_wait_limit.argtypes = [V, V]
    lib.sparsepr_check_reciprocal.argtypes = [P, ctypes.c_int64, P, V]
    lib.sparsepr_check_reciprocal.restype = st
    WP, CP, CC = (ctypes.POINTER(x) for x in (WindowParams, CacheParams, CachePointers))
    CA, SEE, I32 = ctypes.POINTER(CacheAttentionParams), ctypes.POINTER(Visibility), ctypes.c_int32
    lib.sparsepr_window_workspace_bytes.argtypes = [WP, st]
    lib.sparsepr_window_workspace_bytes.restype = sz
    lib.sparsepr_cache_workspace_bytes.argtypes = [CP, CA]
    lib.sparsepr_cache_workspace_bytes.restype = sz
    for name, args in (
            ("window_attention", [P, P, P, st, WP, I32P, I32P, P, P]),
            ("cache_reserve", [CP, CC, I32P, I32P]),
            ("cache_append", [P, P, st, I32, CP, CC, I32P, I32P]),
            ("cache_attention", [P, st, CP, CC, CA, I32P, P, P]),
            ("cache_fork", [CP, CC, I32P, I32P, I32]),
            ("cache_free", [CP, CC, I32P, I32]),
            ("cache_evict", [CP, CC, SEE]),
            ("cache_compact", [CP, CC, I32P])):
        fn = getattr(lib, "sparsepr_" + name)
        fn.argtypes = args + [V, sz, V]
        fn.restype = st
    for name in ("sparsepr_partition", "sparsepr_permute", "sparsepr_route",
                 "sparsepr_block_sparse_attn", "sparsepr_probe_correct", "sparsepr_read_stats",
                 "sparsepr_reset_stats", "sparsepr_check_wait_limit"):
        getattr(lib, name).restype = st
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.sparsepr_status_string(code).decode()


def make_params(p: dict):
    """ctypes Params from a plain parameter dict; returns (params, keep array)
    -- keep the second value alive for as long as the first is used."""
    H = int(p["H"])
    keep = p["keep"]
    if not isinstance(keep, (list, tuple)):
        keep = [keep] * H
    arr = (ctypes.c_double * max(1, H))(*[float(x) for x in keep[:H]])
    prm = Params(H=H, N=int(p["N"]), d=int(p["d"]), n_text=int(p.get("n_text", 0)),
                 Ck=int(p["Ck"]), Cq=int(p["Cq"]), Ms=int(p["Ms"]), n_eig=int(p["n_eig"]),
                 kmeans_iters=int(p["kmeans_iters"]), M=int(p["M"]), r=int(p["r"]),
                 partition=PARTITION_MODES[p.get("partition", "response")],
                 lam=float(p["lam"]), scale=float(p.get("scale", 0.0)),
                 seed=int(p["seed"]) & ((1 << 64) - 1),
                 keep=ctypes.cast(arr, ctypes.POINTER(ctypes.c_double)))
    return prm, arr


_DEVICE_TYPE = "cuda"  # tensors handed to the library live on this device type


def _arg(t, name: str, shape=None, dtype=None):
    """Device pointer of a tensor argument after the checks the C ABI cannot
    make from a bare pointer: shape, dtype, dense row-major layout and a CUDA
    device. Raises ValueError / TypeError before anything is enqueued."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (row-major)" % name)
    if t.device.type != _DEVICE_TYPE:
        raise ValueError("%s must be a CUDA tensor" % name)
    return ctypes.c_void_p(t.data_ptr())


def _ws(ws, name: str = "ws"):
    """(pointer, bytes) of the workspace: a contiguous CUDA byte buffer."""
    return _arg(ws, name, (ws.numel(),) if isinstance(ws, torch.Tensor) else None,
                torch.uint8), ws.numel()


def _dims(p: dict):
    """H, N, d and the group-offset widths (text tokens add one group per side)."""
    H, N, d = int(p["H"]), int(p["N"]), int(p["d"])
    text = 1 if int(p.get("n_text", 0)) > 0 else 0
    return H, N, d, int(p["Cq"]) + text + 1, int(p["Ck"]) + text + 1


def _qkv(p: dict, names_tensors):
    """Checks the [H, N, d] inputs of one dtype (bf16 or fp32, set by the first)."""
    H, N, d = int(p["H"]), int(p["N"]), int(p["d"])
    dt = names_tensors[0][1].dtype if isinstance(names_tensors[0][1], torch.Tensor) else None
    ptrs = [_arg(t, n, (H, N, d), dt) for n, t in names_tensors]
    return ptrs, _dtype_code(names_tensors[0][1])


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise TypeError("Q/K/V must be bf16 or fp32")


def _check(code: int, where: str):
    if code != OK:
        raise SparsePRError(code, where)


def workspace_bytes(p: dict) -> int:
    prm, keep = make_params(p)
    return int(lib.sparsepr_workspace_bytes(ctypes.byref(prm)))


def route_width(p: dict) -> int:
    prm, keep = make_params(p)
    return int(lib.sparsepr_route_width(ctypes.byref(prm)))


# ---- the five calls, same names as the C ABI --------------------------------

I32, I64 = torch.int32, torch.int64


def sparsepr_partition(q, k, p, label_q, label_k, ws, stream=None):
    prm, keep = make_params(p)
    H, N, d, _, _ = _dims(p)
    (pq, pk), dt = _qkv(p, [("q", q), ("k", k)])
    wp, wb = _ws(ws)
    _check(lib.sparsepr_partition(pq, pk, dt, ctypes.byref(prm),
                                  _arg(label_q, "label_q", (H, N), I32),
                                  _arg(label_k, "label_k", (H, N), I32), wp, wb,
                                  _stream(stream)), "sparsepr_partition")


def sparsepr_permute(q, k, v, p, label_q, label_k, perm_q, perm_k, off_q, off_k, qp, kp, vp, ws,
                     stream=None):
    prm, keep = make_params(p)
    H, N, d, wq, wk = _dims(p)
    (pq, pk, pv, pqp, pkp, pvp), dt = _qkv(p, [("q", q), ("k", k), ("v", v), ("qp", qp),
                                              ("kp", kp), ("vp", vp)])
    wp, wb = _ws(ws)
    _check(lib.sparsepr_permute(pq, pk, pv, dt, ctypes.byref(prm),
                                _arg(label_q, "label_q", (H, N), I32),
                                _arg(label_k, "label_k", (H, N), I32),
                                _arg(perm_q, "perm_q", (H, N), I32),
                                _arg(perm_k, "perm_k", (H, N), I32),
                                _arg(off_q, "off_q", (H, wq), I32),
                                _arg(off_k, "off_k", (H, wk), I32), pqp, pkp, pvp, wp, wb,
                                _stream(stream)), "sparsepr_permute")


def _route_args(qp, kp, p, off_q, off_k, csr, k_per_head):
    H, N, d, wq, wk = _dims(p)
    (pq, pk), dt = _qkv(p, [("qp", qp), ("kp", kp)])
    return (pq, pk, dt, _arg(off_q, "off_q", (H, wq), I32), _arg(off_k, "off_k", (H, wk), I32),
            _arg(csr, "csr", (H, int(p["Cq"]), route_width(p)), I32),
            _arg(k_per_head, "k_per_head", (H,), I32))


def sparsepr_route(qp, kp, p, off_q, off_k, csr, k_per_head, ws, stream=None):
    prm, keep = make_params(p)
    pq, pk, dt, poq, pok, pcsr, pkh = _route_args(qp, kp, p, off_q, off_k, csr, k_per_head)
    wp, wb = _ws(ws)
    _check(lib.sparsepr_route(pq, pk, dt, ctypes.byref(prm), poq, pok, pcsr, pkh, wp, wb,
                              _stream(stream)), "sparsepr_route")


def sparsepr_route_noalloc(qp, kp, p, off_q, off_k, csr, k_per_head, stream=None):
    """sparsepr_route without a workspace (its scratch is a fixed device array
    inside the library); for callers that cannot allocate device memory."""
    prm, keep = make_params(p)
    pq, pk, dt, poq, pok, pcsr, pkh = _route_args(qp, kp, p, off_q, off_k, csr, k_per_head)
    _check(lib.sparsepr_route_noalloc(pq, pk, dt, ctypes.byref(prm), poq, pok, pcsr, pkh,
                                      _stream(stream)), "sparsepr_route_noalloc")


def sparsepr_block_sparse_attn(qp, kp, vp, p, off_q, off_k, csr, k_per_head, o_sparse,
                               pairs_sparse, ws, stream=None):
    prm, keep = make_params(p)
    H, N, d, _, _ = _dims(p)
    pq, pk, dt, poq, pok, pcsr, pkh = _route_args(qp, kp, p, off_q, off_k, csr, k_per_head)
    (pv,), _ = _qkv(p, [("vp", vp)])
    if vp.dtype != qp.dtype:
        raise TypeError("vp has dtype %s, expected %s" % (vp.dtype, qp.dtype))
    wp, wb = _ws(ws)
    _check(lib.sparsepr_block_sparse_attn(pq, pk, pv, dt, ctypes.byref(prm), poq, pok, pcsr, pkh,
                                          _arg(o_sparse, "o_sparse", (H, N, d), torch.float32),
                                          _arg(pairs_sparse, "pairs_sparse", (H,), I64), wp, wb,
                                          _stream(stream)), "sparsepr_block_sparse_attn")


def sparsepr_probe_correct(qp, kp, vp, p, off_q, perm_q, o_sparse, pairs_sparse, out, probes,
                           pairs_exec, ws, fit=None, stream=None):
    prm, keep = make_params(p)
    H, N, d, wq, _ = _dims(p)
    M = int(p["M"])
    (pq, pk, pv, pout), dt = _qkv(p, [("qp", qp), ("kp", kp), ("vp", vp), ("out", out)])
    wp, wb = _ws(ws)
    _check(lib.sparsepr_probe_correct(pq, pk, pv, dt, ctypes.byref(prm),
                                      _arg(off_q, "off_q", (H, wq), I32),
                                      _arg(perm_q, "perm_q", (H, N), I32),
                                      _arg(o_sparse, "o_sparse", (H, N, d), torch.float32),
                                      _arg(pairs_sparse, "pairs_sparse", (H,), I64), pout,
                                      _arg(probes, "probes", (H, M) if M > 0 else None, I32),
                                      _arg(pairs_exec, "pairs_exec", (H,), I64),
                                      None if fit is None else
                                      _arg(fit, "fit", (H, d * d + d), torch.float64),
                                      wp, wb, _stream(stream)), "sparsepr_probe_correct")


def sparsepr_probe_diagnostics(p, probes, mass, error, energy, ws, stream=None):
    """Retained mass and error of every probe row, and the residual energy
    split per head (see include/sparsepr.h)."""
    prm, keep = make_params(p)
    H, M = int(p["H"]), int(p["M"])
    f64 = torch.float64
    _check(lib.sparsepr_probe_diagnostics(ctypes.byref(prm), _arg(probes, "probes", (H, M), I32),
                                          _arg(mass, "mass", (H, M), f64),
                                          _arg(error, "error", (H, M), f64),
                                          _arg(energy, "energy", (H, 4), f64), *_ws(ws),
                                          _stream(stream)), "sparsepr_probe_diagnostics")


def sparsepr_support_expansion(qp, kp, p, off_q, off_k, tau, group_stride, individual,
                               aggregate, ws, stream=None):
    """Mean individual and aggregate (union) support size, in key groups, of
    every group_stride-th video query group (see include/sparsepr.h)."""
    prm, keep = make_params(p)
    H, N, d, wq, wk = _dims(p)
    Cq = int(p["Cq"])
    (pq, pk), dt = _qkv(p, [("qp", qp), ("kp", kp)])
    f64 = torch.float64
    _check(lib.sparsepr_support_expansion(pq, pk, dt, ctypes.byref(prm),
                                          _arg(off_q, "off_q", (H, wq), I32),
                                          _arg(off_k, "off_k", (H, wk), I32), float(tau),
                                          int(group_stride),
                                          _arg(individual, "individual", (H, Cq), f64),
                                          _arg(aggregate, "aggregate", (H, Cq), f64), *_ws(ws),
                                          _stream(stream)), "sparsepr_support_expansion")


def sparsepr_density_profile(q, k, p, tau, row_stride, density, ws, stream=None):
    """Mean tau-mass density of every row_stride-th video row, per head."""
    prm, keep = make_params(p)
    H = int(p["H"])
    (pq, pk), dt = _qkv(p, [("q", q), ("k", k)])
    _check(lib.sparsepr_density_profile(pq, pk, dt, ctypes.byref(prm), float(tau), int(row_stride),
                                        _arg(density, "density", (H,), torch.float64), *_ws(ws),
                                        _stream(stream)), "sparsepr_density_profile")


def sparsepr_reset_stats(ws, stream=None):
    _check(lib.sparsepr_reset_stats(_ws(ws)[0], _stream(stream)), "sparsepr_reset_stats")


def sparsepr_check_wait_limit(ws, stream=None):
    _check(lib.sparsepr_check_wait_limit(_ws(ws)[0], _stream(stream)), "sparsepr_check_wait_limit")


def sparsepr_check_reciprocal(x, stream=None):
    """Distance in ulp of the multisection's reciprocal from the correctly
    rounded 1/x, for a 1-D fp64 device tensor x; returns a tensor like x."""
    if x.dtype != torch.float64 or x.dim() != 1 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x: a contiguous 1-D float64 CUDA tensor")
    err = torch.empty_like(x)
    _check(lib.sparsepr_check_reciprocal(x.data_ptr(), x.numel(), err.data_ptr(), _stream(stream)),
           "sparsepr_check_reciprocal")
    return err


# ---- windowed attention and the 8-bit cache ---------------------------------

F8 = torch.float8_e4m3fn


def _visibility(p: dict) -> Visibility:
    return Visibility(p.get("frame", 1), p.get("window", 0), p.get("sinks", 0), p.get("causal", 1))


def make_window_params(p: dict) -> WindowParams:
    """ctypes parameters of the windowed attention from a plain dict (B, Hq,
    Hkv, Nq, Nk, d; frame, window, sinks, causal as in sparsepr_visibility,
    by default token-causal without a window; scale)."""
    return WindowParams(p["B"], p["Hq"], p["Hkv"], p["Nq"], p["Nk"], p["d"], _visibility(p),
                        p.get("scale", 0.0))


def make_cache_params(p: dict) -> CacheParams:
    return CacheParams(p["B"], p["Hkv"], p["d"], p["page"], p["n_pages"], p["max_pages"])


def make_cache_attention_params(a: dict) -> CacheAttentionParams:
    return CacheAttentionParams(a["Hq"], a["Nq"], _visibility(a), a.get("scale", 0.0))


@dataclass
class Cache:
    """A paged cache of keys and values in e4m3 (see include/sparsepr.h), all
    tensors owned by torch."""
    k8: torch.Tensor       # [n_pages, Hkv, page, d] float8_e4m3fn
    v8: torch.Tensor
    k_scale: torch.Tensor  # [n_pages, Hkv] fp32
    v_scale: torch.Tensor
    table: torch.Tensor    # [B, max_pages] int32, -1 = no page
    len: torch.Tensor      # [B] int32
    ref: torch.Tensor      # [n_pages] int32


def allocate_cache(p: dict, device="cuda") -> Cache:
    """An empty cache."""
    if int(lib.sparsepr_cache_workspace_bytes(ctypes.byref(make_cache_params(p)), None)) == 0:
        raise SparsePRError(ERR_INVALID_ARG, "allocate_cache")
    pages, shape = (int(p["n_pages"]), int(p["Hkv"])), (int(p["page"]), int(p["d"]))
    i32 = dict(dtype=torch.int32, device=device)
    return Cache(
        k8=torch.zeros(pages + shape, dtype=torch.uint8, device=device).view(F8),
        v8=torch.zeros(pages + shape, dtype=torch.uint8, device=device).view(F8),
        k_scale=torch.ones(pages, dtype=torch.float32, device=device),
        v_scale=torch.ones(pages, dtype=torch.float32, device=device),
        table=torch.full((int(p["B"]), int(p["max_pages"])), -1, **i32),
        len=torch.zeros(int(p["B"]), **i32), ref=torch.zeros(int(p["n_pages"]), **i32))


def _cleared_workspace(nbytes: int, where: str, device) -> torch.Tensor:
    if nbytes == 0:
        raise SparsePRError(ERR_INVALID_ARG, where)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def allocate_window_workspace(p: dict, dtype: torch.dtype, device="cuda") -> torch.Tensor:
    """Workspace of sparsepr_window_attention with a clear status word."""
    prm = make_window_params(p)
    return _cleared_workspace(int(lib.sparsepr_window_workspace_bytes(
        ctypes.byref(prm), _DTYPE_CODES.get(dtype, -1))), "window_workspace_bytes", device)


def allocate_cache_workspace(p: dict, attn: Optional[dict] = None, device="cuda") -> torch.Tensor:
    """Workspace of the cache calls (with attn: of that attention too) with a
    clear status word."""
    prm = make_cache_params(p)
    a = None if attn is None else ctypes.byref(make_cache_attention_params(attn))
    return _cleared_workspace(int(lib.sparsepr_cache_workspace_bytes(ctypes.byref(prm), a)),
                              "cache_workspace_bytes", device)


_DTYPE_CODES = {torch.bfloat16: BF16, torch.float32: F32}


def _ptr(t, name, shape, dtype, dev):
    """Device pointer (int) of a tensor argument on device index dev: the checks
    of _arg in one expression, _arg itself for the message when one fails."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.is_contiguous() and t.get_device() == dev
            and (dev >= 0 or _DEVICE_TYPE == "cpu")):
        return t.data_ptr()
    _arg(t, name, shape, dtype)
    raise ValueError("%s must be on the device of the workspace" % name)


# the current stream's handle without a Stream object around it, where torch has that
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(where: str, fn, args, ws, dev, stream):
    """One library call on the device of its tensors and, unless a stream is
    given, on that device's current stream."""
    if not (ws.dtype is torch.uint8 and ws.is_contiguous() and (dev >= 0 or _DEVICE_TYPE == "cpu")):
        _ws(ws)
    wp, wb = ws.data_ptr(), ws.numel()
    if dev < 0 or dev == torch.cuda.current_device():
        st = _current_stream(dev) if stream is None else stream.cuda_stream
        code = fn(*args, wp, wb, st)
    else:
        with torch.cuda.device(dev):
            st = (torch.cuda.current_stream() if stream is None else stream).cuda_stream
            code = fn(*args, wp, wb, st)
    if code != OK:
        raise SparsePRError(code, where)


def _device(ws) -> int:
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a torch.Tensor")
    return ws.get_device()


def sparsepr_window_attention(q, k, v, p: dict, out, ws, lse=None, n_q=None, n_k=None,
                              stream=None):
    """Attention with a sliding window of frames and sink frames: q, out
    [B, Hq, Nq, d], k, v [B, Hkv, Nk, d] bf16 or fp32; lse [B, Hq, Nq] fp32,
    n_q and n_k [B] int32, each optional (see include/sparsepr.h)."""
    prm = make_window_params(p)
    B, Hq, Nq, d, dev, t = prm.B, prm.Hq, prm.Nq, prm.d, _device(ws), q.dtype
    dt = _dtype_code(q)
    rows, keys = (B, Hq, Nq, d), (B, prm.Hkv, prm.Nk, d)
    _launch("sparsepr_window_attention", lib.sparsepr_window_attention,
            (_ptr(q, "q", rows, t, dev), _ptr(k, "k", keys, t, dev), _ptr(v, "v", keys, t, dev),
             dt, ctypes.byref(prm), None if n_q is None else _ptr(n_q, "n_q", (B,), I32, dev),
             None if n_k is None else _ptr(n_k, "n_k", (B,), I32, dev),
             _ptr(out, "out", rows, t, dev),
             None if lse is None else _ptr(lse, "lse", (B, Hq, Nq), torch.float32, dev)),
            ws, dev, stream)


def _cache(p: dict, c: Cache, ws):
    """(parameters, their reference, reference to the pointers, device)"""
    B, H, d, page, N, mp = p["B"], p["Hkv"], p["d"], p["page"], p["n_pages"], p["max_pages"]
    prm, dev = CacheParams(B, H, d, page, N, mp), _device(ws)
    k8, v8, ks, vs, table, length, ref = (c.k8, c.v8, c.k_scale, c.v_scale, c.table, c.len, c.ref)
    f32 = torch.float32
    try:  # the checks of _ptr for all seven at once
        fine = (k8.shape == v8.shape == (N, H, page, d) and ks.shape == vs.shape == (N, H)
                and table.shape == (B, mp) and length.shape == (B,) and ref.shape == (N,)
                and k8.dtype is F8 and v8.dtype is F8 and ks.dtype is f32 and vs.dtype is f32
                and table.dtype is I32 and length.dtype is I32 and ref.dtype is I32
                and k8.is_contiguous() and v8.is_contiguous() and ks.is_contiguous()
                and vs.is_contiguous() and table.is_contiguous() and length.is_contiguous()
                and ref.is_contiguous() and (dev >= 0 or _DEVICE_TYPE == "cpu")
                and dev == k8.get_device() == v8.get_device() == ks.get_device()
                == vs.get_device() == table.get_device() == length.get_device()
                == ref.get_device())
    except AttributeError:
        fine = False
    if not fine:
        for t, name, shape, dtype in (
                (k8, "k8", (N, H, page, d), F8), (v8, "v8", (N, H, page, d), F8),
                (ks, "k_scale", (N, H), f32), (vs, "v_scale", (N, H), f32),
                (table, "table", (B, mp), I32), (length, "len", (B,), I32), (ref, "ref", (N,), I32)):
            _ptr(t, name, shape, dtype, dev)
    ptr = CachePointers(k8.data_ptr(), v8.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                        table.data_ptr(), length.data_ptr(), ref.data_ptr())
    return prm, ctypes.byref(prm), ctypes.byref(ptr), dev


def sparsepr_cache_reserve(n_new, p: dict, cache: Cache, start, ws, stream=None):
    """Pages for n_new [B] int32 more tokens per sequence; start [B] int32
    receives the lengths before (-1 throughout if there is no room)."""
    prm, pp, cp, dev = _cache(p, cache, ws)
    _launch("sparsepr_cache_reserve", lib.sparsepr_cache_reserve,
            (pp, cp, _ptr(n_new, "n_new", (prm.B,), I32, dev),
             _ptr(start, "start", (prm.B,), I32, dev)), ws, dev, stream)


def sparsepr_cache_append(k, v, p: dict, cache: Cache, start, n_new, ws, stream=None):
    """Write the tokens k, v [B, Hkv, T, d] (bf16 or fp32; the first n_new[b]
    of each sequence, all T where n_new is None) at start[b] in 8 bits."""
    prm, pp, cp, dev = _cache(p, cache, ws)
    dt = _dtype_code(k)
    shape = (prm.B, prm.Hkv, k.shape[2] if k.dim() == 4 else -1, prm.d)
    _launch("sparsepr_cache_append", lib.sparsepr_cache_append,
            (_ptr(k, "k", shape, k.dtype, dev), _ptr(v, "v", shape, k.dtype, dev), dt, shape[2],
             pp, cp, _ptr(start, "start", (prm.B,), I32, dev),
             None if n_new is None else _ptr(n_new, "n_new", (prm.B,), I32, dev)), ws, dev, stream)


def sparsepr_cache_attention(q, p: dict, cache: Cache, attn: dict, out, ws, lse=None, n_q=None,
                             stream=None):
    """Attention of q [B, Hq, Nq, d] over the cached tokens; attn: Hq, Nq and
    the visibility (see include/sparsepr.h)."""
    prm, pp, cp, dev = _cache(p, cache, ws)
    a = make_cache_attention_params(attn)
    rows = (prm.B, a.Hq, a.Nq, prm.d)
    dt = _dtype_code(q)
    _launch("sparsepr_cache_attention", lib.sparsepr_cache_attention,
            (_ptr(q, "q", rows, q.dtype, dev), dt, pp, cp, ctypes.byref(a),
             None if n_q is None else _ptr(n_q, "n_q", (prm.B,), I32, dev),
             _ptr(out, "out", rows, q.dtype, dev),
             None if lse is None else _ptr(lse, "lse", rows[:3], torch.float32, dev)), ws, dev,
            stream)


def sparsepr_cache_fork(src, dst, p: dict, cache: Cache, ws, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] that shares its pages."""
    _, pp, cp, dev = _cache(p, cache, ws)
    n = src.numel()
    _launch("sparsepr_cache_fork", lib.sparsepr_cache_fork,
            (pp, cp, _ptr(src, "src", (n,), I32, dev), _ptr(dst, "dst", (n,), I32, dev), n), ws,
            dev, stream)


def sparsepr_cache_free(seq, p: dict, cache: Cache, ws, stream=None):
    """Empty the sequences named in seq [n] int32."""
    _, pp, cp, dev = _cache(p, cache, ws)
    n = seq.numel()
    _launch("sparsepr_cache_free", lib.sparsepr_cache_free,
            (pp, cp, _ptr(seq, "seq", (n,), I32, dev), n), ws, dev, stream)


def sparsepr_cache_evict(see: dict, p: dict, cache: Cache, ws, stream=None):
    """Give up the pages that no later query with this causal, windowed
    visibility can see."""
    _, pp, cp, dev = _cache(p, cache, ws)
    v = _visibility(see)
    _launch("sparsepr_cache_evict", lib.sparsepr_cache_evict, (pp, cp, ctypes.byref(v)), ws, dev,
            stream)


def sparsepr_cache_compact(p: dict, cache: Cache, n_used, ws, stream=None):
    """Move the pages in use to the front of the pool; n_used [1] int32
    receives their number."""
    _, pp, cp, dev = _cache(p, cache, ws)
    _launch("sparsepr_cache_compact", lib.sparsepr_cache_compact,
            (pp, cp, _ptr(n_used, "n_used", (1,), I32, dev)), ws, dev, stream)


_REGION_DTYPES = dict(init_k=torch.int32, init_q=torch.int32, zplanes=torch.bfloat16,
                      xnk=torch.float32)


def sparsepr_workspace_region(p: dict, name: str):
    """(byte offset, bytes) of a named intermediate-result region of the
    workspace for these parameters."""
    prm, keep = make_params(p)
    off, nb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.sparsepr_workspace_region(ctypes.byref(prm), name.encode(), ctypes.byref(off),
                                         ctypes.byref(nb)), "sparsepr_workspace_region")
    return int(off.value), int(nb.value)


def workspace_view(ws, p: dict, name: str) -> torch.Tensor:
    """The named region of `ws` as a flat tensor of its element type (fp64;
    int32 for the initial centroid rows, bf16 for the key planes, fp32 for
    the key row norms); a view, no copy."""
    off, nb = sparsepr_workspace_region(p, name)
    return ws[off:off + nb].view(_REGION_DTYPES.get(name, torch.float64))


def sparsepr_read_stats(ws) -> dict:
    s = Stats()
    _check(lib.sparsepr_read_stats(_ws(ws)[0], ctypes.byref(s)), "sparsepr_read_stats")
    H = max(0, min(s.H, MAX_HEADS))
    return dict(status=int(s.status), H=H, key_passes=list(s.key_passes[:H]),
                query_passes=list(s.query_passes[:H]), pairs_sparse=list(s.pairs_sparse[:H]),
                pairs_exec=list(s.pairs_exec[:H]), recheck_rows=list(s.recheck_rows),
                eig_sweeps=list(s.eig_sweeps), near_ties=list(s.near_ties))


# ---- buffers + the whole call ----------------------------------------------

@dataclass
class Buffers:
    """Device buffers of one attention call (all owned by torch)."""
    ws: torch.Tensor
    label_q: torch.Tensor
    label_k: torch.Tensor
    perm_q: torch.Tensor
    perm_k: torch.Tensor
    off_q: torch.Tensor
    off_k: torch.Tensor
    qp: torch.Tensor
    kp: torch.Tensor
    vp: torch.Tensor
    csr: torch.Tensor
    k_per_head: torch.Tensor
    o_sparse: torch.Tensor
    pairs_sparse: torch.Tensor
    out: torch.Tensor
    probes: torch.Tensor
    pairs_exec: torch.Tensor
    fit: Optional[torch.Tensor]


def allocate(p: dict, dtype: torch.dtype, device="cuda", with_fit=False) -> Buffers:
    H, N, d = int(p["H"]), int(p["N"]), int(p["d"])
    Ck, Cq, M = int(p["Ck"]), int(p["Cq"]), int(p["M"])
    text = 1 if int(p.get("n_text", 0)) > 0 else 0  # text tokens form one extra group per side
    wsb = workspace_bytes(p)
    if wsb == 0:
        raise SparsePRError(ERR_INVALID_ARG, "workspace_bytes")
    kmax = route_width(p)
    i32 = dict(dtype=torch.int32, device=device)
    return Buffers(
        ws=torch.empty(wsb, dtype=torch.uint8, device=device),
        label_q=torch.empty((H, N), **i32), label_k=torch.empty((H, N), **i32),
        perm_q=torch.empty((H, N), **i32), perm_k=torch.empty((H, N), **i32),
        off_q=torch.empty((H, Cq + text + 1), **i32), off_k=torch.empty((H, Ck + text + 1), **i32),
        qp=torch.empty((H, N, d), dtype=dtype, device=device),
        kp=torch.empty((H, N, d), dtype=dtype, device=device),
        vp=torch.empty((H, N, d), dtype=dtype, device=device),
        csr=torch.empty((H, Cq, kmax), **i32), k_per_head=torch.empty(H, **i32),
        o_sparse=torch.empty((H, N, d), dtype=torch.float32, device=device),
        pairs_sparse=torch.empty(H, dtype=torch.int64, device=device),
        out=torch.empty((H, N, d), dtype=dtype, device=device),
        probes=torch.empty((H, max(M, 1)), **i32),
        pairs_exec=torch.empty(H, dtype=torch.int64, device=device),
        fit=torch.empty((H, d * d + d), dtype=torch.float64, device=device) if with_fit else None)


def attention(q, k, v, p: dict, bufs: Optional[Buffers] = None, stream=None) -> Buffers:
    """One SparsePR attention call on [H, N, d] device tensors: the five
    library calls in order on one stream. Returns the buffers (bufs.out is
    the corrected output in the original token order)."""
    if bufs is None:
        bufs = allocate(p, q.dtype, q.device)
    b = bufs
    sparsepr_partition(q, k, p, b.label_q, b.label_k, b.ws, stream)
    sparsepr_permute(q, k, v, p, b.label_q, b.label_k, b.perm_q, b.perm_k, b.off_q, b.off_k, b.qp,
                     b.kp, b.vp, b.ws, stream)
    sparsepr_route(b.qp, b.kp, p, b.off_q, b.off_k, b.csr, b.k_per_head, b.ws, stream)
    sparsepr_block_sparse_attn(b.qp, b.kp, b.vp, p, b.off_q, b.off_k, b.csr, b.k_per_head,
                               b.o_sparse, b.pairs_sparse, b.ws, stream)
    sparsepr_probe_correct(b.qp, b.kp, b.vp, p, b.off_q, b.perm_q, b.o_sparse, b.pairs_sparse,
                           b.out, b.probes, b.pairs_exec, b.ws, b.fit, stream)
    return b


def sparsepr_attention(q, k, v, p: dict, bufs: Buffers, stream=None) -> Buffers:
    """The whole call in one library entry point (sparsepr_attention): the
    probe fit runs on a side stream beside the attention of all rows. Fills
    the same buffers as attention(); bufs.out is the output."""
    prm, keep = make_params(p)
    H, N, d, oq, ok = _dims(p)
    (pq, pk, pv), dt = _qkv(p, [("q", q), ("k", k), ("v", v)])
    b = bufs
    I32T = torch.int32
    ptr = lambda t, n, shape, dtype: _arg(t, n, shape, dtype).value  # noqa: E731
    kmax = route_width(p)
    M = int(p["M"])
    cb = CallBuffers(
        label_q=ptr(b.label_q, "label_q", (H, N), I32T), label_k=ptr(b.label_k, "label_k", (H, N), I32T),
        perm_q=ptr(b.perm_q, "perm_q", (H, N), I32T), perm_k=ptr(b.perm_k, "perm_k", (H, N), I32T),
        off_q=ptr(b.off_q, "off_q", (H, oq), I32T), off_k=ptr(b.off_k, "off_k", (H, ok), I32T),
        qp=ptr(b.qp, "qp", (H, N, d), q.dtype), kp=ptr(b.kp, "kp", (H, N, d), q.dtype),
        vp=ptr(b.vp, "vp", (H, N, d), q.dtype),
        csr=ptr(b.csr, "csr", (H, int(p["Cq"]), kmax), I32T),
        k_per_head=ptr(b.k_per_head, "k_per_head", (H,), I32T),
        o_sparse=ptr(b.o_sparse, "o_sparse", (H, N, d), torch.float32),
        pairs_sparse=ptr(b.pairs_sparse, "pairs_sparse", (H,), I64),
        probes=ptr(b.probes, "probes", (H, max(M, 1)), I32T),
        pairs_exec=ptr(b.pairs_exec, "pairs_exec", (H,), I64),
        fit=None if b.fit is None else ptr(b.fit, "fit", (H, d * d + d), torch.float64))
    out = _arg(b.out, "out", (H, N, d), q.dtype)
    wp, wb = _ws(b.ws)
    _check(lib.sparsepr_attention(pq, pk, pv, dt, ctypes.byref(prm), ctypes.byref(cb), out, wp, wb,
                                  _stream(stream)), "sparsepr_attention")
    return b


def dense_params(H: int, N: int, d: int, scale: float = 0.0) -> dict:
    """Parameters of the same attention kernel run densely: one query group
    and one key group covering all N tokens, keep = 1."""
    return dict(H=H, N=N, d=d, n_text=0, Ck=1, Cq=1, Ms=1, n_eig=1, kmeans_iters=1,
                keep=[1.0] * H, M=0, r=1, lam=0.0, scale=scale, seed=0)


def dense_attention(q, k, v, out, ws=None, stream=None, meta=None):
    """Dense softmax attention through the same block-sparse kernel (the
    baseline of the same design): identity order, one group, full route.
    ``meta`` caches the small routing tensors between calls."""
    H, N, d = q.shape
    p = dense_params(H, N, d)
    if meta is None:
        meta = dict(
            off=torch.tensor([[0, N]] * H, dtype=torch.int32, device=q.device),
            csr=torch.zeros((H, 1, 1), dtype=torch.int32, device=q.device),
            kh=torch.ones(H, dtype=torch.int32, device=q.device),
            pairs=torch.empty(H, dtype=torch.int64, device=q.device))
    if ws is None:
        ws = torch.empty(workspace_bytes(p), dtype=torch.uint8, device=q.device)
    sparsepr_block_sparse_attn(q, k, v, p, meta["off"], meta["off"], meta["csr"], meta["kh"], out,
                               meta["pairs"], ws, stream)
    return meta, ws
