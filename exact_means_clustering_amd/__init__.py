"""Exact Lloyd k-means on MI355X (gfx950): Python binding of libflashkm.so.

The functions below only marshal torch tensors into the C ABI declared in
``include/flashkm.h``, ``include/flashkm_codebook.h`` and ``include/flashkm_train.h`` (same names without the
``kmeans_`` prefix): every step of the computation runs in the library's HIP kernels, on the current torch
stream.  PyTorch provides device memory and streams, nothing else.  There is
no CPU fallback: importing raises if the library is missing, and every call
raises ``KMeansError`` on a non-zero status.

Shapes: X is [N, D] or [B, N, D] (fp32 / fp16 / bf16, CUDA, contiguous);
centroids are [K, D] or [B, K, D] fp32.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import inspect
import os

import torch

__all__ = ["KMeansError", "lib_path", "workspace_bytes", "assign", "assign_top2", "assign_soft", "gauss_sum", "seed", "update",
           "fit", "fit_streamed", "tune", "tune_save", "tune_load", "assign_configs", "assign_noalloc",
           "stream_timeline", "embed", "embed_grad", "embed_grad_workspace_bytes", "balance", "balance_grad",
           "balance_workspace_bytes", "route", "route_grad", "adamw_states", "adamw_plan", "adamw", "AdamWPlan", "DTYPES"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libflashkm.so"

KM_OK, KM_EINVAL, KM_EUNSUPPORTED, KM_EWORKSPACE, KM_EHIP, KM_ENOMEM = range(6)
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class KMeansError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"flashkm status {status}: {msg}")
        self.status = status


def lib_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _load(path=None):
    path = path or lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built: run `python exact_means_clustering_amd/build.py` "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.kmeans_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
    lib.kmeans_workspace_bytes.restype = sz
    lib.kmeans_assign.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, P, sz, P]
    lib.kmeans_assign.restype = ctypes.c_int
    lib.kmeans_assign_noalloc.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, P]
    lib.kmeans_assign_noalloc.restype = ctypes.c_int
    lib.kmeans_update.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, P, sz, P]
    lib.kmeans_update.restype = ctypes.c_int
    lib.kmeans_fit.argtypes = [P, i32, i64, i32, i32, P, i32, i32, P, P, P, P, P, sz, P]
    lib.kmeans_fit.restype = ctypes.c_int
    lib.kmeans_fit_streamed.argtypes = [P, i32, i64, i32, P, i32, i32, sz, P, P, P, P, P]
    lib.kmeans_fit_streamed.restype = ctypes.c_int
    lib.kmeans_assign_top2.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, sz, P]
    lib.kmeans_assign_top2.restype = ctypes.c_int
    lib.kmeans_assign_soft.argtypes = [P, i32, i64, i32, i32, P, i32, P, ctypes.c_float, P, P, P, P, sz, P]
    lib.kmeans_assign_soft.restype = ctypes.c_int
    lib.kmeans_gauss_sum.argtypes = [P, i32, i64, i32, i32, P, i32, P, ctypes.c_float, P, P, P, sz, P]
    lib.kmeans_gauss_sum.restype = ctypes.c_int
    lib.kmeans_seed.argtypes = [P, i32, i64, i32, i32, i32, i32, P, P, P, P, P, sz, P]
    lib.kmeans_seed.restype = ctypes.c_int
    lib.kmeans_tune.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, sz, P, P, P, P]
    lib.kmeans_tune.restype = ctypes.c_int
    lib.kmeans_tune_save.argtypes = [ctypes.c_char_p]
    lib.kmeans_tune_save.restype = ctypes.c_int
    lib.kmeans_assign_configs.argtypes = [i32, i32, P, P, i32, P]
    lib.kmeans_stream_timeline.argtypes = [P, i32, P]
    lib.kmeans_stream_timeline.restype = ctypes.c_int
    lib.kmeans_assign_configs.restype = ctypes.c_int
    lib.kmeans_tune_load.argtypes = [ctypes.c_char_p]
    lib.kmeans_tune_load.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.kmeans_embed.argtypes = [P, i32, i64, i32, i32, i32, P, f32, P, i32, P]
    lib.kmeans_embed.restype = ctypes.c_int
    lib.kmeans_embed_grad_workspace_bytes.argtypes = [i64, i32, i32, i32]
    lib.kmeans_embed_grad_workspace_bytes.restype = sz
    lib.kmeans_embed_grad.argtypes = [P, i32, i64, i32, i32, i32, P, f32, i32, P, i32, P, sz, P]
    lib.kmeans_embed_grad.restype = ctypes.c_int
    lib.kmeans_balance_workspace_bytes.argtypes = [i64, i32, i32, i32]
    lib.kmeans_balance_workspace_bytes.restype = sz
    lib.kmeans_balance.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, P, P, P, P, sz, P]
    lib.kmeans_balance.restype = ctypes.c_int
    lib.kmeans_balance_grad.argtypes = [P, i32, i64, i32, i32, P, P, P, P, P]
    lib.kmeans_balance_grad.restype = ctypes.c_int
    f64 = ctypes.c_double
    lib.kmeans_route.argtypes = [P, i32, i64, i32, P, i32, i32, i32, i32, i32, i32, f32, P, P, P, P, P]
    lib.kmeans_route.restype = ctypes.c_int
    lib.kmeans_route_grad.argtypes = [P, i32, i64, i32, P, P, P, i32, i32, i32, f32, i32, P, P]
    lib.kmeans_route_grad.restype = ctypes.c_int
    lib.kmeans_adamw_chunks.argtypes = [P, i32]
    lib.kmeans_adamw_chunks.restype = i64
    lib.kmeans_adamw_table_bytes.argtypes = [P, i32]
    lib.kmeans_adamw_table_bytes.restype = sz
    lib.kmeans_adamw_table.argtypes = [P, i32, i32, i32, i32, P, sz]
    lib.kmeans_adamw_table.restype = ctypes.c_int
    lib.kmeans_adamw.argtypes = [P, i32, i64, i32, i32, i32, i32, f64, f64, f64, f64, f64, i64, P, P, P, P, P]
    lib.kmeans_adamw.restype = ctypes.c_int
    lib.kmeans_last_error.argtypes = []
    lib.kmeans_last_error.restype = ctypes.c_char_p
    return lib


_lib = _load()


def _check(rc: int):
    if rc != KM_OK:
        raise KMeansError(rc, _lib.kmeans_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _shape3(X):
    if X.dim() == 2:
        return 1, X.shape[0], X.shape[1]
    if X.dim() == 3:
        return X.shape
    raise ValueError("X must be [N, D] or [B, N, D]")


def _dtype(X):
    try:
        return DTYPES[X.dtype]
    except KeyError:
        raise KMeansError(KM_EUNSUPPORTED, f"unsupported dtype {X.dtype}") from None


def _need(t, name, dtype=None, like=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise KMeansError(KM_EINVAL, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise KMeansError(KM_EINVAL, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise KMeansError(KM_EINVAL, f"{name} must be {dtype}")
    if like is not None and t.device != like.device:
        raise KMeansError(KM_EINVAL, f"{name} must be on {like.device} (it is on {t.device})")


def _on_tensor_device(fn):
    """Run fn with its first CUDA tensor argument's device current, so the
    default stream and the library's device queries belong to that device."""
    @functools.wraps(fn)
    def run(*args, **kwargs):
        for a in args:
            if isinstance(a, torch.Tensor) and a.is_cuda:
                with torch.cuda.device(a.device):
                    return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return run


def _rows(C, name, B, D):
    """K of a centroid-like tensor [K, D] (B = 1) or [B, K, D] that goes with X."""
    ok = C.shape[-1] == D and (C.dim() == 3 and C.shape[0] == B or C.dim() == 2 and B == 1)
    if not ok:
        raise KMeansError(KM_EINVAL, f"{name} must be [K, {D}] or [{B}, K, {D}] (got {tuple(C.shape)})")
    return C.shape[-2]


def _count(t, name, n):
    if t.numel() != n:
        raise KMeansError(KM_EINVAL, f"{name} must have {n} elements (got {t.numel()})")


def workspace_bytes(N: int, D: int, K: int, B: int = 1, dtype=torch.bfloat16) -> int:
    dt = DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.kmeans_workspace_bytes(N, D, K, B, dt))


def _workspace(N, D, K, B, dt, device, ws):
    """A caller workspace (any dtype, contiguous, on X's device) or a new one;
    returns (tensor, its size in bytes)."""
    need = int(_lib.kmeans_workspace_bytes(N, D, K, B, dt))
    if need == 0:
        _check(_lib.kmeans_workspace_bytes(N, D, K, B, dt) or KM_EINVAL)
    if ws is not None:
        if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous():
            raise KMeansError(KM_EINVAL, f"ws must be a contiguous tensor on {device}")
        if ws.numel() * ws.element_size() >= need:
            return ws, ws.numel() * ws.element_size()
    return torch.empty(need, dtype=torch.uint8, device=device), need


@_on_tensor_device
def assign(X, C, *, want_min_d2: bool = False, ws=None, stream=None, labels=None):
    """Assignment stage: returns (labels int32, min_d2 fp32 or None, inertia fp64 [B])."""
    _need(X, "X")
    _need(C, "C", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C, "C", B, D)
    dt = _dtype(X)
    lab_shape = X.shape[:-1]
    if labels is None:
        labels = torch.empty(lab_shape, dtype=torch.int32, device=X.device)
    else:
        _need(labels, "labels", torch.int32, like=X)
        _count(labels, "labels", B * N)
    md = torch.empty(lab_shape, dtype=torch.float32, device=X.device) if want_min_d2 else None
    inertia = torch.empty(B, dtype=torch.float64, device=X.device)
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_assign(_ptr(X), dt, N, D, B, _ptr(C), K, _ptr(labels), _ptr(md), _ptr(inertia),
                              _ptr(ws), ws_bytes, _stream(stream)))
    return labels, md, inertia


@_on_tensor_device
def assign_noalloc(X, C, *, labels, inertia, min_d2=None, stream=None):
    """Assignment stage into caller tensors with no workspace and no allocation (the library's static
    scratch; calls that overlap on one GPU race): labels int32 [.., N], inertia fp64 [B], min_d2 fp32 [.., N]
    or None.  Returns (labels, min_d2, inertia)."""
    _need(X, "X")
    _need(C, "C", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C, "C", B, D)
    dt = _dtype(X)
    _need(labels, "labels", torch.int32, like=X)
    _count(labels, "labels", B * N)
    _need(inertia, "inertia", torch.float64, like=X)
    _count(inertia, "inertia", B)
    if min_d2 is not None:
        _need(min_d2, "min_d2", torch.float32, like=X)
        _count(min_d2, "min_d2", B * N)
    _check(_lib.kmeans_assign_noalloc(_ptr(X), dt, N, D, B, _ptr(C), K, _ptr(labels), _ptr(min_d2), _ptr(inertia),
                                      _stream(stream)))
    return labels, min_d2, inertia


@_on_tensor_device
def assign_top2(X, C, *, ws=None, stream=None):
    """Two nearest centroids of every point: returns (labels [.., N, 2] int32, distances [.., N, 2] fp32)."""
    _need(X, "X")
    _need(C, "C", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C, "C", B, D)
    dt = _dtype(X)
    labels2 = torch.empty((*X.shape[:-1], 2), dtype=torch.int32, device=X.device)
    d2 = torch.empty((*X.shape[:-1], 2), dtype=torch.float32, device=X.device)
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_assign_top2(_ptr(X), dt, N, D, B, _ptr(C), K, _ptr(labels2), _ptr(d2), _ptr(ws), ws_bytes,
                                   _stream(stream)))
    return labels2, d2


@_on_tensor_device
def assign_soft(X, C, sigma2: float, *, log_w=None, ws=None, stream=None):
    """Gaussian-mixture soft assignment (shared variance sigma2, log-weights log_w [.., K] or None): returns
    (most responsible component int32, log density fp32, its per-instance sum fp64 [B])."""
    _need(X, "X")
    _need(C, "C", torch.float32, like=X)
    if log_w is not None:
        _need(log_w, "log_w", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C, "C", B, D)
    if log_w is not None:
        _count(log_w, "log_w", B * K)
    dt = _dtype(X)
    labels = torch.empty(X.shape[:-1], dtype=torch.int32, device=X.device)
    logp = torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device)
    total = torch.empty(B, dtype=torch.float64, device=X.device)
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_assign_soft(_ptr(X), dt, N, D, B, _ptr(C), K, _ptr(log_w), float(sigma2), _ptr(labels),
                                   _ptr(logp), _ptr(total), _ptr(ws), ws_bytes, _stream(stream)))
    return labels, logp, total


@_on_tensor_device
def gauss_sum(X, Y, w, sigma2: float, *, ws=None, stream=None):
    """Gauss kernel sums G[.., i] = sum_k w[.., k] exp(-||x_i - y_k||^2 / (2 sigma2)): returns (G fp32, sum fp64 [B])."""
    _need(X, "X")
    _need(Y, "Y", torch.float32, like=X)
    _need(w, "w", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(Y, "Y", B, D)
    _count(w, "w", B * K)
    dt = _dtype(X)
    G = torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device)
    total = torch.empty(B, dtype=torch.float64, device=X.device)
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_gauss_sum(_ptr(X), dt, N, D, B, _ptr(Y), K, _ptr(w), float(sigma2), _ptr(G), _ptr(total),
                                 _ptr(ws), ws_bytes, _stream(stream)))
    return G, total


@_on_tensor_device
def seed(X, u, *, method: str = "kmeans++", want_d2: bool = False, ws=None, stream=None):
    """Initial centroids from the caller's uniforms u [.., K] (fp64, CUDA, in [0, 1)): method "random" (rows
    floor(u N)) or "kmeans++" (D^2 sampling).  Returns (row indices int32 [.., K], centroids fp32 [.., K, D],
    squared distance of every row to its nearest pick fp32 [.., N] or None)."""
    _need(X, "X")
    _need(u, "u", torch.float64, like=X)
    B, N, D = _shape3(X)
    K = u.shape[-1]
    if u.numel() != B * K:
        raise KMeansError(KM_EINVAL, "u must be [K] or [B, K]")
    dt = _dtype(X)
    m = {"random": 0, "kmeans++": 1}.get(method)
    if m is None:
        raise KMeansError(KM_EINVAL, f"unknown seeding method {method!r}")
    idx = torch.empty(u.shape, dtype=torch.int32, device=X.device)
    C = torch.empty((*u.shape, D), dtype=torch.float32, device=X.device)
    d2 = torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device) if want_d2 else None
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_seed(_ptr(X), dt, N, D, B, K, m, _ptr(u), _ptr(idx), _ptr(C), _ptr(d2), _ptr(ws), ws_bytes,
                            _stream(stream)))
    return idx, C, d2


@_on_tensor_device
def update(X, labels, C_prev, *, C_new=None, ws=None, stream=None):
    """Centroid update stage: returns (C_new fp32, counts int32)."""
    _need(X, "X")
    _need(labels, "labels", torch.int32, like=X)
    _need(C_prev, "C_prev", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C_prev, "C_prev", B, D)
    _count(labels, "labels", B * N)
    dt = _dtype(X)
    if C_new is None:
        C_new = torch.empty_like(C_prev)
    else:
        _need(C_new, "C_new", torch.float32, like=X)
        _count(C_new, "C_new", B * K * D)
    counts = torch.empty(C_prev.shape[:-1], dtype=torch.int32, device=X.device)
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_update(_ptr(X), dt, N, D, B, _ptr(labels), K, _ptr(C_prev), _ptr(C_new), _ptr(counts),
                              _ptr(ws), ws_bytes, _stream(stream)))
    return C_new, counts


@_on_tensor_device
def fit(X, C0, iters: int, *, history: bool = False, ws=None, stream=None, out=None):
    """Exact Lloyd iteration: returns (labels, C, inertia [B] fp64, history [iters, B] or None).

    ``out`` = (labels, C, inertia, history-or-None) reuses caller tensors for the results: calls with the same
    buffers replay the library's captured graph of the fit instead of capturing a new one."""
    _need(X, "X")
    _need(C0, "C0", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C0, "C0", B, D)
    dt = _dtype(X)
    if out is not None:
        labels, C, inertia, hist = out
        _need(labels, "labels", torch.int32, like=X)
        _need(C, "C", torch.float32, like=X)
        _need(inertia, "inertia", torch.float64, like=X)
        if labels.numel() != B * N or C.numel() != B * K * D or inertia.numel() != B:
            raise KMeansError(KM_EINVAL, "out tensors do not match the problem's shapes")
        if history:
            if hist is None or hist.numel() < max(1, int(iters)) * B:
                raise KMeansError(KM_EINVAL, "history requested but out[3] is missing or too small")
            _need(hist, "history", torch.float64, like=X)
        else:
            hist = None
    else:
        labels = torch.empty(X.shape[:-1], dtype=torch.int32, device=X.device)
        C = torch.empty_like(C0)
        inertia = torch.empty(B, dtype=torch.float64, device=X.device)
        hist = torch.empty((max(1, int(iters)), B), dtype=torch.float64, device=X.device) if history else None
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    _check(_lib.kmeans_fit(_ptr(X), dt, N, D, B, _ptr(C0), K, int(iters), _ptr(labels), _ptr(C), _ptr(inertia),
                           _ptr(hist), _ptr(ws), ws_bytes, _stream(stream)))
    return labels, C, inertia, hist


@_on_tensor_device
def tune(X, C, *, labels=None, ws=None, stream=None):
    """Time every compiled assignment configuration on this shape and record the
    fastest in the library's tuning table.  Returns (pb, waves, ms per launch)."""
    _need(X, "X")
    _need(C, "C", torch.float32, like=X)
    B, N, D = _shape3(X)
    K = _rows(C, "C", B, D)
    dt = _dtype(X)
    if labels is None:
        labels = torch.empty(X.shape[:-1], dtype=torch.int32, device=X.device)
    else:
        _need(labels, "labels", torch.int32, like=X)
        _count(labels, "labels", B * N)
    ws, ws_bytes = _workspace(N, D, K, B, dt, X.device, ws)
    pb, waves, ms = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_float(0.0)
    _check(_lib.kmeans_tune(_ptr(X), dt, N, D, B, _ptr(C), K, _ptr(labels), _ptr(ws), ws_bytes, _stream(stream),
                            ctypes.byref(pb), ctypes.byref(waves), ctypes.byref(ms)))
    return pb.value, waves.value, ms.value


def tune_save(path: str):
    """Write the tuning table as text ("dtype D N B K pb waves" per line)."""
    _check(_lib.kmeans_tune_save(os.fsencode(path)))


def assign_configs(dtype, D: int) -> list:
    """The (pb, waves) assignment configurations compiled for rows of D elements of dtype."""
    dt = DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    pb, waves, n = (ctypes.c_int32 * 8)(), (ctypes.c_int32 * 8)(), ctypes.c_int32(0)
    _check(_lib.kmeans_assign_configs(dt, int(D), pb, waves, 8, ctypes.byref(n)))
    if n.value > 8:
        raise KMeansError(KM_EINVAL, f"{n.value} configurations; the binding reads at most 8")
    return [(pb[i], waves[i]) for i in range(n.value)]


def stream_timeline():
    """Per-chunk timeline of the last fit_streamed on this thread: a list of rows (iteration, chunk, copy-in start,
    copy-in end, compute start, compute end, labels-out start, labels-out end), times in ms from the fit's start."""
    n = ctypes.c_int32(0)
    _check(_lib.kmeans_stream_timeline(None, 0, ctypes.byref(n)))
    buf = (ctypes.c_double * (8 * max(1, n.value)))()
    _check(_lib.kmeans_stream_timeline(buf, n.value, ctypes.byref(n)))
    return [tuple(buf[8 * i + j] for j in range(8)) for i in range(n.value)]


def tune_load(path: str):
    """Add the entries of a tuning-table file (all or nothing)."""
    _check(_lib.kmeans_tune_load(os.fsencode(path)))


@_on_tensor_device
def fit_streamed(X_host, C0, iters: int, device_x_budget: int, *, history: bool = False, stream=None):
    """Out-of-core Lloyd iteration over a pinned host tensor X_host [N, D].

    Returns (labels int32 CPU, C fp32 CUDA, inertia float, history list or None)."""
    if not isinstance(X_host, torch.Tensor) or X_host.is_cuda or not X_host.is_pinned():
        raise KMeansError(KM_EINVAL, "X_host must be a pinned CPU tensor")
    if X_host.dim() != 2 or not X_host.is_contiguous():
        raise KMeansError(KM_EINVAL, "X_host must be a contiguous [N, D] tensor")
    _need(C0, "C0", torch.float32)
    N, D = X_host.shape
    K = _rows(C0, "C0", 1, D)
    dt = _dtype(X_host)
    labels = torch.empty(N, dtype=torch.int32, pin_memory=True)
    C = torch.empty_like(C0)
    inertia = ctypes.c_double(0.0)
    hist = (ctypes.c_double * max(1, int(iters)))() if history else None
    _check(_lib.kmeans_fit_streamed(_ptr(X_host), dt, N, D, _ptr(C0), K, int(iters), int(device_x_budget),
                                    _ptr(labels), _ptr(C), ctypes.byref(inertia),
                                    hist if hist is not None else None, _stream(stream)))
    return labels, C, inertia.value, (list(hist) if hist is not None else None)


# ---- codebook operators (include/flashkm_codebook.h) ------------------------------


def _on_stream(fn):
    """Give fn a keyword ``stream``: it runs with its first CUDA tensor's device, and ``stream`` if one is given,
    current, so what it allocates belongs to the stream that uses it."""
    @functools.wraps(fn)
    def run(*args, stream=None, **kwargs):
        t = args[0] if args else None
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            t = next((a for a in (*args, *kwargs.values()) if isinstance(a, torch.Tensor) and a.is_cuda), None)
            if t is None:
                return fn(*args, **kwargs)
        if stream is not None:
            if stream.device != t.device:
                raise KMeansError(KM_EINVAL, f"stream is on {stream.device}, the tensors on {t.device}")
            with torch.cuda.stream(stream):
                return fn(*args, **kwargs)
        if t.get_device() == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(t.device):
            return fn(*args, **kwargs)
    sig = inspect.signature(fn)
    run.__signature__ = sig.replace(parameters=[
        *sig.parameters.values(), inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return run


# torch's own shortcut to the current stream's handle (2.7 us less per call than building a Stream object)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _current(t):
    return _raw_stream(t.get_device())


def _int32(v, name):
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise KMeansError(KM_EINVAL, f"{name}={v} does not fit 32 bits")
    return v


def _ids(ids, name, like, lead):
    """int32 ids of the rows ``lead`` ([N] or [B, N])."""
    _need(ids, name, torch.int32, like=like)
    if tuple(ids.shape) != tuple(lead):
        raise KMeansError(KM_EINVAL, f"{name} must be {tuple(lead)} (got {tuple(ids.shape)})")


def _into(t, name, shape, dtype, like):
    """A caller's output tensor of exactly this shape and type."""
    _need(t, name, dtype, like=like)
    if tuple(t.shape) != tuple(shape):
        raise KMeansError(KM_EINVAL, f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")


def _scratch(need, device, ws):
    """A caller workspace or a new one; returns (tensor, its size in bytes).  No need of one: a shape was refused."""
    if need == 0:
        msg = _lib.kmeans_last_error().decode(errors="replace")
        raise KMeansError(KM_EUNSUPPORTED if msg.startswith("unsupported") else KM_EINVAL, msg)
    if ws is None:
        if need == 256:  # the shape needs none
            return None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        return ws, need
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise KMeansError(KM_EINVAL, f"ws must be a contiguous tensor on {device}")
    return ws, ws.numel() * ws.element_size()


def _at(t):
    return None if t is None else t.data_ptr()


@_on_stream
def embed(table, ids, *, scale: float = 1.0, out_dtype=None, out=None):
    """Table lookup with scaling: out[.., i, :] = scale * table[.., ids[.., i], :], rounded once; zeros for ids outside
    [0, K).  table [K, D] with ids [N], or [B, K, D] with ids [B, N] int32; out_dtype defaults to the table's.  Runs on
    ``stream`` (default: the current one)."""
    _need(table, "table")
    dt = _dtype(table)
    if table.dim() not in (2, 3):
        raise KMeansError(KM_EINVAL, "table must be [K, D] or [B, K, D]")
    _need(ids, "ids", torch.int32, like=table)
    if ids.dim() != table.dim() - 1 or (table.dim() == 3 and ids.shape[0] != table.shape[0]):
        raise KMeansError(KM_EINVAL, f"ids must be [N] for a table [K, D], [B, N] for [B, K, D] (got {tuple(ids.shape)} "
                                     f"with {tuple(table.shape)})")
    B = _int32(table.shape[0], "B") if table.dim() == 3 else 1
    K, D = _int32(table.shape[-2], "K"), _int32(table.shape[-1], "D")
    if out is None:
        out = torch.empty((*ids.shape, D), dtype=out_dtype or table.dtype, device=table.device)
    else:
        _into(out, "out", (*ids.shape, D), out_dtype, table)
    _check(_lib.kmeans_embed(table.data_ptr(), dt, ids.shape[-1], K, D, B, ids.data_ptr(), float(scale),
                             out.data_ptr(), _dtype(out), _current(table)))
    return out


def embed_grad_workspace_bytes(N: int, K: int, D: int, B: int = 1) -> int:
    return int(_lib.kmeans_embed_grad_workspace_bytes(N, _int32(K, "K"), _int32(D, "D"), _int32(B, "B")))


@_on_stream
def embed_grad(dout, ids, K: int, *, scale: float = 1.0, grad_dtype=None, out=None, accumulate: bool = False, ws=None):
    """Gradient of embed with respect to the table: [.., K, D], the sum of scale * dout[.., i, :] over the rows i with
    ids[.., i] = k (deterministic, fp32 sums rounded once into grad_dtype, fp32 by default).  accumulate adds to ``out``
    and leaves the entries that no row names untouched.  Runs on ``stream`` (default: the current one)."""
    _need(dout, "dout")
    dt = _dtype(dout)
    if dout.dim() not in (2, 3):
        raise KMeansError(KM_EINVAL, "dout must be [N, D] or [B, N, D]")
    _ids(ids, "ids", dout, dout.shape[:-1])
    B = dout.shape[0] if dout.dim() == 3 else 1
    N, D = dout.shape[-2:]
    K = _int32(K, "K")
    need = embed_grad_workspace_bytes(N, K, D, B)
    ws, ws_bytes = _scratch(need, dout.device, ws)
    shape = (K, D) if dout.dim() == 2 else (B, K, D)
    if out is None:
        if accumulate:
            raise KMeansError(KM_EINVAL, "accumulate needs out")
        out = torch.empty(shape, dtype=grad_dtype or torch.float32, device=dout.device)
    else:
        _into(out, "out", shape, grad_dtype, dout)
    _check(_lib.kmeans_embed_grad(dout.data_ptr(), dt, N, K, D, B, ids.data_ptr(), float(scale), int(bool(accumulate)),
                                  out.data_ptr(), _dtype(out), _at(ws), ws_bytes, _current(dout)))
    return out


def balance_workspace_bytes(N: int, K: int, B: int = 1, S: int = 1) -> int:
    return int(_lib.kmeans_balance_workspace_bytes(N, _int32(K, "K"), _int32(B, "B"), _int32(S, "S")))


def _logits(logits):
    _need(logits, "logits")
    if logits.dim() not in (2, 3):
        raise KMeansError(KM_EINVAL, "logits must be [N, K] or [B, N, K]")
    B = _int32(logits.shape[0], "B") if logits.dim() == 3 else 1
    return _dtype(logits), B, logits.shape[-2], _int32(logits.shape[-1], "K")


@_on_stream
def balance(logits, labels, *, valid=None, ws=None):
    """Balance loss of the use of K choices: logits [.., N, K], labels [.., N] or [.., N, S] int32 (the selections, for
    instance from assign or assign_top2), valid [.., N] bool or None.  Returns (loss fp32 [B], counts int32 [.., K],
    mean probabilities fp32 [.., K], (lse fp32 [.., N], coef fp32 [.., K])); the last pair is what balance_grad needs.
    Runs on ``stream`` (default: the current one)."""
    dt, B, N, K = _logits(logits)
    _need(labels, "labels", torch.int32, like=logits)
    lead = tuple(logits.shape[:-1])
    if labels.dim() not in (len(lead), len(lead) + 1) or tuple(labels.shape[:len(lead)]) != lead:
        raise KMeansError(KM_EINVAL, f"labels must be {lead} or {lead} + (S,) (got {tuple(labels.shape)})")
    S = labels.shape[-1] if labels.dim() > len(lead) else 1
    if valid is not None:
        _into(valid, "valid", lead, torch.bool, logits)
    ws, ws_bytes = _scratch(balance_workspace_bytes(N, K, B, S), logits.device, ws)
    per = (K,) if logits.dim() == 2 else (B, K)
    loss = torch.empty(B, dtype=torch.float32, device=logits.device)
    counts = torch.empty(per, dtype=torch.int32, device=logits.device)
    prob = torch.empty(per, dtype=torch.float32, device=logits.device)
    coef = torch.empty(per, dtype=torch.float32, device=logits.device)
    lse = torch.empty(lead, dtype=torch.float32, device=logits.device)
    _check(_lib.kmeans_balance(logits.data_ptr(), dt, N, K, B, labels.data_ptr(), S, _at(valid), loss.data_ptr(),
                               counts.data_ptr(), prob.data_ptr(), lse.data_ptr(), coef.data_ptr(), _at(ws), ws_bytes,
                               _current(logits)))
    return loss, counts, prob, (lse, coef)


@_on_stream
def balance_grad(logits, saved, dloss, *, out=None):
    """Gradient of the balance loss with respect to the logits: ``saved`` = the (lse, coef) of balance, dloss fp32 [B]
    the derivative of what follows with respect to the loss.  Returns dlogits, of the logits' shape and type.  Runs on
    ``stream`` (default: the current one)."""
    dt, B, N, K = _logits(logits)
    lse, coef = saved
    _into(lse, "lse", logits.shape[:-1], torch.float32, logits)
    _into(coef, "coef", (K,) if logits.dim() == 2 else (B, K), torch.float32, logits)
    _into(dloss, "dloss", (B,), torch.float32, logits)
    if out is None:
        out = torch.empty_like(logits)
    else:
        _into(out, "out", logits.shape, logits.dtype, logits)
    _check(_lib.kmeans_balance_grad(logits.data_ptr(), dt, N, K, B, lse.data_ptr(), coef.data_ptr(), dloss.data_ptr(),
                                    out.data_ptr(), _current(logits)))
    return out


# ---- training operators (include/flashkm_train.h) ---------------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score):
    try:
        return _SCORES[score]
    except (KeyError, TypeError):
        raise KMeansError(KM_EUNSUPPORTED, f"unknown score {score!r} (softmax or sigmoid)") from None


@_on_stream
def route(logits, S: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups=None, group_best: int = 2,
          renormalise: bool = True, scale: float = 1.0, valid=None):
    """Routing of rows to S of K choices: logits [.., N, K]; scores by ``score`` ("softmax" or "sigmoid"); bias [K] fp32 or
    None is added for the selection alone; with ``groups`` > 1 only the top_groups groups of the largest worth (the sum
    of their group_best largest biased scores) take part; valid [.., N] bool or None.  Returns (ids int32, weights fp32,
    chosen logits fp32), [.., N, S] each: ids in the order of the biased scores, ties to the lowest index, -1 (weight 0,
    chosen -inf) where no choice is left; weights scale * score, divided by their row's sum if ``renormalise``.  ids are
    labels for balance; chosen is what route_grad needs.  Runs on ``stream`` (default: the current one)."""
    dt, _, _, K = _logits(logits)
    S = _int32(S, "S")
    lead = logits.shape[:-1]
    if bias is not None:
        _into(bias, "bias", (K,), torch.float32, logits)
    if valid is not None:
        _into(valid, "valid", lead, torch.bool, logits)
    if not 1 <= S <= 64:  # (no outputs of a size that the call refuses)
        raise KMeansError(KM_EINVAL if S < 1 else KM_EUNSUPPORTED, f"S={S} must be 1 to 64")
    shape = (*lead, S)
    ids = logits.new_empty(shape, dtype=torch.int32)
    weights = torch.empty_like(ids, dtype=torch.float32)
    chosen = torch.empty_like(weights)
    groups = _int32(groups, "groups")
    _check(_lib.kmeans_route(logits.data_ptr(), dt, lead.numel(), K, _at(bias), _score(score), groups,
                             groups if top_groups is None else _int32(top_groups, "top_groups"),
                             _int32(group_best, "group_best"), S, int(bool(renormalise)), float(scale), _at(valid),
                             ids.data_ptr(), weights.data_ptr(), chosen.data_ptr(), _current(logits)))
    return ids, weights, chosen


@_on_stream
def route_grad(logits, ids, chosen, dweights, *, score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
               out=None, accumulate: bool = False):
    """Gradient of route's weights with respect to the logits, the ids held fixed: ids and chosen of route, dweights
    [.., N, S] fp32 the derivative of what follows, the other arguments as in route.  Returns dlogits, of the logits'
    shape and type; accumulate adds to ``out`` (for instance balance_grad's gradient) and leaves the entries that the
    gradient does not reach untouched.  Runs on ``stream`` (default: the current one)."""
    dt, _, _, K = _logits(logits)
    lead = logits.shape[:-1]
    _need(ids, "ids", torch.int32, like=logits)
    if ids.dim() != logits.dim() or ids.shape[:-1] != lead:
        raise KMeansError(KM_EINVAL, f"ids must be {tuple(lead)} + (S,) (got {tuple(ids.shape)})")
    _into(chosen, "chosen", ids.shape, torch.float32, logits)
    _into(dweights, "dweights", ids.shape, torch.float32, logits)
    if out is None:
        if accumulate:
            raise KMeansError(KM_EINVAL, "accumulate needs out")
        out = torch.empty_like(logits)
    else:
        _into(out, "out", logits.shape, logits.dtype, logits)
    _check(_lib.kmeans_route_grad(logits.data_ptr(), dt, lead.numel(), K, ids.data_ptr(), chosen.data_ptr(),
                                  dweights.data_ptr(), _int32(ids.shape[-1], "S"), _score(score),
                                  int(bool(renormalise)), float(scale), int(bool(accumulate)), out.data_ptr(),
                                  _current(logits)))
    return out


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("numel", ctypes.c_int64), ("decay", ctypes.c_float)]


ADAMW_BLOCK = 256  # elements of an 8-bit state that share a scale
_STOCHASTIC = 256  # KM_ADAMW_STOCHASTIC


def adamw_states(params, bits: int = 32):
    """Zero states for the tensors ``params``: (exp_avg, exp_avg_sq, scales).  In 32 bits two lists of fp32 tensors of the
    parameters' shapes and None; in 8 bits lists of float8_e4m3fn and float8_e5m2 tensors and the pair of lists of their
    fp32 scales, one for each 256 consecutive elements (a state's value is code * scale)."""
    if bits == 32:
        return ([torch.zeros_like(p, dtype=torch.float32, memory_format=torch.contiguous_format) for p in params],
                [torch.zeros_like(p, dtype=torch.float32, memory_format=torch.contiguous_format) for p in params], None)
    if bits != 8:
        raise KMeansError(KM_EUNSUPPORTED, f"unsupported bits={bits} (32 or 8)")
    zero = lambda p, dt: torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(dt)  # noqa: E731
    scale = lambda p: torch.zeros(-(-p.numel() // ADAMW_BLOCK), dtype=torch.float32, device=p.device)  # noqa: E731
    return ([zero(p, torch.float8_e4m3fn) for p in params], [zero(p, torch.float8_e5m2) for p in params],
            ([scale(p) for p in params], [scale(p) for p in params]))


class AdamWPlan:
    """The tensors of adamw calls, checked and laid out once (made by adamw_plan): it keeps their memory alive, and steps
    what is there, also after a tensor was given other memory."""

    def __init__(self, groups, device, stream, memory):
        self._groups, self.device, self._stream, self._memory = groups, device, stream, memory


def adamw_plan(params, grads, exp_avg, exp_avg_sq, *, scales=None, masters=None, decay=None):
    """Lay out the tensors of AdamW steps: lists of one length of contiguous CUDA tensors on one device.  params and grads
    of any of the three types (they may be mixed; each pair of types is a launch of its own), exp_avg and exp_avg_sq
    fp32, or float8_e4m3fn and float8_e5m2 with ``scales`` (two lists of fp32 tensors, see adamw_states); masters: a list
    of fp32 copies of the parameters on which the step is taken, with None for those without (and for fp32 parameters),
    or None; decay: a factor of weight_decay for each tensor, or None (1).  The plan holds these tensors' memory and does
    not follow a tensor that is given other memory (``p.data = ...``, a gradient made anew): later gradients are written
    into the same tensors, else a new plan is made.  A captured step needs the plan as long as it is replayed."""
    params = list(params)
    n = len(params)
    if n == 0:
        raise KMeansError(KM_EINVAL, "params must not be empty")
    lists = {"grads": list(grads), "exp_avg": list(exp_avg), "exp_avg_sq": list(exp_avg_sq),
             "masters": [None] * n if masters is None else list(masters),
             "decay": [1.0] * n if decay is None else [float(d) for d in decay]}
    if scales is not None:
        lists["scales[0]"], lists["scales[1]"] = list(scales[0]), list(scales[1])
    for name, v in lists.items():
        if len(v) != n:
            raise KMeansError(KM_EINVAL, f"{name} must have {n} entries (got {len(v)})")
    bits = 32 if scales is None else 8
    kinds = (torch.float32, torch.float32) if bits == 32 else (torch.float8_e4m3fn, torch.float8_e5m2)
    groups, memory = {}, []
    for i, p in enumerate(params):
        g, m, v, w = (lists[k][i] for k in ("grads", "exp_avg", "exp_avg_sq", "masters"))
        _need(p, f"params[{i}]", like=params[0])
        _into(g, f"grads[{i}]", p.shape, g.dtype if isinstance(g, torch.Tensor) else None, params[0])
        _into(m, f"exp_avg[{i}]", p.shape, kinds[0], params[0])
        _into(v, f"exp_avg_sq[{i}]", p.shape, kinds[1], params[0])
        t = _AdamWTensor(p.data_ptr(), g.data_ptr(), None, m.data_ptr(), v.data_ptr(), None, None, p.numel(),
                         lists["decay"][i])
        if w is not None:
            _into(w, f"masters[{i}]", p.shape, torch.float32, params[0])
            t.master = w.data_ptr()
        if bits == 8:
            a, b = lists["scales[0]"][i], lists["scales[1]"][i]
            for k, x in enumerate((a, b)):
                _into(x, f"scales[{k}][{i}]", (-(-p.numel() // ADAMW_BLOCK),), torch.float32, params[0])
            t.exp_avg_scale, t.exp_avg_sq_scale = a.data_ptr(), b.data_ptr()
        # (the storages themselves: a tensor may let go of its own)
        memory += [x.untyped_storage() for x in (p, g, m, v, w, *((a, b) if bits == 8 else ())) if x is not None]
        if p.numel():
            groups.setdefault((_dtype(p), _dtype(g), w is not None), []).append(t)
        else:
            _dtype(p), _dtype(g)
    made = []
    device = params[0].device
    with torch.cuda.device(device):
        for (pdt, gdt, has), ts in groups.items():
            array = (_AdamWTensor * len(ts))(*ts)
            need = int(_lib.kmeans_adamw_table_bytes(array, len(ts)))
            if need == 0:
                _check(KM_EINVAL)
            chunks = int(_lib.kmeans_adamw_chunks(array, len(ts)))
            host = torch.zeros(need, dtype=torch.uint8)
            _check(_lib.kmeans_adamw_table(array, len(ts), pdt, gdt, bits, host.data_ptr(), need))
            made.append((host.to(device), len(ts), chunks, pdt, gdt, bits, int(has)))
        if len(groups) > 1:  # nothing may overlap across the launches either
            _across(groups, bits)
        stream = _raw_stream(device.index)
    return AdamWPlan(made, device, stream, memory)


def _across(groups, bits):
    """Refuse arrays that a step writes where another group's tensors lie."""
    size = {0: 4, 1: 2, 2: 2}
    ranges = []
    for key, ts in groups.items():
        for t in ts:
            n, state = t.numel, 4 if bits == 32 else 1
            scale = -(-n // ADAMW_BLOCK) * 4
            for name, at, nbytes, out in (("param", t.param, n * size[key[0]], True),
                                          ("grad", t.grad, n * size[key[1]], False),
                                          ("master", t.master, n * 4, True), ("exp_avg", t.exp_avg, n * state, True),
                                          ("exp_avg_sq", t.exp_avg_sq, n * state, True),
                                          ("exp_avg_scale", t.exp_avg_scale, scale, True),
                                          ("exp_avg_sq_scale", t.exp_avg_sq_scale, scale, True)):
                if at:
                    ranges.append((at, at + nbytes, name, out))
    ranges.sort()
    reach = {False: (0, ""), True: (0, "")}  # the furthest end of everything, and of what is written
    for a, b, name, out in ranges:
        end, other = reach[not out]
        if a < end:
            raise KMeansError(KM_EINVAL, f"{name} overlaps {other} of another tensor")
        reach[False] = max(reach[False], (b, name))
        if out:
            reach[True] = max(reach[True], (b, name))


def _scalar_at(t, name, dtype, device):
    """A device scalar of a call, or None."""
    if not isinstance(t, torch.Tensor):
        return None
    _need(t, name, dtype)
    if t.numel() != 1 or t.device != device:
        raise KMeansError(KM_EINVAL, f"{name} must be one value on {device}")
    return t.data_ptr()


def adamw(plan: AdamWPlan, *, lr, step, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
          grad_scale=None, skip=None, rounding: str = "nearest", stream=None):
    """One AdamW step over the plan's tensors, in place:
    m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2, p = p (1 - lr weight_decay) - lr mhat / (sqrt(vhat) + eps), with
    g = grad_scale * grad and mhat, vhat without the bias of a zero start after ``step`` steps (the first is 1).  lr may
    be an fp32 CUDA tensor and step an int64 one, of one value, which are read on the device (for captured calls);
    grad_scale is None or an fp32 CUDA tensor; skip is None or a bool or uint8 CUDA tensor: nothing changes where it is
    true.  rounding: how states in 8 bits are rounded to their codes.  "nearest" holds each state as near as its format
    allows, but over a run v stays frozen relative to the largest of its 256 elements (a step moves it by less than half a
    code), so elements whose gradients change take steps that are several times too small or too large;
    "stochastic" rounds either way so that what is held follows the averages without bias, and is the one to train with
    for more than some hundred steps.  Its random numbers come from the step and the element's place, so each step needs
    its own number, and a run repeats bit for bit.  Runs on ``stream`` (default: the current one)."""
    if not isinstance(plan, AdamWPlan):
        raise KMeansError(KM_EINVAL, "plan must be made by adamw_plan")
    device = plan.device
    if stream is not None and stream.device != device:
        raise KMeansError(KM_EINVAL, f"stream is on {stream.device}, the tensors on {device}")
    lr_at = _scalar_at(lr, "lr", torch.float32, device)
    step_at = _scalar_at(step, "step", torch.int64, device)
    if grad_scale is not None and not isinstance(grad_scale, torch.Tensor):
        raise KMeansError(KM_EINVAL, "grad_scale must be a CUDA tensor")
    scale_at = _scalar_at(grad_scale, "grad_scale", torch.float32, device)
    if skip is not None and (not isinstance(skip, torch.Tensor) or skip.dtype not in (torch.bool, torch.uint8)):
        raise KMeansError(KM_EINVAL, "skip must be a bool or uint8 CUDA tensor")
    skip_at = _scalar_at(skip, "skip", skip.dtype if skip is not None else None, device)
    if rounding not in ("nearest", "stochastic"):
        raise KMeansError(KM_EUNSUPPORTED, f"unknown rounding {rounding!r} (nearest or stochastic)")
    if rounding == "stochastic" and any(group[5] != 8 for group in plan._groups):
        raise KMeansError(KM_EINVAL, "rounding='stochastic' is for states in 8 bits")
    how = _STOCHASTIC if rounding == "stochastic" else 0
    with contextlib.nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device):
        raw = _raw_stream(device.index) if stream is None else stream.cuda_stream
        if raw != plan._stream:  # the table must outlive the step there
            on = stream if stream is not None else torch.cuda.current_stream()
            for group in plan._groups:
                group[0].record_stream(on)
        for table, count, chunks, pdt, gdt, bits, masters in plan._groups:
            _check(_lib.kmeans_adamw(table.data_ptr(), count, chunks, pdt, gdt, bits | how, masters,
                                     0.0 if lr_at else float(lr), float(betas[0]), float(betas[1]), float(eps),
                                     float(weight_decay), 1 if step_at else int(step), lr_at, step_at, scale_at,
                                     skip_at, raw))
