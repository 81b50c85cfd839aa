"""Chunk-parallel gated linear attention (GLA, Mamba-2 SSD) for GB300.

Thin Python binding over the C ABI in ``include/glacore.h`` (library
``libglacore.so``, built from ``csrc/`` by ``_build.py``).  This module only
marshals arguments: PyTorch provides device memory and the current stream;
every step of the computation runs in the library's CUDA kernels.  There is
no CPU or PyTorch fallback: if the library cannot be loaded every call
raises.

Entry points (same names as the C ABI):
    gla_fwd(q, k, v, g, ...)            -> (o, final_state)
    gla_bwd(q, k, v, g, do, ...)        -> (dq, dk, dv, dg, dh0)
    ssd_fwd / ssd_bwd                   (scalar per-head gate, g [B,T,H])
    delta_fwd / delta_bwd               (gated delta rule, g and beta [B,T,H])
    gla_step / ssd_step / delta_step    -> o (new tokens on a pool of states)
    qk_norm_fwd / qk_norm_bwd           -> (q, k) / (dq, dk, dwq, dwk)
    layer_norm_fwd / layer_norm_bwd     -> (y, mean, rstd) / (dx, dw, db)
    linear_ce_fwd / linear_ce_bwd       -> (loss, lse) / (dx, dw)
    count_docs(segment_ids)             -> int
    get_device_error()                  -> None or raises GlacoreError

Layouts: q, k [B,T,Hqk,K]; v, o, do [B,T,H,V]; g [B,T,H,K] (GLA) or
[B,T,H] (SSD), fp32; states [n_seqs,H,K,V] fp32; segment_ids [B,T] int32.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

__all__ = [
    "GlacoreError", "load", "gla_fwd", "gla_bwd", "ssd_fwd", "ssd_bwd", "count_docs",
    "get_device_error", "workspace_size", "Problem", "selftest_wait", "norm_gate_fwd", "norm_gate_bwd",
    "short_conv_fwd", "short_conv_bwd", "gla_fwd_state", "gla_bwd_state", "state_scan",
    "gla_step", "ssd_step", "layer_norm_fwd", "layer_norm_bwd", "linear_ce_fwd", "linear_ce_bwd",
    "delta_fwd", "delta_bwd", "delta_step", "qk_norm_fwd", "qk_norm_bwd",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libglacore.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE, ERR_DOCS, ERR_RANGE, ERR_INDEX = range(9)
F32, BF16 = 0, 1

EXPORTS = (
    "gla_fwd", "gla_bwd", "ssd_fwd", "ssd_bwd", "gla_fwd_workspace_size", "gla_bwd_workspace_size",
    "ssd_fwd_workspace_size", "ssd_bwd_workspace_size", "glacore_count_docs",
    "glacore_get_device_error", "glacore_status_string", "glacore_version",
    "glacore_set_timing_events", "glacore_timing_count", "glacore_timing_label", "gla_bwd_noalloc",
    "glacore_selftest_wait", "norm_gate_fwd", "norm_gate_bwd", "norm_gate_bwd_workspace_size",
    "short_conv_fwd", "short_conv_bwd", "short_conv_bwd_workspace_size",
    "gla_fwd_state", "gla_bwd_state", "glacore_state_scan", "glacore_last_cuda_error",
    "gla_step", "ssd_step", "layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace_size",
    "linear_ce_fwd", "linear_ce_bwd", "linear_ce_fwd_workspace_size", "linear_ce_bwd_workspace_size",
    "delta_fwd", "delta_bwd", "delta_step", "delta_fwd_workspace_size", "delta_bwd_workspace_size",
    "qk_norm_fwd", "qk_norm_bwd", "qk_norm_bwd_workspace_size",
)


class GlacoreError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = _status_string(status)
        if status == ERR_CUDA:
            try:
                msg += ": " + load().glacore_last_cuda_error().decode()
            except OSError:
                pass
        super().__init__(f"glacore status {status} ({msg}){': ' + what if what else ''}")


class Problem(ctypes.Structure):
    """Mirror of ``glacore_problem`` in include/glacore.h."""

    _fields_ = [
        ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
        ("Hqk", ctypes.c_int64), ("K", ctypes.c_int64), ("V", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("chunk_size", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved0", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("segment_ids", ctypes.c_void_p), ("n_seqs", ctypes.c_int64),
        ("initial_state", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
    ]


class QkNorm(ctypes.Structure):
    """Mirror of ``glacore_qk_norm`` in include/glacore.h."""

    _fields_ = [
        ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64),
        ("D", ctypes.c_int64), ("R", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("l2", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
        ("reserved0", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p),
        ("cos_table", ctypes.c_void_p), ("sin_table", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("n_positions", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


_lib = None
_lock = threading.Lock()


def load(path: str | None = None):
    """Loads libglacore.so (building it first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if path is None:
            from . import _build

            if _build.needs_build():
                _build.build()
        lib = ctypes.CDLL(p)
        P = ctypes.c_void_p
        PP = ctypes.POINTER(Problem)
        for n in ("gla_fwd", "ssd_fwd"):
            f = getattr(lib, n)
            f.restype = ctypes.c_int
            f.argtypes = [PP, P, P, P]
        for n in ("gla_bwd", "ssd_bwd", "gla_bwd_noalloc"):
            f = getattr(lib, n)
            f.restype = ctypes.c_int
            f.argtypes = [PP, P, P, P, P, P, P, P, P]
        for n in ("gla_fwd_workspace_size", "gla_bwd_workspace_size", "ssd_fwd_workspace_size",
                  "ssd_bwd_workspace_size"):
            f = getattr(lib, n)
            f.restype = ctypes.c_size_t
            f.argtypes = [PP]
        lib.glacore_count_docs.restype = ctypes.c_int
        lib.glacore_count_docs.argtypes = [P, ctypes.c_int64, ctypes.c_int64, P, P]
        lib.glacore_get_device_error.restype = ctypes.c_int
        lib.glacore_get_device_error.argtypes = [P]
        lib.glacore_last_cuda_error.restype = ctypes.c_char_p
        lib.glacore_last_cuda_error.argtypes = []
        lib.glacore_status_string.restype = ctypes.c_char_p
        lib.glacore_status_string.argtypes = [ctypes.c_int]
        lib.glacore_version.restype = ctypes.c_int
        lib.glacore_version.argtypes = []
        lib.glacore_set_timing_events.restype = None
        lib.glacore_set_timing_events.argtypes = [P, ctypes.c_int]
        lib.glacore_timing_count.restype = ctypes.c_int
        lib.glacore_timing_count.argtypes = []
        lib.glacore_timing_label.restype = ctypes.c_char_p
        lib.glacore_timing_label.argtypes = [ctypes.c_int]
        lib.glacore_selftest_wait.restype = ctypes.c_int
        lib.glacore_selftest_wait.argtypes = [ctypes.c_int64, P]
        I64, I32, F = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        lib.norm_gate_fwd.restype = ctypes.c_int
        lib.norm_gate_fwd.argtypes = [P, P, P, I64, I64, I32, F, P, P]
        lib.norm_gate_bwd_workspace_size.restype = ctypes.c_size_t
        lib.norm_gate_bwd_workspace_size.argtypes = [I64, I64]
        lib.norm_gate_bwd.restype = ctypes.c_int
        lib.norm_gate_bwd.argtypes = [P, P, P, P, I64, I64, I32, F, P, P, P, P, ctypes.c_size_t, P]
        lib.short_conv_fwd.restype = ctypes.c_int
        lib.short_conv_fwd.argtypes = [P, P, P, P, I64, I64, I64, I32, I32, I32, P, P]
        lib.short_conv_bwd_workspace_size.restype = ctypes.c_size_t
        lib.short_conv_bwd_workspace_size.argtypes = [I64, I64, I64, I32]
        for n in ("gla_fwd_state",):
            getattr(lib, n).restype = ctypes.c_int
            getattr(lib, n).argtypes = [PP, P, P, P]
        lib.gla_bwd_state.restype = ctypes.c_int
        lib.gla_bwd_state.argtypes = [PP, P, P, P, P]
        lib.glacore_state_scan.restype = ctypes.c_int
        lib.glacore_state_scan.argtypes = [P, P, I64, I64, I64, I64, P, I64, I32, P, P]
        lib.short_conv_bwd.restype = ctypes.c_int
        lib.short_conv_bwd.argtypes = [P, P, P, P, P, I64, I64, I64, I32, I32, I32, P, P, P, P, ctypes.c_size_t, P]
        for n in ("gla_step", "ssd_step"):
            getattr(lib, n).restype = ctypes.c_int
            getattr(lib, n).argtypes = [P, P, I64, P, P, P]
        lib.layer_norm_fwd.restype = ctypes.c_int
        lib.layer_norm_fwd.argtypes = [P, P, P, I64, I64, I64, I32, F, P, P, P, P]
        lib.layer_norm_bwd_workspace_size.restype = ctypes.c_size_t
        lib.layer_norm_bwd_workspace_size.argtypes = [I64, I64]
        lib.layer_norm_bwd.restype = ctypes.c_int
        lib.layer_norm_bwd.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I32, P, P, P, P, ctypes.c_size_t, P]
        for n in ("linear_ce_fwd", "linear_ce_bwd"):
            getattr(lib, n + "_workspace_size").restype = ctypes.c_size_t
            getattr(lib, n + "_workspace_size").argtypes = [I64, I64, I64, I32]
            getattr(lib, n).restype = ctypes.c_int
        lib.linear_ce_fwd.argtypes = [P, P, P, I64, I64, I64, I64, I32, P, P, P, ctypes.c_size_t, P]
        lib.linear_ce_bwd.argtypes = [P, P, P, P, P, I64, I64, I64, I64, I32, P, P, P, ctypes.c_size_t, P]
        for n in ("delta_fwd_workspace_size", "delta_bwd_workspace_size", "qk_norm_bwd_workspace_size"):
            getattr(lib, n).restype = ctypes.c_size_t
            getattr(lib, n).argtypes = [P]
        for n, args in (("delta_fwd", 5), ("delta_bwd", 11), ("qk_norm_fwd", 4), ("qk_norm_bwd", 8)):
            getattr(lib, n).restype = ctypes.c_int
            getattr(lib, n).argtypes = [P] * args
        lib.delta_step.restype = ctypes.c_int
        lib.delta_step.argtypes = [P, P, P, I64, P, P, P]
        if path is None:
            _lib = lib
        return lib


def _status_string(s: int) -> str:
    try:
        return load().glacore_status_string(int(s)).decode()
    except OSError:
        return "unknown"


def _check(status: int, what: str):
    if status != OK:
        raise GlacoreError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(t):
    """The current stream of t's device as an integer handle, without the
    stream object (a call that takes a few microseconds feels the object)."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _call(fn, t, *args):
    """fn(*args, stream): on t's device and its current stream."""
    if torch._C._cuda_getDevice() == t.get_device():
        return fn(*args, _raw_stream(t))
    with torch.cuda.device(t.device):
        return fn(*args, _raw_stream(t))


def _addr(t):
    """Device address for a pointer argument (None: NULL)."""
    return None if t is None else t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _contig(t, dtype=None):
    if t is None:
        return None
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("glacore takes CUDA tensors")
    return t if t.is_contiguous() else t.contiguous()


def _same_device(device, **tensors):
    """Refuses a tensor (None: not given) that is not on `device`, the call's."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")


def _given(t, name, shape, dtype, device):
    """A caller's own output tensor, as the kernels write it: of this type and
    as many values (whatever axes it has), contiguous, on the call's device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device or t.numel() != math.prod(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of the values of {list(shape)} on {device}")
    return t


def _new(shape, dtype, device, poison):
    if poison:
        return torch.full(shape, float("nan"), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def count_docs(segment_ids: torch.Tensor) -> int:
    """Number of documents in segment_ids [B,T] (runs a kernel, then syncs)."""
    seg = _contig(segment_ids, torch.int32)
    B, T = seg.shape
    out = torch.empty(1, dtype=torch.int64, device=seg.device)
    _check(load().glacore_count_docs(_ptr(seg), B, T, _ptr(out), _stream(seg.device)), "count_docs")
    return int(out.item())


class LaunchTimer:
    """Per-kernel CUDA-event timing through the library's measurement hook.

    ``with LaunchTimer(n) as t: gla_fwd(...)`` records one event after each
    kernel launch of the call (of several: the last one's); ``t.labels`` names the kernels and
    ``t.events`` holds the torch events (elapsed times are read after a
    synchronize)."""

    def __init__(self, n: int = 8):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        for e in self.events:  # create the underlying CUDA events
            e.record()
        self._arr = (ctypes.c_void_p * n)(*[e.cuda_event for e in self.events])
        self.labels = []

    def __enter__(self):
        load().glacore_set_timing_events(ctypes.cast(self._arr, ctypes.c_void_p), len(self.events))
        return self

    def __exit__(self, *exc):
        lib = load()
        n = lib.glacore_timing_count()
        self.labels = [lib.glacore_timing_label(i).decode() for i in range(n)]
        lib.glacore_set_timing_events(None, 0)
        return False


def get_device_error():
    """Reads and clears the device error word; raises GlacoreError if set."""
    _check(load().glacore_get_device_error(_stream(torch.cuda.current_device())), "device")


def selftest_wait(cycles: int, device=None):
    """Runs the library's bounded-wait self-test on the current stream: a
    wait that can never complete, with a limit of ``cycles`` SM clocks.  The
    timeout lands in the device error word (read it with get_device_error)."""
    dev = torch.cuda.current_device() if device is None else device
    _check(load().glacore_selftest_wait(int(cycles), _stream(dev)), "selftest_wait")


def _rows(t):
    """(tensor, token stride): a [B, T, heads, D] tensor whose heads and
    channels are contiguous and whose tokens are evenly spaced (for example
    a slice of one fused projection [B, T, 3 * H * K]) is passed in place
    with its token stride; anything else is made contiguous (stride 0)."""
    if not t.is_cuda:
        raise ValueError("glacore takes CUDA tensors")
    if t.is_contiguous():
        return t, 0
    B, T, Hh, D = t.shape
    st = t.stride()
    if st[3] == 1 and st[2] == D and st[1] >= Hh * D and (B == 1 or st[0] == T * st[1]):
        return t, st[1]
    return t.contiguous(), 0


def _problem(q, k, v, g, scale, segment_ids, initial_state, chunk_size, n_seqs, head_gate):
    (q, qs), (k, ks), (v, vs) = _rows(q), _rows(k), _rows(v)
    g = _contig(g, torch.float32)
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    B, T, Hqk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    if tuple(k.shape) != (B, T, Hqk, K) or tuple(v.shape[:2]) != (B, T):
        raise ValueError("shape mismatch between q, k, v")
    if head_gate and tuple(g.shape) != (B, T, H):
        raise ValueError("SSD gate must be [B,T,H]")
    if not head_gate and tuple(g.shape) != (B, T, H, K):
        raise ValueError("GLA gate must be [B,T,H,K]")
    seg = _contig(segment_ids, torch.int32) if segment_ids is not None else None
    if seg is None:
        n = B if T > 0 else 0
    else:
        n = n_seqs if n_seqs is not None else count_docs(seg)
    h0 = _contig(initial_state, torch.float32) if initial_state is not None else None
    if h0 is not None and tuple(h0.shape) != (n, H, K, V):
        raise ValueError(f"initial_state must be [{n},{H},{K},{V}]")
    _same_device(q.device, k=k, v=v, g=g, segment_ids=seg, initial_state=h0)
    if scale is None:
        scale = K ** -0.5 if not head_gate else 1.0
    p = Problem(B=B, T=T, H=H, Hqk=Hqk, K=K, V=V, dtype=_dtype_code(q), chunk_size=int(chunk_size),
                scale=float(scale), reserved0=0, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(),
                g=g.data_ptr(), segment_ids=seg.data_ptr() if seg is not None else None, n_seqs=n,
                initial_state=h0.data_ptr() if h0 is not None else None, workspace=None,
                workspace_bytes=0, q_stride=qs, k_stride=ks, v_stride=vs)
    keep = (q, k, v, g, seg, h0)
    return p, keep


def workspace_size(p: Problem, kind: str) -> int:
    return int(getattr(load(), kind + "_workspace_size")(ctypes.byref(p)))


def _workspace(p, kind, device, workspace):
    need = workspace_size(p, kind)
    if need == 0:
        return None
    _same_device(device, workspace=workspace)
    if workspace is not None and workspace.numel() >= need and workspace.data_ptr() % 256 == 0:
        ws = workspace
    else:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    p.workspace = ws.data_ptr()
    p.workspace_bytes = ws.numel()
    return ws


def _fwd(kind, q, k, v, g, scale=None, segment_ids=None, initial_state=None,
         output_final_state=False, chunk_size=0, n_seqs=None, out=None, final_out=None,
         workspace=None, poison=False):
    head_gate = kind == "ssd"
    p, keep = _problem(q, k, v, g, scale, segment_ids, initial_state, chunk_size, n_seqs, head_gate)
    dev = keep[0].device
    o = out if out is not None else _new(tuple(keep[2].shape), keep[0].dtype, dev, poison)
    _given(o, "out", keep[2].shape, keep[0].dtype, dev)
    ht = None
    if output_final_state:
        ht = final_out if final_out is not None else _new((p.n_seqs, p.H, p.K, p.V), torch.float32, dev,
                                                          poison)
        _given(ht, "final_out", (p.n_seqs, p.H, p.K, p.V), torch.float32, dev)
    ws = _workspace(p, kind + "_fwd", dev, workspace)
    st = getattr(load(), kind + "_fwd")(ctypes.byref(p), _ptr(o), _ptr(ht), _stream(dev))
    _check(st, kind + "_fwd")
    del ws, keep
    return o, ht


def _bwd(kind, q, k, v, g, do, scale=None, segment_ids=None, initial_state=None, dht=None,
         chunk_size=0, n_seqs=None, outs=None, workspace=None, poison=False):
    head_gate = kind == "ssd"
    p, keep = _problem(q, k, v, g, scale, segment_ids, initial_state, chunk_size, n_seqs, head_gate)
    dev = keep[0].device
    do = _contig(do, keep[0].dtype)
    dht = _contig(dht, torch.float32) if dht is not None else None
    if tuple(do.shape) != tuple(keep[2].shape):
        raise ValueError("do must match v")
    if dht is not None and tuple(dht.shape) != (p.n_seqs, p.H, p.K, p.V):
        raise ValueError("dht must be [n_seqs,H,K,V]")
    _same_device(dev, do=do, dht=dht)
    if outs is not None:
        dq, dk, dv, dg, dh0 = outs
        for t, name, like in ((dq, "dq", keep[0]), (dk, "dk", keep[1]), (dv, "dv", keep[2]), (dg, "dg", keep[3])):
            _given(t, name, like.shape, like.dtype, dev)
        if dh0 is not None:
            _given(dh0, "dh0", (p.n_seqs, p.H, p.K, p.V), torch.float32, dev)
    else:
        dq = _new(tuple(keep[0].shape), keep[0].dtype, dev, poison)
        dk = _new(tuple(keep[1].shape), keep[0].dtype, dev, poison)
        dv = _new(tuple(keep[2].shape), keep[0].dtype, dev, poison)
        dg = _new(tuple(keep[3].shape), torch.float32, dev, poison)
        dh0 = _new((p.n_seqs, p.H, p.K, p.V), torch.float32, dev, poison) if initial_state is not None else None
    ws = _workspace(p, kind + "_bwd", dev, workspace)
    st = getattr(load(), kind + "_bwd")(ctypes.byref(p), _ptr(do), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv),
                                        _ptr(dg), _ptr(dh0), _stream(dev))
    _check(st, kind + "_bwd")
    del ws, keep
    return dq, dk, dv, dg, dh0


def gla_fwd(q, k, v, g, scale=None, segment_ids=None, initial_state=None, output_final_state=False,
            chunk_size=0, n_seqs=None, **kw):
    """GLA forward.  Returns (o, final_state or None)."""
    return _fwd("gla", q, k, v, g, scale, segment_ids, initial_state, output_final_state, chunk_size,
                n_seqs, **kw)


def gla_bwd(q, k, v, g, do, scale=None, segment_ids=None, initial_state=None, dht=None, chunk_size=0,
            n_seqs=None, **kw):
    """GLA backward.  Returns (dq, dk, dv, dg, dh0 or None)."""
    return _bwd("gla", q, k, v, g, do, scale, segment_ids, initial_state, dht, chunk_size, n_seqs, **kw)


def ssd_fwd(q, k, v, g, scale=1.0, segment_ids=None, initial_state=None, output_final_state=False,
            chunk_size=0, n_seqs=None, **kw):
    """Mamba-2 SSD forward (g is the per-head log decay [B,T,H])."""
    return _fwd("ssd", q, k, v, g, scale, segment_ids, initial_state, output_final_state, chunk_size,
                n_seqs, **kw)


def ssd_bwd(q, k, v, g, do, scale=1.0, segment_ids=None, initial_state=None, dht=None, chunk_size=0,
            n_seqs=None, **kw):
    """Mamba-2 SSD backward.  Returns (dq, dk, dv, dg, dh0 or None)."""
    return _bwd("ssd", q, k, v, g, do, scale, segment_ids, initial_state, dht, chunk_size, n_seqs, **kw)


# ---- the recurrence token by token -------------------------------------------
# glacore_problem as bytes: a call of a few microseconds feels a ctypes
# structure filled field by field
_PACK = struct.Struct("@6qiifi5PqPPN3q")
assert _PACK.size == ctypes.sizeof(Problem)


def _tokens(t):
    """_rows for the few tokens of a step, with the usual cases first: a
    [B, T, heads, D] tensor with contiguous heads whose tokens (over B, where T
    is 1) are evenly spaced goes in place."""
    if not t.is_cuda:
        raise ValueError("glacore takes CUDA tensors")
    B, T, Hh, D = t.shape
    s0, s1, s2, s3 = t.stride()
    if s3 == 1 and (s2 == D or Hh == 1):
        if T == 1:
            if s0 >= Hh * D:
                return t, s0
        elif s1 >= Hh * D and (B == 1 or s0 == T * s1):
            return t, s1
    return t.contiguous(), 0


def _step(kind, q, k, v, g, state, state_indices, scale, out, poison, beta=None):
    B, T, Hqk, K = q.shape
    H, V = v.shape[2:]
    dt = q.dtype
    if k.dtype != dt or v.dtype != dt:
        raise TypeError("q, k, v must share one dtype")
    if k.shape != q.shape or v.shape[0] != B or v.shape[1] != T:
        raise ValueError("shape mismatch between q, k, v")
    if tuple(g.shape) != ((B, T, H, K) if kind == "gla" else (B, T, H)):
        raise ValueError("gla_step's gate must be [B,T,H,K]" if kind == "gla" else f"{kind}_step's gate must be [B,T,H]")
    if beta is not None and beta.shape != g.shape:
        raise ValueError("delta_step's beta must be [B,T,H]")
    (q, qs), (k, ks), (v, vs) = _tokens(q), _tokens(k), _tokens(v)
    g, beta = _contig(g, torch.float32), _contig(beta, torch.float32)
    dev = q.get_device()
    if not (k.get_device() == v.get_device() == g.get_device() == state.get_device() == dev) or (
            state_indices is not None and state_indices.get_device() != dev) or (
            beta is not None and beta.get_device() != dev):
        _same_device(q.device, k=k, v=v, g=g, beta=beta, state=state, state_indices=state_indices)
    if not state.is_cuda or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor (it is updated in place)")
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, K, V):
        raise ValueError(f"state must be [n_slots,{H},{K},{V}]")
    idx = _contig(state_indices, torch.int32)
    if idx is not None and (idx.dim() != 1 or idx.shape[0] != B):
        raise ValueError("state_indices must be [B]")
    shape = (B, T, H, V)
    o = _given(out, "out", shape, dt, q.device) if out is not None else _new(shape, dt, q.device, poison)
    if scale is None:
        scale = K ** -0.5
    p = _PACK.pack(B, T, H, Hqk, K, V, _dtype_code(q), 0, scale, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                   g.data_ptr(), 0, B if T else 0, 0, 0, 0, qs, ks, vs)
    lib = _lib or load()
    if kind == "delta":
        st = _call(lib.delta_step, q, p, beta.data_ptr(), state.data_ptr(), state.shape[0], _addr(idx), o.data_ptr())
    else:
        st = (lib.gla_step if kind == "gla" else lib.ssd_step)(p, state.data_ptr(), state.shape[0], _addr(idx),
                                                               o.data_ptr(), _raw_stream(q))
    if st:
        _check(st, kind + "_step")
    return o


def gla_step(q, k, v, g, state, state_indices=None, scale=None, out=None, poison=False):
    """New tokens of B sequences (q, k, v, g as in gla_fwd, T usually 1) on the
    pool ``state`` [n_slots,H,K,V] fp32, which is updated in place.
    state_indices [B] int32 names each sequence's slot (distinct; negative:
    idle row, o = 0; None: slot b).  Returns o [B,T,H,V]."""
    return _step("gla", q, k, v, g, state, state_indices, scale, out, poison)


def ssd_step(q, k, v, g, state, state_indices=None, scale=1.0, out=None, poison=False):
    """gla_step with one log decay per head, g [B,T,H]."""
    return _step("ssd", q, k, v, g, state, state_indices, scale, out, poison)


# ---- the gated delta rule ------------------------------------------------------
class _DeltaProblem:
    """Checked operands of delta_fwd / delta_bwd and their glacore_problem as bytes."""

    __slots__ = ("q", "k", "v", "g", "beta", "seg", "h0", "n", "dtype", "device", "states", "fields")

    def __init__(self, q, k, v, g, beta, scale, segment_ids, initial_state, n_seqs):
        (q, qs), (k, ks), (v, vs) = _tokens(q), _tokens(k), _tokens(v)
        g, beta = _contig(g, torch.float32), _contig(beta, torch.float32)
        if not (q.dtype == k.dtype == v.dtype):
            raise TypeError("q, k, v must share one dtype")
        B, T, Hqk, K = q.shape
        H, V = v.shape[2:]
        if k.shape != q.shape or v.shape[0] != B or v.shape[1] != T:
            raise ValueError("shape mismatch between q, k, v")
        if tuple(g.shape) != (B, T, H) or beta.shape != g.shape:
            raise ValueError("the gate and beta must be [B,T,H]")
        seg, h0 = _contig(segment_ids, torch.int32), _contig(initial_state, torch.float32)
        if seg is not None and tuple(seg.shape) != (B, T):
            raise ValueError("segment_ids must be [B,T]")
        at = q.get_device()
        for t in (k, v, g, beta, seg, h0):
            if t is not None and t.get_device() != at:
                _same_device(q.device, k=k, v=v, g=g, beta=beta, segment_ids=seg, initial_state=h0)
        if seg is None:
            n = B if T > 0 else 0
        else:
            n = n_seqs if n_seqs is not None else count_docs(seg)
        self.states = (n, H, K, V)
        if h0 is not None and tuple(h0.shape) != self.states:
            raise ValueError(f"initial_state must be [{n},{H},{K},{V}]")
        self.q, self.k, self.v, self.g, self.beta, self.seg, self.h0, self.n = q, k, v, g, beta, seg, h0, n
        self.dtype, self.device = q.dtype, q.device
        self.fields = (B, T, H, Hqk, K, V, _dtype_code(q), 0, K ** -0.5 if scale is None else scale, 0, q.data_ptr(),
                       k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(seg) or 0, n, _addr(h0) or 0), (qs, ks, vs)

    def scratch(self, need_of, workspace):
        """(workspace or None, the problem's bytes with it)."""
        first, strides = self.fields
        p = _PACK.pack(*first, 0, 0, *strides)
        need = need_of(p)
        if not need:
            return None, p
        ws = _scratch(need, self.device, workspace)
        return ws, _PACK.pack(*first, ws.data_ptr(), ws.numel(), *strides)


def delta_fwd(q, k, v, g, beta, scale=None, segment_ids=None, initial_state=None, output_final_state=False,
              n_seqs=None, out=None, final_out=None, workspace=None, poison=False):
    """Gated delta rule over whole sequences:
        u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),  S_t = exp(g_t) S_{t-1} + k_t u_t^T,  o_t = scale S_t^T q_t
    q, k [B,T,Hqk,K] (k of unit length: qk_norm_fwd), v [B,T,H,V], g (log
    decay) and beta [B,T,H] fp32; scale K^-1/2 unless given.  segment_ids,
    initial_state and n_seqs as in ssd_fwd.  Returns (o, final_state or None)."""
    p = _DeltaProblem(q, k, v, g, beta, scale, segment_ids, initial_state, n_seqs)
    dev, dt, shape = p.device, p.dtype, p.v.shape
    o = _given(out, "out", shape, dt, dev) if out is not None else _new(tuple(shape), dt, dev, poison)
    ht = None
    if output_final_state:
        ht = (_given(final_out, "final_out", p.states, torch.float32, dev) if final_out is not None
              else _new(p.states, torch.float32, dev, poison))
    lib = _lib or load()
    ws, packed = p.scratch(lib.delta_fwd_workspace_size, workspace)
    st = _call(lib.delta_fwd, p.q, packed, p.beta.data_ptr(), o.data_ptr(), _addr(ht))
    if st:
        _check(st, "delta_fwd")
    return o, ht


def delta_bwd(q, k, v, g, beta, do, scale=None, segment_ids=None, initial_state=None, dht=None, n_seqs=None, outs=None,
              workspace=None, poison=False):
    """Gradients of delta_fwd.  do [B,T,H,V] and dht [n_seqs,H,K,V] (or None)
    are those of o and the final state.  Returns (dq, dk, dv, dg, dbeta, dh0
    or None)."""
    p = _DeltaProblem(q, k, v, g, beta, scale, segment_ids, initial_state, n_seqs)
    dev, dt = p.device, p.dtype
    do, dht = _contig(do, dt), _contig(dht, torch.float32)
    if do.shape != p.v.shape:
        raise ValueError("do must match v")
    if dht is not None and tuple(dht.shape) != p.states:
        raise ValueError("dht must be [n_seqs,H,K,V]")
    _same_device(dev, do=do, dht=dht)
    like = (p.q, p.k, p.v, p.g, p.beta)
    if outs is not None:
        dq, dk, dv, dg, dbeta, dh0 = outs
        for t, name, x in zip((dq, dk, dv, dg, dbeta), ("dq", "dk", "dv", "dg", "dbeta"), like):
            _given(t, name, x.shape, x.dtype, dev)
        if dh0 is not None:
            _given(dh0, "dh0", p.states, torch.float32, dev)
    else:
        dq, dk, dv, dg, dbeta = (_new(tuple(x.shape), x.dtype, dev, poison) for x in like)
        dh0 = _new(p.states, torch.float32, dev, poison) if initial_state is not None else None
    lib = _lib or load()
    ws, packed = p.scratch(lib.delta_bwd_workspace_size, workspace)
    st = _call(lib.delta_bwd, p.q, packed, p.beta.data_ptr(), do.data_ptr(), _addr(dht), dq.data_ptr(),
               dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _addr(dh0))
    if st:
        _check(st, "delta_bwd")
    return dq, dk, dv, dg, dbeta, dh0


def delta_step(q, k, v, g, beta, state, state_indices=None, scale=None, out=None, poison=False):
    """New tokens of B sequences by the gated delta rule, on a pool of states
    as in gla_step; g and beta [B,T,H]."""
    return _step("delta", q, k, v, g, state, state_indices, scale, out, poison, beta)


# ---- operations around the recurrence ---------------------------------------
# glacore_qk_norm as bytes (see _PACK)
_QK_PACK = struct.Struct("@6q3if8P3qPN")
_WS_PACK = struct.Struct("@PN")  # its last two fields
assert _QK_PACK.size == ctypes.sizeof(QkNorm)


def _qk_args(q, k, wq, wk, cos, sin, positions, eps, norm, interleaved):
    if q.dim() != 4 or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("qk_norm: q must be [B, T, Hq, D] and k [B, T, Hk, D]")
    if q.dtype != k.dtype:
        raise TypeError("qk_norm: q and k must share one dtype")
    if norm not in ("rms", "l2"):
        raise ValueError("qk_norm: norm must be 'rms' or 'l2'")
    if (cos is None) != (sin is None) or (cos is None and positions is not None):
        raise ValueError("qk_norm: cos, sin and positions go together")
    B, T, Hq, D = q.shape
    (q, qs), (k, ks) = _tokens(q), _tokens(k)
    wq, wk, cos, sin = (_contig(t, torch.float32) for t in (wq, wk, cos, sin))
    positions = _contig(positions, torch.int32)
    if (wq is not None and wq.shape != (D,)) or (wk is not None and wk.shape != (D,)):
        raise ValueError("qk_norm: wq and wk must be [D]")
    R = P = 0
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape or 2 * cos.shape[1] > D:
            raise ValueError("qk_norm: cos and sin must be [n_positions, R] with 2 R <= D")
        P, R = cos.shape
        if positions is None and T > P:
            raise ValueError("qk_norm: more tokens than positions in the tables")
        if positions is not None and positions.shape != (B, T):
            raise ValueError("qk_norm: positions must be [B, T]")
    dev = q.get_device()
    for t in (k, wq, wk, cos, sin, positions):
        if t is not None and t.get_device() != dev:
            _same_device(q.device, k=k, wq=wq, wk=wk, cos=cos, sin=sin, positions=positions)

    p = _QK_PACK.pack(B, T, Hq, k.shape[2], D, R, _dtype_code(q), int(norm == "l2"), int(bool(interleaved)), eps, 0,
                      q.data_ptr(), k.data_ptr(), _addr(wq) or 0, _addr(wk) or 0, _addr(cos) or 0, _addr(sin) or 0,
                      _addr(positions) or 0, P, qs, ks, 0, 0)
    return q, k, p, (wq, wk, cos, sin, positions)


def qk_norm_fwd(q, k, wq=None, wk=None, cos=None, sin=None, positions=None, eps=1e-6, norm="rms", interleaved=False,
                outs=None):
    """Norm of every query and key head and the rotation by position in one
    pass: per row of D channels x * (mean(x^2) + eps)^-1/2 * w ("l2": the sum
    in the mean's place), then its first R pairs of channels, (i, i + R) or
    interleaved (2 i, 2 i + 1), rotated by the angle whose cos and sin
    [n_positions, R] fp32 hold at the token's position.  q [B,T,Hq,D], k
    [B,T,Hk,D] (bf16 or fp32; views of one projection go in place), wq, wk [D]
    fp32 or None, positions [B,T] int32 or None (0 .. T - 1).  Returns (q, k)."""
    q, k, p, keep = _qk_args(q, k, wq, wk, cos, sin, positions, eps, norm, interleaved)
    dt, dev = q.dtype, q.device
    if outs is not None:
        qo, ko = _given(outs[0], "q out", q.shape, dt, dev), _given(outs[1], "k out", k.shape, dt, dev)
    else:
        qo, ko = torch.empty(q.shape, dtype=dt, device=dev), torch.empty(k.shape, dtype=dt, device=dev)
    st = _call((_lib or load()).qk_norm_fwd, q, p, qo.data_ptr(), ko.data_ptr())
    if st:
        _check(st, "qk_norm_fwd")
    return qo, ko


def qk_norm_bwd(q, k, dqo, dko, wq=None, wk=None, cos=None, sin=None, positions=None, eps=1e-6, norm="rms",
                interleaved=False, outs=None, workspace=None):
    """Gradients of qk_norm_fwd from those of its outputs: (dq, dk, dwq, dwk),
    the last two [D] fp32 (also without weights)."""
    q, k, p, keep = _qk_args(q, k, wq, wk, cos, sin, positions, eps, norm, interleaved)
    dt, dev = q.dtype, q.device
    if dqo.shape != q.shape or dko.shape != k.shape:
        raise ValueError("qk_norm: dqo and dko must match q and k")
    dqo, dko = _contig(dqo, dt), _contig(dko, dt)
    if not dqo.get_device() == dko.get_device() == q.get_device():
        _same_device(dev, dqo=dqo, dko=dko)
    D = q.shape[3]
    if outs is not None:
        dq, dk, dwq, dwk = outs
        for t, name, shape, ty in ((dq, "dq", q.shape, dt), (dk, "dk", k.shape, dt), (dwq, "dwq", (D,), torch.float32),
                                   (dwk, "dwk", (D,), torch.float32)):
            _given(t, name, shape, ty, dev)
    else:
        dq, dk = torch.empty(q.shape, dtype=dt, device=dev), torch.empty(k.shape, dtype=dt, device=dev)
        dwq, dwk = (torch.empty(D, dtype=torch.float32, device=dev) for _ in range(2))
    lib = _lib or load()
    ws = _scratch(lib.qk_norm_bwd_workspace_size(p), dev, workspace)
    p = p[:-16] + _WS_PACK.pack(ws.data_ptr(), ws.numel())
    st = _call(lib.qk_norm_bwd, q, p, dqo.data_ptr(), dko.data_ptr(), dq.data_ptr(),
               dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr())
    if st:
        _check(st, "qk_norm_bwd")
    return dq, dk, dwq, dwk


def _rows2d(t, name):
    """(tensor, rows, D, row stride) of a [..., D] tensor seen as rows of D
    values: evenly spaced rows are passed in place, anything else is copied."""
    if not t.is_cuda:
        raise ValueError("glacore takes CUDA tensors")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must be [..., D] with D >= 1")
    D = t.shape[-1]
    rows = t.numel() // D
    if t.is_contiguous():
        return t, rows, D, 0
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= D:
        return t, rows, D, t.stride(0)
    return t.contiguous(), rows, D, 0


def layer_norm_fwd(x, w=None, b=None, eps=1e-5, out=None):
    """Layer norm over the last axis: y = (x - mean) * rstd * w + b.  x [..., D]
    (bf16 or fp32; a 2-D x may have a row stride), w, b [D] fp32 or None.
    Returns (y, mean, rstd), the row statistics fp32 with x's leading shape."""
    x, rows, D, xs = _rows2d(x, "x")
    w, b = _contig(w, torch.float32), _contig(b, torch.float32)
    if (w is not None and w.shape != (D,)) or (b is not None and b.shape != (D,)):
        raise ValueError("layer_norm: w and b must be [D]")
    shape, dev = x.shape, x.device
    at = x.get_device()
    if (w is not None and w.get_device() != at) or (b is not None and b.get_device() != at):
        _same_device(dev, w=w, b=b)
    y = _given(out, "out", shape, x.dtype, dev) if out is not None else torch.empty(shape, dtype=x.dtype, device=dev)
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    st = (_lib or load()).layer_norm_fwd(x.data_ptr(), _addr(w), _addr(b), rows, D, xs, _dtype_code(x), eps,
                                         y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _raw_stream(x))
    if st:
        _check(st, "layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd(x, w, mean, rstd, dy, outs=None, workspace=None):
    """Returns (dx, dw, db) of layer_norm_fwd from its row statistics (dw and
    db fp32, also when the layer has no w or b)."""
    if x.shape != dy.shape or x.dtype != dy.dtype:
        raise ValueError("layer_norm: x and dy must match")
    x, rows, D, xs = _rows2d(x, "x")
    dy, _, _, ys = _rows2d(dy, "dy")
    w, mean, rstd = _contig(w, torch.float32), _contig(mean, torch.float32), _contig(rstd, torch.float32)
    if (w is not None and w.shape != (D,)) or mean.numel() != rows or rstd.numel() != rows:
        raise ValueError("layer_norm: w must be [D], mean and rstd one value per row")
    dev = x.device
    _same_device(dev, w=w, mean=mean, rstd=rstd, dy=dy)
    if outs is not None:
        dx, dw, db = outs
        _given(dx, "dx", x.shape, x.dtype, dev)
        _given(dw, "dw", (D,), torch.float32, dev)
        _given(db, "db", (D,), torch.float32, dev)
    else:
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        dw = torch.empty(D, dtype=torch.float32, device=dev)
        db = torch.empty(D, dtype=torch.float32, device=dev)
    lib = _lib or load()
    ws = _scratch(lib.layer_norm_bwd_workspace_size(rows, D), dev, workspace)
    st = lib.layer_norm_bwd(x.data_ptr(), _addr(w), mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(), rows, D, xs, ys,
                            _dtype_code(x), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel(),
                            _raw_stream(x))
    if st:
        _check(st, "layer_norm_bwd")
    return dx, dw, db


def norm_gate_fwd(o, z, w, eps=1e-5, out=None):
    """Per-head RMSNorm times a swish gate over the last axis (V):
    y = o * rsqrt(mean(o^2) + eps) * w * z * sigmoid(z).  o, z [..., V]
    (bf16 or fp32, same dtype), w [V] fp32."""
    o, z = _contig(o), _contig(z)
    w = _contig(w, torch.float32)
    if o.shape != z.shape or o.dtype != z.dtype or tuple(w.shape) != (o.shape[-1],):
        raise ValueError("norm_gate: o and z must match and w must be [V]")
    V = o.shape[-1]
    rows = o.numel() // V if V else 0
    _same_device(o.device, z=z, w=w)
    y = _given(out, "out", o.shape, o.dtype, o.device) if out is not None else torch.empty_like(o)
    st = load().norm_gate_fwd(_ptr(o), _ptr(z), _ptr(w), rows, V, _dtype_code(o), float(eps), _ptr(y),
                              _stream(o.device))
    _check(st, "norm_gate_fwd")
    return y


def norm_gate_bwd(o, z, w, dy, eps=1e-5, outs=None, workspace=None):
    """Returns (do, dz, dw) of norm_gate_fwd."""
    o, z, dy = _contig(o), _contig(z), _contig(dy)
    w = _contig(w, torch.float32)
    if not (o.shape == z.shape == dy.shape) or not (o.dtype == z.dtype == dy.dtype):
        raise ValueError("norm_gate: o, z and dy must match")
    _same_device(o.device, z=z, w=w, dy=dy, workspace=workspace)
    V = o.shape[-1]
    rows = o.numel() // V if V else 0
    if outs is not None:
        do, dz, dw = outs
        _given(do, "do", o.shape, o.dtype, o.device)
        _given(dz, "dz", o.shape, o.dtype, o.device)
        _given(dw, "dw", (V,), torch.float32, o.device)
    else:
        do, dz = torch.empty_like(o), torch.empty_like(z)
        dw = torch.empty(V, dtype=torch.float32, device=o.device)
    lib = load()
    need = int(lib.norm_gate_bwd_workspace_size(rows, V))
    ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
        max(need, 256), dtype=torch.uint8, device=o.device)
    st = lib.norm_gate_bwd(_ptr(o), _ptr(z), _ptr(w), _ptr(dy), rows, V, _dtype_code(o), float(eps), _ptr(do),
                           _ptr(dz), _ptr(dw), _ptr(ws), ws.numel(), _stream(o.device))
    _check(st, "norm_gate_bwd")
    return do, dz, dw


def _ce_args(x, w, target):
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1] or x.dtype != w.dtype:
        raise ValueError("linear_ce: x must be [N, D] and w [V, D] of one dtype")
    if x.device != w.device or x.device != target.device:
        raise ValueError("linear_ce: x, w and target must be on one device")
    target = _contig(target, torch.int64)
    if tuple(target.shape) != (x.shape[0],):
        raise ValueError("linear_ce: target must be [N]")
    x, N, D, xs = _rows2d(x, "x")
    if x.data_ptr() % 16 or (x.dtype == torch.bfloat16 and D % 8 == 0 and xs % 8):
        x, xs = x.clone(memory_format=torch.contiguous_format), 0
    w = _contig(w)
    if w.data_ptr() % 16:
        w = w.clone()
    return x, w, target, N, D, w.shape[0], xs


def _scratch(need, device, workspace):
    _same_device(device, workspace=workspace)
    if workspace is not None and workspace.numel() >= need and workspace.data_ptr() % 256 == 0:
        return workspace
    return torch.empty(max(need, 256), dtype=torch.uint8, device=device)


def linear_ce_fwd(x, w, target, outs=None, workspace=None):
    """Softmax cross entropy of the output projection: for logits z = x w^T
    (never kept), lse = logsumexp(z) and loss = lse - z[target] per token.
    x [N, D] (may have a row stride), w [V, D] (bf16 or fp32), target [N] int64
    (negative: not scored, loss 0).  Returns (loss, lse), [N] fp32."""
    x, w, target, N, D, V, xs = _ce_args(x, w, target)
    code = _dtype_code(x)
    if outs is not None:
        loss, lse = (_given(o, n, (N,), torch.float32, x.device) for o, n in zip(outs, ("loss", "lse")))
    else:
        loss = torch.empty(N, dtype=torch.float32, device=x.device)
        lse = torch.empty(N, dtype=torch.float32, device=x.device)
    lib = _lib or load()
    ws = _scratch(lib.linear_ce_fwd_workspace_size(N, D, V, code), x.device, workspace)
    st = lib.linear_ce_fwd(x.data_ptr(), w.data_ptr(), target.data_ptr(), N, D, V, xs, code, loss.data_ptr(),
                           lse.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(x))
    if st:
        _check(st, "linear_ce_fwd")
    return loss, lse


def linear_ce_bwd(x, w, target, lse, dloss, outs=None, workspace=None):
    """Gradients of sum(dloss * loss) of linear_ce_fwd, from its lse: returns
    (dx [N, D], dw [V, D]) in the operands' dtype.  dloss [N] fp32 (1 / count
    for a mean)."""
    x, w, target, N, D, V, xs = _ce_args(x, w, target)
    lse, dloss = _contig(lse, torch.float32), _contig(dloss, torch.float32)
    if tuple(lse.shape) != (N,) or tuple(dloss.shape) != (N,):
        raise ValueError("linear_ce: lse and dloss must be [N]")
    _same_device(x.device, lse=lse, dloss=dloss)
    code = _dtype_code(x)
    if outs is not None:
        dx, dw = outs
        _given(dx, "dx", (N, D), x.dtype, x.device)
        _given(dw, "dw", (V, D), x.dtype, x.device)
    else:
        dx = torch.empty((N, D), dtype=x.dtype, device=x.device)
        dw = torch.empty((V, D), dtype=x.dtype, device=x.device)
    lib = _lib or load()
    ws = _scratch(lib.linear_ce_bwd_workspace_size(N, D, V, code), x.device, workspace)
    st = lib.linear_ce_bwd(x.data_ptr(), w.data_ptr(), target.data_ptr(), lse.data_ptr(), dloss.data_ptr(), N, D, V,
                           xs, code, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(x))
    if st:
        _check(st, "linear_ce_bwd")
    return dx, dw


def short_conv_fwd(x, w, b=None, segment_ids=None, activation=True, out=None):
    """Depthwise causal short convolution (+ SiLU) of x [B,T,D]; w [Kc,D]
    fp32 (tap k reads x_{t-(Kc-1-k)}), b [D] fp32 or None, segment_ids
    [B,T] int32 or None."""
    x = _contig(x)
    w = _contig(w, torch.float32)
    b = _contig(b, torch.float32) if b is not None else None
    seg = _contig(segment_ids, torch.int32) if segment_ids is not None else None
    B, T, D = x.shape
    Kc = w.shape[0]
    if tuple(w.shape) != (Kc, D) or (b is not None and tuple(b.shape) != (D,)):
        raise ValueError("short_conv: w must be [Kc, D] and b [D]")
    _same_device(x.device, w=w, b=b, segment_ids=seg)
    y = _given(out, "out", x.shape, x.dtype, x.device) if out is not None else torch.empty_like(x)
    st = load().short_conv_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(seg), B, T, D, Kc, _dtype_code(x),
                               1 if activation else 0, _ptr(y), _stream(x.device))
    _check(st, "short_conv_fwd")
    return y


def short_conv_bwd(x, w, b, dy, segment_ids=None, activation=True, outs=None, workspace=None):
    """Returns (dx, dw, db) of short_conv_fwd (db also when b is None)."""
    x, dy = _contig(x), _contig(dy)
    w = _contig(w, torch.float32)
    b = _contig(b, torch.float32) if b is not None else None
    seg = _contig(segment_ids, torch.int32) if segment_ids is not None else None
    B, T, D = x.shape
    Kc = w.shape[0]
    _same_device(x.device, w=w, b=b, dy=dy, segment_ids=seg, workspace=workspace)
    if outs is not None:
        dx, dw, db = outs
        _given(dx, "dx", x.shape, x.dtype, x.device)
        _given(dw, "dw", (Kc, D), torch.float32, x.device)
        _given(db, "db", (D,), torch.float32, x.device)
    else:
        dx = torch.empty_like(x)
        dw = torch.empty(Kc, D, dtype=torch.float32, device=x.device)
        db = torch.empty(D, dtype=torch.float32, device=x.device)
    lib = load()
    need = int(lib.short_conv_bwd_workspace_size(B, T, D, Kc))
    ws = workspace if workspace is not None and workspace.numel() >= need else torch.empty(
        max(need, 256), dtype=torch.uint8, device=x.device)
    st = lib.short_conv_bwd(_ptr(x), _ptr(w), _ptr(b), _ptr(seg), _ptr(dy), B, T, D, Kc, _dtype_code(x),
                            1 if activation else 0, _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), ws.numel(),
                            _stream(x.device))
    _check(st, "short_conv_bwd")
    return dx, dw, db


# ---- sequence split across devices ------------------------------------------
def gla_fwd_state(q, k, v, g, scale=None):
    """Local end state (from a zero initial state) and total decay of every
    row: (L [B,H,K,V] fp32, D [B,H,K] fp32).  GLA, no segment_ids."""
    p, keep = _problem(q, k, v, g, scale, None, None, 0, None, False)
    dev = keep[0].device
    L = torch.empty((p.n_seqs, p.H, p.K, p.V), dtype=torch.float32, device=dev)
    D = torch.empty((p.n_seqs, p.H, p.K), dtype=torch.float32, device=dev)
    _check(load().gla_fwd_state(ctypes.byref(p), _ptr(L), _ptr(D), _stream(dev)), "gla_fwd_state")
    del keep
    return L, D


def gla_bwd_state(q, k, v, g, do, scale=None):
    """Local state gradient at the start of every row (from a zero gradient
    at its end) and total decay: (L [B,H,K,V] fp32, D [B,H,K] fp32)."""
    p, keep = _problem(q, k, v, g, scale, None, None, 0, None, False)
    dev = keep[0].device
    do = _contig(do, keep[0].dtype)
    L = torch.empty((p.n_seqs, p.H, p.K, p.V), dtype=torch.float32, device=dev)
    D = torch.empty((p.n_seqs, p.H, p.K), dtype=torch.float32, device=dev)
    _check(load().gla_bwd_state(ctypes.byref(p), _ptr(do), _ptr(L), _ptr(D), _stream(dev)), "gla_bwd_state")
    del keep
    return L, D


def state_scan(L, D, r, seed=None, reverse=False):
    """Fold of the stacked piece states L [R, *mats, K, V] / decays
    D [R, *mats, K] for piece r (forward: pieces before r; reverse: after r),
    starting from seed [*mats, K, V] (or zero)."""
    L = _contig(L, torch.float32)
    D = _contig(D, torch.float32)
    seed = _contig(seed, torch.float32) if seed is not None else None
    R, K, V = L.shape[0], L.shape[-2], L.shape[-1]
    mats = L[0].numel() // (K * V)
    out = torch.empty(L.shape[1:], dtype=torch.float32, device=L.device)
    _check(load().glacore_state_scan(_ptr(L), _ptr(D), R, mats, K, V, _ptr(seed), int(r), 1 if reverse else 0,
                                     _ptr(out), _stream(L.device)), "state_scan")
    return out
