"""Thin ctypes binding of the C ABI in ``include/ssd.h``.

The functions carry the C names (``ssd_workspace_size``, ``ssd_forward``,
``ssd_backward``, ``ssd_status_string``) and only marshal arguments: torch
tensors become device pointers, the torch stream becomes a ``cudaStream_t``,
and a non-OK status becomes an :class:`SSDError`.  Every step of the scan runs
in the library's kernels; there is no fallback of any kind.  If the library
cannot be loaded the call raises.

Convenience wrappers :func:`forward` and :func:`backward` allocate outputs
and the workspace with torch (device memory only) and call the ABI.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

VARIANTS = {"mamba2": 0, "mamba1": 1, "mimo": 2}
DTYPES = {"f32": 0, "bf16": 1}
_TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}

SSD_OK, SSD_ERR_TIMEOUT = 0, 7


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {ssd_status_string(status)} (status {status})")


class ssd_problem(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("chunk", ctypes.c_int64),
                ("mimo_rank", ctypes.c_int64)]


EXPORTS = ("ssd_workspace_size", "ssd_forward", "ssd_backward", "ssd_forward_static", "ssd_profile_start",
           "ssd_profile_stop", "ssd_status_string", "ssd_version", "ssd_states_size", "ssd_forward_stash",
           "ssd_backward_stashed", "ssd_forward_static_status", "ssd_read_status", "ssd_wait_selftest",
           "ssd_checkpoints_size", "ssd_forward_checkpointed", "ssd_backward_checkpointed",
           "ssd_kda_workspace_size", "ssd_kda_forward", "ssd_kda_backward", "ssd_delta_workspace_size",
           "ssd_delta_stash_size", "ssd_delta_forward", "ssd_delta_backward", "ssd_delta_step",
           "ssd_norm_workspace_size", "ssd_norm_forward", "ssd_norm_backward")


class ssd_kda_problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("value_heads", ctypes.c_int64), ("key_dim", ctypes.c_int64), ("value_dim", ctypes.c_int64)]


class ssd_delta_problem(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("packed", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("value_heads", ctypes.c_int64), ("key_dim", ctypes.c_int64),
                ("value_dim", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


class ssd_norm_problem(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("x_stride", ctypes.c_int64)]


class ssd_kernel_time(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("ms", ctypes.c_float)]

_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load (building first if needed) the in-tree shared library."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.build()
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library missing: {p}")
        lib = ctypes.CDLL(p)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        lib.ssd_workspace_size.argtypes = [ctypes.POINTER(ssd_problem), i32, ctypes.POINTER(sz)]
        lib.ssd_workspace_size.restype = i32
        lib.ssd_forward.argtypes = [ctypes.POINTER(ssd_problem)] + [vp] * 8 + [vp, sz, vp]
        lib.ssd_forward.restype = i32
        lib.ssd_backward.argtypes = [ctypes.POINTER(ssd_problem)] + [vp] * 14 + [vp, sz, vp]
        lib.ssd_backward.restype = i32
        lib.ssd_status_string.argtypes = [i32]
        lib.ssd_status_string.restype = ctypes.c_char_p
        lib.ssd_forward_static.argtypes = [ctypes.POINTER(ssd_problem)] + [vp] * 8 + [vp]
        lib.ssd_forward_static.restype = i32
        lib.ssd_profile_start.argtypes = [i32]
        lib.ssd_profile_start.restype = i32
        lib.ssd_profile_stop.argtypes = [ctypes.POINTER(ssd_kernel_time), i32, ctypes.POINTER(i32)]
        lib.ssd_profile_stop.restype = i32
        lib.ssd_version.argtypes = []
        lib.ssd_version.restype = i32
        lib.ssd_states_size.argtypes = [ctypes.POINTER(ssd_problem), ctypes.POINTER(sz)]
        lib.ssd_states_size.restype = i32
        lib.ssd_forward_stash.argtypes = [ctypes.POINTER(ssd_problem)] + [vp] * 9 + [sz, vp, sz, vp]
        lib.ssd_forward_stash.restype = i32
        lib.ssd_backward_stashed.argtypes = [ctypes.POINTER(ssd_problem)] + [vp] * 8 + [sz] + [vp] * 7 + [sz, vp]
        lib.ssd_backward_stashed.restype = i32
        lib.ssd_forward_static_status.argtypes = [ctypes.POINTER(ctypes.c_int32), vp]
        lib.ssd_forward_static_status.restype = i32
        lib.ssd_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
        lib.ssd_read_status.restype = i32
        lib.ssd_wait_selftest.argtypes = [vp, ctypes.c_uint32, vp]
        lib.ssd_wait_selftest.restype = i32
        i64 = ctypes.c_int64
        lib.ssd_checkpoints_size.argtypes = [ctypes.POINTER(ssd_problem), i64, ctypes.POINTER(sz)]
        lib.ssd_checkpoints_size.restype = i32
        lib.ssd_forward_checkpointed.argtypes = [ctypes.POINTER(ssd_problem)] + [vp] * 8 + [i64, vp, sz, vp, sz, vp]
        lib.ssd_forward_checkpointed.restype = i32
        lib.ssd_backward_checkpointed.argtypes = ([ctypes.POINTER(ssd_problem)] + [vp] * 7 + [i64, vp, sz] + [vp] * 6 +
                                                 [vp, sz, vp])
        lib.ssd_backward_checkpointed.restype = i32
        kp = ctypes.POINTER(ssd_kda_problem)
        lib.ssd_kda_workspace_size.argtypes = [kp, i32, ctypes.POINTER(sz)]
        lib.ssd_kda_workspace_size.restype = i32
        lib.ssd_kda_forward.argtypes = [kp] + [vp] * 6 + [ctypes.c_float, vp, vp, vp, sz, vp]
        lib.ssd_kda_forward.restype = i32
        lib.ssd_kda_backward.argtypes = [kp] + [vp] * 8 + [ctypes.c_float] + [vp] * 6 + [vp, sz, vp]
        lib.ssd_kda_backward.restype = i32
        dp, f32 = ctypes.POINTER(ssd_delta_problem), ctypes.c_float
        lib.ssd_delta_workspace_size.argtypes = [dp, i32, i32, ctypes.POINTER(sz)]
        lib.ssd_delta_workspace_size.restype = i32
        lib.ssd_delta_stash_size.argtypes = [dp, ctypes.POINTER(sz)]
        lib.ssd_delta_stash_size.restype = i32
        lib.ssd_delta_forward.argtypes = [dp] + [vp] * 7 + [f32, vp, vp, vp, sz, vp, sz, vp]
        lib.ssd_delta_forward.restype = i32
        lib.ssd_delta_backward.argtypes = [dp] + [vp] * 9 + [f32] + [vp] * 6 + [vp, sz, vp, sz, vp]
        lib.ssd_delta_backward.restype = i32
        lib.ssd_delta_step.argtypes = [dp] + [vp] * 7 + [i64, f32, vp, vp]
        lib.ssd_delta_step.restype = i32
        np_ = ctypes.POINTER(ssd_norm_problem)
        lib.ssd_norm_workspace_size.argtypes = [np_, ctypes.POINTER(sz)]
        lib.ssd_norm_workspace_size.restype = i32
        lib.ssd_norm_forward.argtypes = [np_] + [vp] * 3 + [f32] + [vp] * 4
        lib.ssd_norm_forward.restype = i32
        lib.ssd_norm_backward.argtypes = [np_] + [vp] * 9 + [sz, vp]
        lib.ssd_norm_backward.restype = i32
        _lib = lib
        return lib


def problem(cfg: dict) -> ssd_problem:
    """An ``ssd_problem`` from a config dict (see ``configs.py``)."""
    return ssd_problem(VARIANTS[cfg["variant"]], DTYPES[cfg["dtype"]], cfg["batch"], cfg["seqlen"], cfg["nheads"],
                       cfg["headdim"], cfg["dstate"], cfg["ngroups"], cfg["chunk"], cfg["mimo_rank"])


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None):
    """The ``cudaStream_t`` of a call.  With the index of the tensors' device the current stream's handle is looked up
    without making a stream object, which a call of a few microseconds notices."""
    if stream is None:
        if device is not None and _raw_stream is not None:
            return _raw_stream(device)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def ssd_status_string(status: int) -> str:
    return load().ssd_status_string(int(status)).decode()


def ssd_workspace_size(prob: ssd_problem, backward: bool) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_workspace_size(ctypes.byref(prob), int(bool(backward)), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_workspace_size")
    return out.value


def ssd_forward(prob, x, dt_raw, A, B, C, s0, y, s_final, ws, ws_bytes, stream=None) -> None:
    st = load().ssd_forward(ctypes.byref(prob), _ptr(x), _ptr(dt_raw), _ptr(A), _ptr(B), _ptr(C), _ptr(s0),
                            _ptr(y), _ptr(s_final), _ptr(ws), int(ws_bytes), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_forward")


def ssd_forward_static(prob, x, dt_raw, A, B, C, s0, y, s_final, stream=None) -> None:
    """Forward without a workspace: the library's fixed 32 MiB device array is
    the scratch (see include/ssd.h).  Raises SSDError on a non-OK status."""
    st = load().ssd_forward_static(ctypes.byref(prob), _ptr(x), _ptr(dt_raw), _ptr(A), _ptr(B), _ptr(C), _ptr(s0),
                                   _ptr(y), _ptr(s_final), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_forward_static")


def ssd_forward_static_status(stream=None, read: bool = True) -> tuple:
    """(status, code) of the fixed array's device status word, read after the work enqueued on `stream`;
    with read=False only the start-up step (module load and address lookup) runs and code is None."""
    if not read:
        return load().ssd_forward_static_status(None, _stream(stream)), None
    code = ctypes.c_int32(-1)
    st = load().ssd_forward_static_status(ctypes.byref(code), _stream(stream))
    return st, code.value


def ssd_read_status(ws, stream=None) -> tuple:
    """(status, code) of the device status word in the first 4 bytes of the workspace `ws`."""
    code = ctypes.c_int32(-1)
    st = load().ssd_read_status(_ptr(ws), ctypes.byref(code), _stream(stream))
    return st, code.value


def ssd_wait_selftest(ws, limit_us: int, stream=None) -> int:
    """Launch the kernel whose bounded wait runs out after limit_us; returns the call's status."""
    return load().ssd_wait_selftest(_ptr(ws), int(limit_us), _stream(stream))


def ssd_backward(prob, dy, ds_final, x, dt_raw, A, B, C, s0, dx, ddt_raw, dA, dB, dC, ds0, ws, ws_bytes,
                 stream=None) -> None:
    st = load().ssd_backward(ctypes.byref(prob), _ptr(dy), _ptr(ds_final), _ptr(x), _ptr(dt_raw), _ptr(A), _ptr(B),
                             _ptr(C), _ptr(s0), _ptr(dx), _ptr(ddt_raw), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(ds0),
                             _ptr(ws), int(ws_bytes), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_backward")


def ssd_states_size(prob: ssd_problem) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_states_size(ctypes.byref(prob), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_states_size")
    return out.value


def ssd_forward_stash(prob, x, dt_raw, A, B, C, s0, y, s_final, states, states_bytes, ws, ws_bytes,
                      stream=None) -> None:
    st = load().ssd_forward_stash(ctypes.byref(prob), _ptr(x), _ptr(dt_raw), _ptr(A), _ptr(B), _ptr(C), _ptr(s0),
                                  _ptr(y), _ptr(s_final), _ptr(states), int(states_bytes), _ptr(ws), int(ws_bytes),
                                  _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_forward_stash")


def ssd_checkpoints_size(prob: ssd_problem, every: int) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_checkpoints_size(ctypes.byref(prob), int(every), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_checkpoints_size")
    return out.value


def ssd_forward_checkpointed(prob, x, dt_raw, A, B, C, s0, y, s_final, every, ckpt, ckpt_bytes, ws, ws_bytes,
                             stream=None) -> None:
    st = load().ssd_forward_checkpointed(ctypes.byref(prob), _ptr(x), _ptr(dt_raw), _ptr(A), _ptr(B), _ptr(C),
                                         _ptr(s0), _ptr(y), _ptr(s_final), int(every), _ptr(ckpt), int(ckpt_bytes),
                                         _ptr(ws), int(ws_bytes), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_forward_checkpointed")


def ssd_backward_checkpointed(prob, dy, ds_final, x, dt_raw, A, B, C, every, ckpt, ckpt_bytes, dx, ddt_raw, dA, dB,
                              dC, ds0, ws, ws_bytes, stream=None) -> None:
    st = load().ssd_backward_checkpointed(ctypes.byref(prob), _ptr(dy), _ptr(ds_final), _ptr(x), _ptr(dt_raw), _ptr(A),
                                          _ptr(B), _ptr(C), int(every), _ptr(ckpt), int(ckpt_bytes), _ptr(dx),
                                          _ptr(ddt_raw), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(ds0), _ptr(ws),
                                          int(ws_bytes), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_backward_checkpointed")


def ssd_backward_stashed(prob, dy, ds_final, x, dt_raw, A, B, C, states, states_bytes, dx, ddt_raw, dA, dB, dC,
                         ds0, ws, ws_bytes, stream=None) -> None:
    st = load().ssd_backward_stashed(ctypes.byref(prob), _ptr(dy), _ptr(ds_final), _ptr(x), _ptr(dt_raw), _ptr(A),
                                     _ptr(B), _ptr(C), _ptr(states), int(states_bytes), _ptr(dx), _ptr(ddt_raw),
                                     _ptr(dA), _ptr(dB), _ptr(dC), _ptr(ds0), _ptr(ws), int(ws_bytes),
                                     _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_backward_stashed")


def ssd_profile_start(capacity: int) -> None:
    st = load().ssd_profile_start(int(capacity))
    if st != SSD_OK:
        raise SSDError(st, "ssd_profile_start")


def ssd_profile_stop(capacity: int = 1 << 16) -> list:
    """Returns [(kernel name, ms)] for every launch recorded since start."""
    buf = (ssd_kernel_time * capacity)()
    n = ctypes.c_int(0)
    st = load().ssd_profile_stop(buf, int(capacity), ctypes.byref(n))
    if st != SSD_OK:
        raise SSDError(st, "ssd_profile_stop")
    return [(buf[i].kernel.decode(), float(buf[i].ms)) for i in range(n.value)]


# ---------------------------------------------------------------- conveniences
def _workspace(prob, backward, device):
    n = ssd_workspace_size(prob, backward)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device), n


def forward(cfg: dict, x, dt_raw, A, B, C, s0=None, stream=None, workspace=None):
    """Allocate y and s_final, run ``ssd_forward``; returns (y, s_final)."""
    prob = problem(cfg)
    dev = x.device
    y = torch.empty_like(x)
    sf_shape = (cfg["batch"], cfg["nheads"], cfg["dstate"]) if cfg["variant"] == "mamba1" else \
        (cfg["batch"], cfg["nheads"], cfg["headdim"], cfg["dstate"])
    s_final = torch.empty(sf_shape, dtype=torch.float32, device=dev)
    ws, n = workspace if workspace is not None else _workspace(prob, False, dev)
    ssd_forward(prob, x, dt_raw, A, B, C, s0, y, s_final, ws, n, stream)
    return y, s_final


def backward(cfg: dict, dy, ds_final, x, dt_raw, A, B, C, s0=None, stream=None, workspace=None):
    """Allocate the gradients, run ``ssd_backward``; returns a dict with
    dx, ddt_raw, dA (None for MIMO), dB, dC, ds0."""
    prob = problem(cfg)
    dev = x.device
    out = {"dx": torch.empty_like(x), "ddt_raw": torch.empty_like(dt_raw),
           "dA": None if A is None else torch.empty_like(A), "dB": torch.empty_like(B), "dC": torch.empty_like(C),
           "ds0": torch.empty_like(ds_final)}
    ws, n = workspace if workspace is not None else _workspace(prob, True, dev)
    ssd_backward(prob, dy, ds_final, x, dt_raw, A, B, C, s0, out["dx"], out["ddt_raw"], out["dA"], out["dB"],
                 out["dC"], out["ds0"], ws, n, stream)
    return out


def forward_stash(cfg: dict, x, dt_raw, A, B, C, s0=None, stream=None, workspace=None):
    """``forward`` that also keeps the chunk states; returns (y, s_final, states)
    with states a uint8 device tensor for ``backward_stashed``."""
    prob = problem(cfg)
    dev = x.device
    y = torch.empty_like(x)
    s_final = torch.empty((cfg["batch"], cfg["nheads"], cfg["headdim"], cfg["dstate"]), dtype=torch.float32,
                          device=dev)
    nst = ssd_states_size(prob)
    states = torch.empty(nst, dtype=torch.uint8, device=dev)
    ws, n = workspace if workspace is not None else _workspace(prob, False, dev)
    ssd_forward_stash(prob, x, dt_raw, A, B, C, s0, y, s_final, states, nst, ws, n, stream)
    return y, s_final, states


def backward_stashed(cfg: dict, dy, ds_final, x, dt_raw, A, B, C, states, stream=None, workspace=None):
    """``backward`` from the chunk states ``forward_stash`` kept (no s0, no
    forward replay); returns the same dict."""
    prob = problem(cfg)
    dev = x.device
    out = {"dx": torch.empty_like(x), "ddt_raw": torch.empty_like(dt_raw), "dA": torch.empty_like(A),
           "dB": torch.empty_like(B), "dC": torch.empty_like(C), "ds0": torch.empty_like(ds_final)}
    ws, n = workspace if workspace is not None else _workspace(prob, True, dev)
    ssd_backward_stashed(prob, dy, ds_final, x, dt_raw, A, B, C, states, states.numel(), out["dx"], out["ddt_raw"],
                         out["dA"], out["dB"], out["dC"], out["ds0"], ws, n, stream)
    return out


def forward_checkpointed(cfg: dict, x, dt_raw, A, B, C, s0=None, every: int = 8, stream=None, workspace=None):
    """``forward`` that also keeps fp32 checkpoints every ``every`` chunks; returns (y, s_final, ckpt) with ckpt
    a float32 device tensor [b, H, ceil(nc / every), P, N] for ``backward_checkpointed``."""
    prob = problem(cfg)
    dev = x.device
    y = torch.empty_like(x)
    s_final = torch.empty((cfg["batch"], cfg["nheads"], cfg["headdim"], cfg["dstate"]), dtype=torch.float32,
                          device=dev)
    nbytes = ssd_checkpoints_size(prob, every)
    nc = -(-cfg["seqlen"] // cfg["chunk"])
    nk = -(-nc // every)
    ckpt = torch.empty((cfg["batch"], cfg["nheads"], nk, cfg["headdim"], cfg["dstate"]), dtype=torch.float32,
                       device=dev)
    assert ckpt.numel() * 4 == nbytes
    ws, n = workspace if workspace is not None else _workspace(prob, False, dev)
    ssd_forward_checkpointed(prob, x, dt_raw, A, B, C, s0, y, s_final, every, ckpt, nbytes, ws, n, stream)
    return y, s_final, ckpt


def backward_checkpointed(cfg: dict, dy, ds_final, x, dt_raw, A, B, C, ckpt, every: int = 8, stream=None,
                          workspace=None):
    """``backward`` that replays the chunk states from ``forward_checkpointed``'s checkpoints (no s0); returns the
    same dict."""
    prob = problem(cfg)
    dev = x.device
    out = {"dx": torch.empty_like(x), "ddt_raw": torch.empty_like(dt_raw), "dA": torch.empty_like(A),
           "dB": torch.empty_like(B), "dC": torch.empty_like(C), "ds0": torch.empty_like(ds_final)}
    ws, n = workspace if workspace is not None else _workspace(prob, True, dev)
    ssd_backward_checkpointed(prob, dy, ds_final, x, dt_raw, A, B, C, every, ckpt, ckpt.numel() * 4, out["dx"],
                              out["ddt_raw"], out["dA"], out["dB"], out["dC"], out["ds0"], ws, n, stream)
    return out


# ------------------------------------------------------------- KDA (gated delta rule)
def kda_problem(cfg: dict) -> ssd_kda_problem:
    return ssd_kda_problem(cfg["batch"], cfg["seqlen"], cfg["nheads"], cfg["value_heads"], cfg["key_dim"],
                           cfg["value_dim"])


def ssd_kda_workspace_size(prob: ssd_kda_problem, backward: bool) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_kda_workspace_size(ctypes.byref(prob), int(bool(backward)), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_kda_workspace_size")
    return out.value


def ssd_kda_forward(prob, q, k, v, g, beta, s0, scale, o, s_final, ws, ws_bytes, stream=None) -> None:
    st = load().ssd_kda_forward(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(s0),
                                float(scale), _ptr(o), _ptr(s_final), _ptr(ws), int(ws_bytes), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_kda_forward")


def ssd_kda_backward(prob, dout, ds_final, q, k, v, g, beta, s0, scale, dq, dk, dv, dg, dbeta, ds0, ws, ws_bytes,
                     stream=None) -> None:
    st = load().ssd_kda_backward(ctypes.byref(prob), _ptr(dout), _ptr(ds_final), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(beta), _ptr(s0), float(scale), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
                                 _ptr(dbeta), _ptr(ds0), _ptr(ws), int(ws_bytes), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_kda_backward")


def _kda_workspace(prob, backward, device):
    n = ssd_kda_workspace_size(prob, backward)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device), n


def kda_forward(cfg: dict, q, k, v, g, beta, s0=None, scale=None, stream=None, workspace=None):
    """Allocate o, s_final and run ``ssd_kda_forward``; scale defaults to key_dim^-1/2."""
    prob = kda_problem(cfg)
    scale = cfg["key_dim"] ** -0.5 if scale is None else scale
    o = torch.empty_like(v)
    s_final = torch.empty((cfg["batch"], cfg["value_heads"], cfg["key_dim"], cfg["value_dim"]), dtype=torch.float32,
                          device=v.device)
    ws, n = workspace if workspace is not None else _kda_workspace(prob, False, v.device)
    ssd_kda_forward(prob, q, k, v, g, beta, s0, scale, o, s_final, ws, n, stream)
    return o, s_final


def kda_backward(cfg: dict, dout, ds_final, q, k, v, g, beta, s0=None, scale=None, stream=None, workspace=None):
    """Allocate the gradients and run ``ssd_kda_backward``; returns dq, dk, dv, dg, dbeta, ds0."""
    prob = kda_problem(cfg)
    scale = cfg["key_dim"] ** -0.5 if scale is None else scale
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v), "dg": torch.empty_like(g),
           "dbeta": torch.empty_like(beta), "ds0": torch.empty_like(ds_final)}
    ws, n = workspace if workspace is not None else _kda_workspace(prob, True, v.device)
    ssd_kda_backward(prob, dout, ds_final, q, k, v, g, beta, s0, scale, out["dq"], out["dk"], out["dv"], out["dg"],
                     out["dbeta"], out["ds0"], ws, n, stream)
    return out


# ------------------------------------------------------------- gated delta rule, one decay per head
# The conveniences below are called once a token: what they look up by a call's sizes is kept (a few hundred
# problem descriptions and sizes, by value), and the checks take the common case first.
_kept: dict = {}


def _keep(key, make):
    got = _kept.get(key)
    if got is None:
        if len(_kept) >= 512:
            _kept.clear()
        got = _kept[key] = make()
    return got


def _delta_key(cfg: dict, packed: bool, qs: int, ks: int, vs: int) -> tuple:
    return ("delta", cfg["dtype"], cfg.get("gate_dtype", "f32"), packed, cfg["batch"], cfg["seqlen"], cfg["nheads"],
            cfg["value_heads"], cfg["key_dim"], cfg["value_dim"], qs, ks, vs)


def _delta_struct(key: tuple) -> ssd_delta_problem:
    return ssd_delta_problem(DTYPES[key[1]], DTYPES[key[2]], int(key[3]), 0, *key[4:])


def delta_problem(cfg: dict, q=None, k=None, v=None, packed: bool = False) -> ssd_delta_problem:
    """An ``ssd_delta_problem`` from a config dict (``configs.DELTA_CONFIGS``); q, k, v (if given) set the strides from
    step to step and are checked against the sizes."""
    return _delta_struct(_delta_of(cfg, q, k, v, packed))


def _delta_of(cfg: dict, q, k, v, packed: bool) -> tuple:
    """The key of a call's problem, from its q, k, v."""
    lead = (1 if packed else cfg["batch"], cfg["seqlen"])
    h, hv, kd, vd = cfg["nheads"], cfg["value_heads"], cfg["key_dim"], cfg["value_dim"]
    dt = _TORCH_DTYPE[cfg["dtype"]]
    return _delta_key(cfg, packed, 0 if q is None else _step_stride("q", q, lead + (h, kd), dt),
                      0 if k is None else _step_stride("k", k, lead + (h, kd), dt),
                      0 if v is None else _step_stride("v", v, lead + (hv, vd), dt))


def _step_stride(name: str, t, shape: tuple, dtype) -> int:
    """Elements from a step to the next of a tensor [b, T, heads, dim] whose heads are dense and whose batches follow
    one another at T steps (0: dense); raises ValueError for any other tensor."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    got = tuple(t.shape)
    b, steps, heads, dim = shape
    if got != shape and not (b == 1 and got == shape[1:]):
        raise ValueError(f"{name}: shape {got}, expected {shape}")
    if t.is_contiguous():
        return 0
    sb, st, sh, sd = t.stride() if t.dim() == 4 else (0,) + tuple(t.stride())
    if steps == 1:  # one step a batch: the batches are the steps
        st = sb if b > 1 else heads * dim
    if (dim > 1 and sd != 1) or (heads > 1 and sh != dim) or (b > 1 and sb != steps * st) or st < heads * dim:
        raise ValueError(f"{name}: strides {tuple(t.stride())}: heads have to be dense and batches follow one another")
    return st


def _dense(name: str, t, shape: tuple, dtype) -> None:
    if t is None or (t.shape == shape and t.dtype == dtype and t.is_contiguous()):
        return
    if t.dtype != dtype or not t.is_contiguous() or not (shape[0] == 1 and tuple(t.shape) == shape[1:]):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} (contiguous: {t.is_contiguous()}), expected contiguous "
                         f"{dtype} {shape}")


def ssd_delta_workspace_size(prob: ssd_delta_problem, backward: bool, stashed: bool = False) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_delta_workspace_size(ctypes.byref(prob), int(bool(backward)), int(bool(stashed)), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_delta_workspace_size")
    return out.value


def ssd_delta_stash_size(prob: ssd_delta_problem) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_delta_stash_size(ctypes.byref(prob), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_delta_stash_size")
    return out.value


def ssd_delta_forward(prob, q, k, v, g, beta, s0, cu_seqlens, scale, o, s_final, stash, stash_bytes, ws, ws_bytes,
                      stream=None) -> None:
    st = (_lib or load()).ssd_delta_forward(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                            _ptr(s0), _ptr(cu_seqlens), scale, _ptr(o), _ptr(s_final), _ptr(stash),
                                            stash_bytes, _ptr(ws), ws_bytes, _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_delta_forward")


def ssd_delta_backward(prob, dout, ds_final, q, k, v, g, beta, s0, cu_seqlens, scale, dq, dk, dv, dg, dbeta, ds0, stash,
                       stash_bytes, ws, ws_bytes, stream=None) -> None:
    st = (_lib or load()).ssd_delta_backward(ctypes.byref(prob), _ptr(dout), _ptr(ds_final), _ptr(q), _ptr(k), _ptr(v),
                                             _ptr(g), _ptr(beta), _ptr(s0), _ptr(cu_seqlens), scale, _ptr(dq),
                                             _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(ds0), _ptr(stash),
                                             stash_bytes, _ptr(ws), ws_bytes, _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_delta_backward")


def ssd_delta_step(prob, q, k, v, g, beta, state, slots, num_slots, scale, o, stream=None) -> None:
    st = (_lib or load()).ssd_delta_step(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                         _ptr(state), _ptr(slots), num_slots, scale, _ptr(o), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_delta_step")


def _delta_check(key, g, beta, s0, cu_seqlens):
    _, _, gdt, packed, b, t, _, hv, kd, vd = key[:10]
    lead = (1 if packed else b, t)
    gt = _TORCH_DTYPE[gdt]
    _dense("g", g, lead + (hv,), gt)
    _dense("beta", beta, lead + (hv,), gt)
    if s0 is not None:
        _dense("s0", s0, (b, hv, kd, vd), torch.float32)
    if cu_seqlens is not None:
        _dense("cu_seqlens", cu_seqlens, (b + 1,), torch.int32)
    return lead


def _device(first, *others) -> int:
    """The index of the CUDA device that all tensors of a call are on (None is passed over).  It has to be the current
    one: the library launches there, whatever device a stream's handle or a pointer belongs to."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device}: one CUDA device expected")
    if dev < 0:
        raise ValueError(f"tensors on {first.device}: a CUDA device expected")
    if dev != torch.cuda.current_device():
        raise ValueError(f"tensors on {first.device}, but the current device (or that of the stream given) is "
                         f"cuda:{torch.cuda.current_device()}: make theirs current first")
    return dev


def _on(stream, device, *tensors):
    """The context of a call on a stream of the caller's (a torch stream or a ``cudaStream_t``): what the call allocates
    belongs to that stream, as a workspace that is freed on return has to.  The call's own tensors, which may belong to
    another, stay until a torch stream has come to their use; a handle's owner keeps them, since it may end before they do."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    else:
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
    return torch.cuda.stream(stream)


def _like(t):
    """An uninitialised dense tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def delta_stash(cfg: dict, device="cuda", packed: bool = False):
    """A buffer for what ``delta_forward`` keeps for ``delta_backward`` (uint8)."""
    key = _delta_key(cfg, packed, 0, 0, 0)
    n = _keep(key + ("stash",), lambda: ssd_delta_stash_size(_delta_struct(key)))
    return torch.empty(n, dtype=torch.uint8, device=device)


def _delta_workspace(key, backward, stashed, device):
    n = _keep(key + (backward, stashed),
              lambda: max(ssd_delta_workspace_size(_delta_struct(key), backward, stashed), 256))
    return torch.empty(n, dtype=torch.uint8, device=device), n


def delta_status(device="cuda"):
    """A tensor for the ``status`` of ``delta_forward`` and ``delta_backward``: the device status words of the calls that
    it is handed to end up in it (the largest; 0: every wait of their kernels ended in time).  ``check_status`` reads it."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def check_status(status) -> None:
    """Reads `status` on the current stream (made to come after the calls' stream by the caller, where that is another),
    waiting for it, and raises SSDError if a kernel's wait gave up: results of those calls are missing or wrong."""
    code = int(status)
    if code:
        raise SSDError(SSD_ERR_TIMEOUT, f"delta rule (device status word {code})")


def _join_status(status, ws) -> None:
    """The status word of a call, the first 4 bytes of its workspace, into the caller's tensor, on the call's stream."""
    torch.maximum(status, ws.view(torch.uint8)[:4].view(torch.int32).view(status.shape), out=status)


def delta_forward(cfg: dict, q, k, v, g, beta, s0=None, scale=None, cu_seqlens=None, stash=None, stream=None,
                  workspace=None, status=None):
    """Allocate o and s_final, run ``ssd_delta_forward``; returns (o, s_final).  With ``cu_seqlens`` (int32,
    [batch + 1]) the sequences are packed on one axis of seqlen steps (steps of no sequence are zero in o and in the
    gradients); ``stash`` (``delta_stash``) is filled for ``delta_backward``; scale defaults to key_dim^-1/2.  On
    ``stream`` (a torch stream, or a ``cudaStream_t`` whose owner keeps the tensors until it has used them), the outputs
    belong to it.  ``status`` (``delta_status``): where to leave the device status word, which is gone with the
    workspace otherwise."""
    if stream is not None:
        with _on(stream, v.device, q, k, v, g, beta, s0, cu_seqlens, stash, workspace and workspace[0], status):
            return delta_forward(cfg, q, k, v, g, beta, s0, scale, cu_seqlens, stash, None, workspace, status)
    key = _delta_of(cfg, q, k, v, cu_seqlens is not None)
    prob = _keep(key, lambda: _delta_struct(key))
    _delta_check(key, g, beta, s0, cu_seqlens)
    _dense("status", status, (1,), torch.int32)
    scale = cfg["key_dim"] ** -0.5 if scale is None else scale
    at = _device(v, q, k, g, beta, s0, cu_seqlens, stash, status, workspace and workspace[0])
    dev = v.device
    o = _like(v)
    s_final = torch.empty((key[4], key[7], key[8], key[9]), dtype=torch.float32, device=dev)
    ws, n = workspace if workspace is not None else _delta_workspace(key, False, stash is not None, dev)
    ssd_delta_forward(prob, q, k, v, g, beta, s0, cu_seqlens, scale, o, s_final, stash,
                      0 if stash is None else stash.numel(), ws, n, _stream(None, at))
    if status is not None:
        _join_status(status, ws)
    return o, s_final


def delta_backward(cfg: dict, dout, q, k, v, g, beta, ds_final=None, s0=None, scale=None, cu_seqlens=None, stash=None,
                   stream=None, workspace=None, status=None):
    """Allocate the gradients and run ``ssd_delta_backward``; returns dq, dk, dv, dg, dbeta and ds0 (None where s0 is
    None).  ``stash``: what ``delta_forward`` filled on the same inputs; without it the chunk states are made again.
    ``status``: as for ``delta_forward``."""
    if stream is not None:
        with _on(stream, v.device, dout, q, k, v, g, beta, ds_final, s0, cu_seqlens, stash, workspace and workspace[0],
                 status):
            return delta_backward(cfg, dout, q, k, v, g, beta, ds_final, s0, scale, cu_seqlens, stash, None, workspace,
                                  status)
    key = _delta_of(cfg, q, k, v, cu_seqlens is not None)
    prob = _keep(key, lambda: _delta_struct(key))
    lead = _delta_check(key, g, beta, s0, cu_seqlens)
    _dense("dout", dout, lead + (key[7], key[9]), v.dtype)
    if ds_final is not None:
        _dense("ds_final", ds_final, (key[4], key[7], key[8], key[9]), torch.float32)
    _dense("status", status, (1,), torch.int32)
    scale = cfg["key_dim"] ** -0.5 if scale is None else scale
    at = _device(v, q, k, g, beta, dout, ds_final, s0, cu_seqlens, stash, status, workspace and workspace[0])
    dev = v.device
    out = {"dq": _like(q), "dk": _like(k), "dv": _like(v), "dg": _like(g), "dbeta": _like(beta),
           "ds0": None if s0 is None else _like(s0)}
    ws, n = workspace if workspace is not None else _delta_workspace(key, True, stash is not None, dev)
    ssd_delta_backward(prob, dout, ds_final, q, k, v, g, beta, s0, cu_seqlens, scale, out["dq"], out["dk"], out["dv"],
                       out["dg"], out["dbeta"], out["ds0"], stash, 0 if stash is None else stash.numel(), ws, n,
                       _stream(None, at))
    if status is not None:
        _join_status(status, ws)
    return out


def delta_step(cfg: dict, q, k, v, g, beta, state, slots=None, scale=None, stream=None):
    """Allocate o and run ``ssd_delta_step``: seqlen steps of each sequence on its slot of ``state`` [slots, HV, K, V]
    (fp32), which is updated in place; returns o."""
    if stream is not None:
        with _on(stream, v.device, q, k, v, g, beta, state, slots):
            return delta_step(cfg, q, k, v, g, beta, state, slots, scale)
    key = _delta_of(cfg, q, k, v, False)
    prob = _keep(key, lambda: _delta_struct(key))
    _delta_check(key, g, beta, None, None)
    ns = state.shape[0]
    _dense("state", state, (ns, key[7], key[8], key[9]), torch.float32)
    _dense("slots", slots, (key[4],), torch.int32)
    scale = cfg["key_dim"] ** -0.5 if scale is None else scale
    at = _device(v, q, k, g, beta, state, slots)
    o = _like(v)
    ssd_delta_step(prob, q, k, v, g, beta, state, slots, ns, scale, o, _stream(None, at))
    return o


# ------------------------------------------------------------- layer norm
def _name(dtype) -> str:
    for k, v in _TORCH_DTYPE.items():
        if v == dtype:
            return k
    raise ValueError(f"{dtype}: float32 or bfloat16 expected")


def _norm_of(x, weight) -> tuple:
    """The key of a call's problem: (type, weight's type, rows, dim, stride)."""
    dim = x.shape[-1]
    stride = 0
    if not x.is_contiguous():
        if x.dim() != 2 or (dim > 1 and x.stride(1) != 1) or x.stride(0) < dim:
            raise ValueError(f"x: strides {tuple(x.stride())}: rows have to be dense, at one stride")
        stride = x.stride(0)
    return x.dtype, torch.float32 if weight is None else weight.dtype, x.numel() // max(dim, 1), dim, stride


def _norm_struct(key: tuple) -> ssd_norm_problem:
    return ssd_norm_problem(DTYPES[_name(key[0])], DTYPES[_name(key[1])], *key[2:])


def norm_problem(x, weight=None) -> ssd_norm_problem:
    """An ``ssd_norm_problem`` for x [.., D]: contiguous, or two-dimensional with a stride from row to row."""
    return _norm_struct(_norm_of(x, weight))


def ssd_norm_workspace_size(prob: ssd_norm_problem) -> int:
    out = ctypes.c_size_t(0)
    st = load().ssd_norm_workspace_size(ctypes.byref(prob), ctypes.byref(out))
    if st != SSD_OK:
        raise SSDError(st, "ssd_norm_workspace_size")
    return out.value


def ssd_norm_forward(prob, x, weight, bias, eps, y, mean, rstd, stream=None) -> None:
    st = (_lib or load()).ssd_norm_forward(ctypes.byref(prob), _ptr(x), _ptr(weight), _ptr(bias), eps, _ptr(y),
                                           _ptr(mean), _ptr(rstd), _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_norm_forward")


def ssd_norm_backward(prob, dy, x, mean, rstd, weight, dx, dw, db, ws, ws_bytes, stream=None) -> None:
    st = (_lib or load()).ssd_norm_backward(ctypes.byref(prob), _ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight),
                                            _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), ws_bytes, _stream(stream))
    if st != SSD_OK:
        raise SSDError(st, "ssd_norm_backward")


def norm_forward(x, weight=None, bias=None, eps: float = 1e-5, stream=None):
    """Layer norm of x [.., D]; weight and bias [D] (either may be None) of one type.  Returns y (contiguous), mean and
    rstd (fp32, one per row)."""
    if stream is not None:
        with _on(stream, x.device, x, weight, bias):
            return norm_forward(x, weight, bias, eps)
    key = _norm_of(x, weight if weight is not None else bias)
    prob = _keep(key, lambda: _norm_struct(key))
    if weight is not None:
        _dense("weight", weight, (key[3],), key[1])
    if bias is not None:
        _dense("bias", bias, (key[3],), key[1])
    at = _device(x, weight, bias)
    y = _like(x)
    dev = x.device
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    ssd_norm_forward(prob, x, weight, bias, eps, y, mean, rstd, _stream(None, at))
    return y, mean, rstd


def norm_backward(dy, x, mean, rstd, weight=None, stream=None, workspace=None):
    """The gradients of ``norm_forward``: dx (contiguous), and dw and db in the weight's type (fp32 without a
    weight)."""
    if stream is not None:
        with _on(stream, x.device, dy, x, mean, rstd, weight, workspace and workspace[0]):
            return norm_backward(dy, x, mean, rstd, weight, None, workspace)
    key = _norm_of(x, weight)
    prob = _keep(key, lambda: _norm_struct(key))
    if dy.dtype != x.dtype or dy.shape != x.shape or not dy.is_contiguous():
        raise ValueError(f"dy: {dy.dtype} {tuple(dy.shape)}, expected contiguous {x.dtype} {tuple(x.shape)}")
    if weight is not None:
        _dense("weight", weight, (key[3],), key[1])
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.numel() != key[2] or not t.is_contiguous():
            raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected contiguous float32, one per row")
    at = _device(x, dy, mean, rstd, weight, workspace and workspace[0])
    dx = _like(x)
    dev = x.device
    dw, db = torch.empty(key[3], dtype=key[1], device=dev), torch.empty(key[3], dtype=key[1], device=dev)
    if workspace is None:
        n = _keep(key + ("ws",), lambda: ssd_norm_workspace_size(prob))
        workspace = torch.empty(n, dtype=torch.uint8, device=dev), n
    ssd_norm_backward(prob, dy, x, mean, rstd, weight, dx, dw, db, workspace[0], workspace[1],
                      _stream(None, at))
    return {"dx": dx, "dw": dw, "db": db}
