"""Thin Python binding of the m3scan C ABI (include/m3scan.h).

Argument marshalling only: every step of the layer core runs in the CUDA
library.  PyTorch supplies device memory and the stream; outputs that the
caller does not pass are allocated here with ``torch.empty``.  If the
library cannot be loaded the calls raise -- there is no other path.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

from . import build as _build

M3_F32 = 0
M3_BF16 = 1

STATUS = {
    0: "M3_OK",
    1: "M3_ERR_NULL",
    2: "M3_ERR_DIMS",
    3: "M3_ERR_UNSUPPORTED",
    4: "M3_ERR_ALIGN",
    5: "M3_ERR_WORKSPACE",
    6: "M3_ERR_CUDA",
    7: "M3_ERR_TIMEOUT",
}

# bytes at the start of every workspace that hold the library's status block
STATUS_BYTES = 256

# every symbol include/m3scan.h declares
EXPORTS = ("m3scan_plan", "m3scan_fwd", "m3scan_bwd", "m3scan_fwd_state", "m3scan_bwd_state",
           "m3scan_bwd_scan", "m3scan_conv_bwd", "m3scan_decode", "m3scan_bwd_noalloc", "m3scan_status_string", "m3scan_last_cuda_error",
           "m3scan_version", "m3scan_get_status", "m3scan_device_status",
           "m3scan_selftest_wait_timeout", "m3scan_norm_plan", "m3scan_norm_fwd", "m3scan_norm_bwd",
           "m3scan_delta_plan", "m3scan_delta_fwd", "m3scan_delta_bwd", "m3scan_delta_decode",
           "m3scan_qkrot_plan", "m3scan_qkrot_fwd", "m3scan_qkrot_bwd",
           "m3scan_linattn_plan", "m3scan_linattn_fwd", "m3scan_linattn_bwd", "m3scan_linattn_decode")

# size of the library's own scratch array used by m3scan_bwd_noalloc
NOALLOC_SCRATCH_BYTES = 16 << 20


class M3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib_handle().m3scan_status_string(status).decode() if _LIB else STATUS.get(status)
        if status == 6 and _LIB:
            msg += f" ({_LIB.m3scan_last_cuda_error().decode()})"
        super().__init__(f"{where}: {msg}")


class M3Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seq_len", ctypes.c_int64),
                ("d_inner", ctypes.c_int64), ("d_state", ctypes.c_int64),
                ("d_conv", ctypes.c_int64), ("chunk", ctypes.c_int64),
                ("segments", ctypes.c_int64),
                ("accumulate_param_grads", ctypes.c_int32),
                ("threads_per_channel", ctypes.c_int32),
                ("bc_stride", ctypes.c_int64), ("dbc_stride", ctypes.c_int64),
                ("deterministic", ctypes.c_int32), ("reserved0", ctypes.c_int32)]


class M3Plan(ctypes.Structure):
    _fields_ = [("chunk", ctypes.c_int64), ("n_chunks", ctypes.c_int64),
                ("fwd_segments", ctypes.c_int64), ("bwd_segments", ctypes.c_int64),
                ("ckpt_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("fwd_launches", ctypes.c_int32), ("bwd_launches", ctypes.c_int32),
                ("fwd_threads_per_channel", ctypes.c_int32),
                ("bwd_threads_per_channel", ctypes.c_int32)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class M3FwdState(ctypes.Structure):
    """m3_fwd_state: carried state in and out of a forward window."""
    _fields_ = [("ssm_state", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("ssm_state_out", ctypes.c_void_p), ("conv_state_out", ctypes.c_void_p)]


class M3BwdState(ctypes.Structure):
    """m3_bwd_state: the conv state the forward used, the upstream gradients of
    the state outputs and the gradients of the state inputs."""
    _fields_ = [("conv_state", ctypes.c_void_p), ("d_ssm_state_out", ctypes.c_void_p),
                ("d_conv_state_out", ctypes.c_void_p), ("d_ssm_state", ctypes.c_void_p),
                ("d_conv_state", ctypes.c_void_p)]


class M3NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("eps", ctypes.c_float),
                ("accumulate_param_grads", ctypes.c_int32)]


class M3NormPlan(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64)]


class M3DeltaDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seq_len", "k_heads", "v_heads", "head_k", "head_v", "q_stride", "k_stride",
        "v_stride", "dq_stride", "dk_stride", "dv_stride")] + [
            ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int32)]


class M3DeltaPlan(ctypes.Structure):
    _fields_ = [("chunk", ctypes.c_int64), ("n_chunks", ctypes.c_int64),
                ("ckpt_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("fwd_workspace_bytes", ctypes.c_int64),
                ("fwd_launches", ctypes.c_int32), ("bwd_launches", ctypes.c_int32)]


class M3QkrotDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seq_len", "q_heads", "k_heads", "head_dim", "rot_dim", "q_stride", "k_stride",
        "q_out_stride", "k_out_stride", "dq_stride", "dk_stride", "dq_out_stride", "dk_out_stride",
        "position_stride")] + [("eps", ctypes.c_float), ("interleaved", ctypes.c_int32),
                               ("accumulate_param_grads", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class M3QkrotPlan(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64)]


class M3LinattnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seq_len", "k_heads", "v_heads", "head_k", "head_v", "q_stride", "k_stride",
        "v_stride", "dq_stride", "dk_stride", "dv_stride")] + [
            ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class M3LinattnPlan(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64), ("fwd_workspace_bytes", ctypes.c_int64),
                ("fwd_launches", ctypes.c_int32), ("bwd_launches", ctypes.c_int32)]


_LIB = None
_LOCK = threading.Lock()
_vp = ctypes.c_void_p
_fp = ctypes.c_void_p  # float* passed as an address


def library_path() -> str:
    return _build.LIB_PATH


def _lib_handle(build_if_missing: bool = True):
    global _LIB
    with _LOCK:
        if _LIB is None:
            path = _build.LIB_PATH
            if build_if_missing and not os.path.exists(path):
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libm3scan not built: {path} is missing")
            lib = ctypes.CDLL(path)
            lib.m3scan_plan.restype = ctypes.c_int
            lib.m3scan_plan.argtypes = [ctypes.POINTER(M3Dims), ctypes.c_int,
                                        ctypes.POINTER(M3Plan)]
            lib.m3scan_fwd.restype = ctypes.c_int
            lib.m3scan_fwd.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                       + [_fp] * 5 + [_vp, _vp, _fp, _vp, ctypes.c_size_t, _vp])
            lib.m3scan_bwd.restype = ctypes.c_int
            lib.m3scan_bwd.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                       + [_fp] * 5 + [_fp, _vp] + [_vp] * 4 + [_fp] * 2
                                       + [_fp] * 5 + [_vp, ctypes.c_size_t, _vp])
            lib.m3scan_fwd_state.restype = ctypes.c_int
            lib.m3scan_fwd_state.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                             + [_fp] * 5 + [_vp, _vp, _fp]
                                             + [ctypes.POINTER(M3FwdState)]
                                             + [_vp, ctypes.c_size_t, _vp])
            lib.m3scan_bwd_state.restype = ctypes.c_int
            lib.m3scan_bwd_state.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                             + [_fp] * 5 + [_fp, _vp] + [_vp] * 4 + [_fp] * 2
                                             + [_fp] * 5 + [ctypes.POINTER(M3BwdState)]
                                             + [_vp, ctypes.c_size_t, _vp])
            lib.m3scan_bwd_scan.restype = ctypes.c_int
            lib.m3scan_bwd_scan.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                            + [_fp] * 5 + [_fp, _vp] + [_vp] * 3 + [_fp] * 5
                                            + [ctypes.POINTER(M3BwdState)]
                                            + [_vp, ctypes.c_size_t, _vp])
            lib.m3scan_conv_bwd.restype = ctypes.c_int
            lib.m3scan_conv_bwd.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int, _vp, _fp, _fp,
                                             _vp, _vp, _vp, _fp, _fp,
                                             ctypes.POINTER(M3BwdState),
                                             _vp, ctypes.c_size_t, _vp])
            lib.m3scan_decode.restype = ctypes.c_int
            lib.m3scan_decode.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                          + [_fp] * 5 + [_fp, _vp, _vp, _vp, _vp])
            lib.m3scan_bwd_noalloc.restype = ctypes.c_int
            lib.m3scan_bwd_noalloc.argtypes = ([ctypes.POINTER(M3Dims), ctypes.c_int] + [_vp] * 5
                                               + [_fp] * 5 + [_fp, _vp] + [_vp] * 4
                                               + [_fp] * 2 + [_fp] * 5 + [_vp])
            lib.m3scan_status_string.restype = ctypes.c_char_p
            lib.m3scan_status_string.argtypes = [ctypes.c_int]
            lib.m3scan_last_cuda_error.restype = ctypes.c_char_p
            lib.m3scan_last_cuda_error.argtypes = []
            lib.m3scan_version.restype = ctypes.c_int32
            lib.m3scan_version.argtypes = []
            lib.m3scan_device_status.restype = ctypes.c_int
            lib.m3scan_device_status.argtypes = [ctypes.POINTER(ctypes.c_int32)]
            lib.m3scan_get_status.restype = ctypes.c_int
            lib.m3scan_get_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_int)]
            lib.m3scan_selftest_wait_timeout.restype = ctypes.c_int
            lib.m3scan_selftest_wait_timeout.argtypes = [_vp, _vp]
            pn, pd = ctypes.POINTER(M3NormDims), ctypes.POINTER(M3DeltaDims)
            pr, pl = ctypes.POINTER(M3QkrotDims), ctypes.POINTER(M3LinattnDims)
            ci, sz = ctypes.c_int, ctypes.c_size_t
            for name, args in (
                    ("m3scan_norm_plan", [pn, ci, ctypes.POINTER(M3NormPlan)]),
                    ("m3scan_norm_fwd", [pn, ci] + [_vp] * 9),
                    ("m3scan_norm_bwd", [pn, ci, _vp, _vp, ci] + [_vp] * 9 + [sz, _vp]),
                    ("m3scan_delta_plan", [pd, ci, ctypes.POINTER(M3DeltaPlan)]),
                    ("m3scan_delta_fwd", [pd, ci] + [_vp] * 10 + [sz, _vp]),
                    ("m3scan_delta_bwd", [pd, ci] + [_vp] * 15 + [sz, _vp]),
                    ("m3scan_delta_decode", [pd, ci] + [_vp] * 8),
                    ("m3scan_qkrot_plan", [pr, ci, ctypes.POINTER(M3QkrotPlan)]),
                    ("m3scan_qkrot_fwd", [pr, ci] + [_vp] * 9),
                    ("m3scan_qkrot_bwd", [pr, ci] + [_vp] * 13 + [sz, _vp]),
                    ("m3scan_linattn_plan", [pl, ci, ctypes.POINTER(M3LinattnPlan)]),
                    ("m3scan_linattn_fwd", [pl, ci] + [_vp] * 8 + [sz, _vp]),
                    ("m3scan_linattn_bwd", [pl, ci] + [_vp] * 12 + [sz, _vp]),
                    ("m3scan_linattn_decode", [pl, ci] + [_vp] * 7)):
                getattr(lib, name).restype = ctypes.c_int
                getattr(lib, name).argtypes = args
            _LIB = lib
    return _LIB


def load():
    """Load libm3scan (building it first if it is missing)."""
    return _lib_handle()


def make_dims(batch, seq_len, d_inner, d_state=16, d_conv=4, chunk=0, segments=0,
              accumulate_param_grads=False, bc_stride=0, dbc_stride=0,
              threads_per_channel=0, deterministic=False) -> M3Dims:
    return M3Dims(int(batch), int(seq_len), int(d_inner), int(d_state), int(d_conv),
                  int(chunk), int(segments), int(bool(accumulate_param_grads)),
                  int(threads_per_channel), int(bc_stride), int(dbc_stride),
                  int(bool(deterministic)), 0)


def m3scan_plan(dims: M3Dims, act: int) -> M3Plan:
    out = M3Plan()
    st = _lib_handle().m3scan_plan(ctypes.byref(dims), int(act), ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_plan")
    return out


def m3scan_status_string(status: int) -> str:
    return _lib_handle().m3scan_status_string(int(status)).decode()


def m3scan_version() -> int:
    return int(_lib_handle().m3scan_version())


def m3scan_selftest_wait_timeout(stream: int = 0, workspace=None) -> None:
    """Enqueue the diagnostic block whose tile wait never completes (it
    reports to the device word and, if given, to ``workspace``'s status
    block)."""
    ws = None if workspace is None else workspace.ptr
    st = _lib_handle().m3scan_selftest_wait_timeout(ws, ctypes.c_void_p(stream))
    if st != 0:
        raise M3Error(st, "m3scan_selftest_wait_timeout")


def m3scan_get_status(workspace, stream=None) -> int:
    """Status of the calls made with ``workspace`` (a ``Workspace``) since the
    last query, then cleared: 0 (M3_OK) or 7 (M3_ERR_TIMEOUT).  Waits for
    ``stream`` (default: the current torch stream)."""
    out = ctypes.c_int(0)
    st = _lib_handle().m3scan_get_status(workspace.ptr, _stream_handle(stream), ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_get_status")
    return int(out.value)


def m3scan_device_status() -> int:
    """Device status since the last query (0 = every kernel ran normally),
    then cleared; waits for the device's queued work."""
    out = ctypes.c_int32(0)
    st = _lib_handle().m3scan_device_status(ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_device_status")
    return int(out.value)


def raw_fwd(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D,
            gated, y_dbg, ckpt, workspace, workspace_bytes, stream) -> int:
    """Call m3scan_fwd with integer addresses; returns the status code."""
    return _lib_handle().m3scan_fwd(ctypes.byref(dims), int(act), x, delta_raw, z, Bm, Cm,
                                    conv_w, conv_b, dt_bias, a_log, D, gated, y_dbg, ckpt,
                                    workspace, int(workspace_bytes), stream)


def raw_bwd(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt,
            d_gated, d_x, d_delta_raw, dz, du_dbg, dB, dC, d_conv_w, d_conv_b, d_dt_bias,
            d_a_log, dD, workspace, workspace_bytes, stream) -> int:
    """Call m3scan_bwd with integer addresses; returns the status code."""
    return _lib_handle().m3scan_bwd(ctypes.byref(dims), int(act), x, delta_raw, z, Bm, Cm,
                                    conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated, d_x,
                                    d_delta_raw, dz, du_dbg, dB, dC, d_conv_w, d_conv_b,
                                    d_dt_bias, d_a_log, dD, workspace, int(workspace_bytes),
                                    stream)


def raw_fwd_state(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D,
                  gated, y_dbg, ckpt, state, workspace, workspace_bytes, stream) -> int:
    """Call m3scan_fwd_state (``state`` an M3FwdState or None); returns the
    status code."""
    sp = ctypes.byref(state) if state is not None else None
    return _lib_handle().m3scan_fwd_state(ctypes.byref(dims), int(act), x, delta_raw, z, Bm, Cm,
                                          conv_w, conv_b, dt_bias, a_log, D, gated, y_dbg, ckpt,
                                          sp, workspace, int(workspace_bytes), stream)


def raw_bwd_state(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt,
                  d_gated, d_x, d_delta_raw, dz, du_dbg, dB, dC, d_conv_w, d_conv_b, d_dt_bias,
                  d_a_log, dD, state, workspace, workspace_bytes, stream) -> int:
    """Call m3scan_bwd_state (``state`` an M3BwdState or None); returns the
    status code."""
    sp = ctypes.byref(state) if state is not None else None
    return _lib_handle().m3scan_bwd_state(ctypes.byref(dims), int(act), x, delta_raw, z, Bm, Cm,
                                          conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated, d_x,
                                          d_delta_raw, dz, du_dbg, dB, dC, d_conv_w, d_conv_b,
                                          d_dt_bias, d_a_log, dD, sp, workspace,
                                          int(workspace_bytes), stream)


def raw_bwd_scan(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt,
                 d_gated, du, d_delta_raw, dz, dB, dC, d_dt_bias, d_a_log, dD, state, workspace,
                 workspace_bytes, stream) -> int:
    """Call m3scan_bwd_scan (``state`` an M3BwdState or None); returns the
    status code."""
    sp = ctypes.byref(state) if state is not None else None
    return _lib_handle().m3scan_bwd_scan(ctypes.byref(dims), int(act), x, delta_raw, z, Bm, Cm,
                                         conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated, du,
                                         d_delta_raw, dz, dB, dC, d_dt_bias, d_a_log, dD, sp,
                                         workspace, int(workspace_bytes), stream)


def raw_conv_bwd(dims, act, x, conv_w, conv_b, du, du_extra, d_x, d_conv_w, d_conv_b, state,
                 workspace, workspace_bytes, stream) -> int:
    """Call m3scan_conv_bwd (``state`` an M3BwdState or None); returns the
    status code."""
    sp = ctypes.byref(state) if state is not None else None
    return _lib_handle().m3scan_conv_bwd(ctypes.byref(dims), int(act), x, conv_w, conv_b, du,
                                         du_extra, d_x, d_conv_w, d_conv_b, sp, workspace,
                                         int(workspace_bytes), stream)


def raw_decode(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D,
               ssm_state, conv_state, gated, y_dbg, stream) -> int:
    """Call m3scan_decode with integer addresses; returns the status code."""
    return _lib_handle().m3scan_decode(ctypes.byref(dims), int(act), x, delta_raw, z, Bm, Cm,
                                       conv_w, conv_b, dt_bias, a_log, D, ssm_state, conv_state,
                                       gated, y_dbg, stream)


def raw_bwd_noalloc(dims, act, x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D,
                    ckpt, d_gated, d_x, d_delta_raw, dz, du_dbg, dB, dC, d_conv_w, d_conv_b,
                    d_dt_bias, d_a_log, dD, stream) -> int:
    """Call m3scan_bwd_noalloc (no workspace; the library's fixed scratch
    array is used) with integer addresses; returns the status code.  For
    callers that cannot allocate device memory themselves."""
    return _lib_handle().m3scan_bwd_noalloc(ctypes.byref(dims), int(act), x, delta_raw, z, Bm,
                                            Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt,
                                            d_gated, d_x, d_delta_raw, dz, du_dbg, dB, dC,
                                            d_conv_w, d_conv_b, d_dt_bias, d_a_log, dD, stream)


# ---------------------------------------------------------------------------
# torch-tensor wrappers (allocation and pointer marshalling only)
# ---------------------------------------------------------------------------

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _act_code(t) -> int:
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return M3_BF16
    if t.dtype is torch.float32:
        return M3_F32
    raise TypeError(f"activation dtype must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype=None, device=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _stream_handle(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _placed(call):
    """A call runs with its first tensor's device current, and with ``stream=``
    with that stream current.  The library launches on the current device;
    and what a call allocates (results, scratch) is the memory of the stream it
    runs on: that of another stream may still be in use by what was enqueued
    there before."""
    first = call.__code__.co_varnames[0]

    @functools.wraps(call)
    def placed(*args, stream=None, **kw):
        t = args[0] if args else kw.get(first)
        index = -1 if t is None else t.get_device()
        cuda = (_TORCH or _torch()).cuda
        if stream is not None:
            if index >= 0 and stream.device.index != index:
                raise ValueError(f"{first} is on cuda:{index}, stream on {stream.device}")
            with cuda.stream(stream):
                return call(*args, stream=stream, **kw)
        if index >= 0 and index != cuda.current_device():
            with cuda.device(index):
                return call(*args, **kw)
        return call(*args, **kw)
    return placed


class Workspace:
    """A device workspace sized for a plan (reusable across calls).  Its
    status block (the first STATUS_BYTES) starts at zero, as the library
    requires."""

    def __init__(self, nbytes: int, device):
        torch = _torch()
        self.nbytes = max(int(nbytes), STATUS_BYTES)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.buf[:STATUS_BYTES].zero_()

    @property
    def ptr(self):
        return self.buf.data_ptr()


def plan_for(x, chunk=0, segments=0):
    Bsz, T, D = x.shape
    dims = make_dims(Bsz, T, D, chunk=chunk, segments=segments)
    return dims, m3scan_plan(dims, _act_code(x))


@_placed
def m3scan_fwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, *, chunk=0,
               segments=0, gated=None, y_dbg=None, want_y=False, ckpt=None, workspace=None,
               stream=None, threads_per_channel=0):
    """Forward of the layer core.  Returns (gated, ckpt, y_dbg or None)."""
    return _fwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, chunk, segments,
                gated, y_dbg, want_y, ckpt, workspace, stream, None, threads_per_channel)[:3]


@_placed
def m3scan_fwd_state(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, *,
                     ssm_state=None, conv_state=None, chunk=0, segments=0, gated=None,
                     y_dbg=None, want_y=False, ckpt=None, ssm_state_out=None,
                     conv_state_out=None, workspace=None, stream=None, threads_per_channel=0):
    """Forward of one window from a carried state (None = zero).  Returns
    (gated, ckpt, y_dbg or None, ssm_state_out [B,16,D] f32,
    conv_state_out [B,3,D] activation dtype)."""
    torch = _torch()
    Bsz, _, Dn = x.shape
    N, W = Bm.shape[-1], conv_w.shape[-1]
    if ssm_state_out is None:
        ssm_state_out = torch.empty((Bsz, N, Dn), dtype=torch.float32, device=x.device)
    if conv_state_out is None:
        conv_state_out = torch.empty((Bsz, W - 1, Dn), dtype=x.dtype, device=x.device)
    _check(ssm_state, "ssm_state", torch.float32, x.device)
    _check(conv_state, "conv_state", x.dtype, x.device)
    _check(ssm_state_out, "ssm_state_out", torch.float32, x.device)
    _check(conv_state_out, "conv_state_out", x.dtype, x.device)
    st = M3FwdState(_ptr(ssm_state), _ptr(conv_state), _ptr(ssm_state_out),
                    _ptr(conv_state_out))
    gated, ckpt, y_dbg = _fwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, chunk,
                              segments, gated, y_dbg, want_y, ckpt, workspace, stream, st,
                              threads_per_channel)[:3]
    return gated, ckpt, y_dbg, ssm_state_out, conv_state_out


def _fwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, chunk, segments, gated,
         y_dbg, want_y, ckpt, workspace, stream, state, tpc=0):
    torch = _torch()
    act = x.dtype
    dev = x.device
    for n, t in (("x", x), ("delta_raw", delta_raw), ("z", z), ("B", Bm), ("C", Cm)):
        _check(t, n, act, dev)
    for n, t in (("conv_w", conv_w), ("conv_b", conv_b), ("dt_bias", dt_bias),
                 ("a_log", a_log), ("D", D)):
        _check(t, n, torch.float32, dev)
    Bsz, T, Dn = x.shape
    dims = make_dims(Bsz, T, Dn, d_state=Bm.shape[-1], d_conv=conv_w.shape[-1], chunk=chunk,
                     segments=segments, threads_per_channel=tpc)
    code = _act_code(x)
    pl = m3scan_plan(dims, code)
    if gated is None:
        gated = torch.empty_like(x)
    if want_y and y_dbg is None:
        y_dbg = torch.empty_like(x)
    if ckpt is None:
        ckpt = torch.empty((Bsz, pl.n_chunks, Bm.shape[-1], Dn), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = Workspace(pl.workspace_bytes, dev)
    args = (dims, code, _ptr(x), _ptr(delta_raw), _ptr(z), _ptr(Bm), _ptr(Cm),
            _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), _ptr(a_log), _ptr(D),
            _ptr(gated), _ptr(y_dbg), _ptr(ckpt))
    tail = (workspace.ptr, workspace.nbytes, _stream_handle(stream))
    if state is None:
        st = raw_fwd(*args, *tail)
    else:
        st = raw_fwd_state(*args, state, *tail)
    if st != 0:
        raise M3Error(st, "m3scan_fwd" if state is None else "m3scan_fwd_state")
    return gated, ckpt, y_dbg


@_placed
def m3scan_bwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated, *,
               chunk=0, segments=0, want_du=False, accumulate_param_grads=False, out=None,
               workspace=None, stream=None, threads_per_channel=0, deterministic=False):
    """Backward of the layer core.  Returns a dict of gradients (tensors).
    ``deterministic``: dB, dC and the parameter gradients as fixed-order sums
    (identical bits on every call, a larger workspace) instead of float-atomic
    sums; the per-element gradients are the same bits either way."""
    return _bwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated,
                chunk, segments, want_du, accumulate_param_grads, out, workspace, stream, None,
                threads_per_channel, deterministic)


@_placed
def m3scan_bwd_state(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated,
                     *, conv_state=None, d_ssm_state_out=None, d_conv_state_out=None, chunk=0,
                     segments=0, want_du=False, accumulate_param_grads=False, out=None,
                     workspace=None, stream=None, threads_per_channel=0, deterministic=False):
    """Backward of one window made by ``m3scan_fwd_state``.  Returns the
    gradients of ``m3scan_bwd`` plus ``d_ssm_state`` [B,16,D] f32 and
    ``d_conv_state`` [B,3,D] (activation dtype)."""
    torch = _torch()
    Bsz, _, Dn = x.shape
    N, W = Bm.shape[-1], conv_w.shape[-1]
    o = dict(out or {})
    o.setdefault("d_ssm_state", torch.empty((Bsz, N, Dn), dtype=torch.float32, device=x.device))
    o.setdefault("d_conv_state", torch.empty((Bsz, W - 1, Dn), dtype=x.dtype, device=x.device))
    _check(conv_state, "conv_state", x.dtype, x.device)
    _check(d_ssm_state_out, "d_ssm_state_out", torch.float32, x.device)
    _check(d_conv_state_out, "d_conv_state_out", x.dtype, x.device)
    _check(o["d_ssm_state"], "d_ssm_state", torch.float32, x.device)
    _check(o["d_conv_state"], "d_conv_state", x.dtype, x.device)
    st = M3BwdState(_ptr(conv_state), _ptr(d_ssm_state_out), _ptr(d_conv_state_out),
                    _ptr(o["d_ssm_state"]), _ptr(o["d_conv_state"]))
    return _bwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated,
                chunk, segments, want_du, accumulate_param_grads, o, workspace, stream, st,
                threads_per_channel, deterministic)


def _bwd(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt, d_gated, chunk,
         segments, want_du, accumulate_param_grads, out, workspace, stream, state, tpc=0,
         det=False):
    torch = _torch()
    act = x.dtype
    dev = x.device
    for n, t in (("x", x), ("delta_raw", delta_raw), ("z", z), ("B", Bm), ("C", Cm),
                 ("d_gated", d_gated)):
        _check(t, n, act, dev)
    for n, t in (("conv_w", conv_w), ("conv_b", conv_b), ("dt_bias", dt_bias),
                 ("a_log", a_log), ("D", D), ("ckpt", ckpt)):
        _check(t, n, torch.float32, dev)
    Bsz, T, Dn = x.shape
    N = Bm.shape[-1]
    W = conv_w.shape[-1]
    dims = make_dims(Bsz, T, Dn, d_state=N, d_conv=W, chunk=chunk, segments=segments,
                     accumulate_param_grads=accumulate_param_grads, threads_per_channel=tpc,
                     deterministic=det)
    code = _act_code(x)
    pl = m3scan_plan(dims, code)
    o = dict(out or {})
    o.setdefault("d_x", torch.empty_like(x))
    o.setdefault("d_delta_raw", torch.empty_like(x))
    o.setdefault("dz", torch.empty_like(x))
    if want_du:
        o.setdefault("du", torch.empty_like(x))
    f32 = dict(dtype=torch.float32, device=dev)
    o.setdefault("dB", torch.empty((Bsz, T, N), **f32))
    o.setdefault("dC", torch.empty((Bsz, T, N), **f32))
    o.setdefault("d_conv_w", torch.zeros((Dn, W), **f32))
    o.setdefault("d_conv_b", torch.zeros((Dn,), **f32))
    o.setdefault("d_dt_bias", torch.zeros((Dn,), **f32))
    o.setdefault("d_a_log", torch.zeros((Dn, N), **f32))
    o.setdefault("dD", torch.zeros((Dn,), **f32))
    for k, v in o.items():
        _check(v, k, None, dev)
    if workspace is None:
        workspace = Workspace(pl.workspace_bytes, dev)
    args = (dims, code, _ptr(x), _ptr(delta_raw), _ptr(z), _ptr(Bm), _ptr(Cm),
            _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), _ptr(a_log), _ptr(D), _ptr(ckpt),
            _ptr(d_gated), _ptr(o["d_x"]), _ptr(o["d_delta_raw"]), _ptr(o["dz"]),
            _ptr(o.get("du")), _ptr(o["dB"]), _ptr(o["dC"]), _ptr(o["d_conv_w"]),
            _ptr(o["d_conv_b"]), _ptr(o["d_dt_bias"]), _ptr(o["d_a_log"]), _ptr(o["dD"]))
    tail = (workspace.ptr, workspace.nbytes, _stream_handle(stream))
    if state is None:
        st = raw_bwd(*args, *tail)
    else:
        st = raw_bwd_state(*args, state, *tail)
    if st != 0:
        raise M3Error(st, "m3scan_bwd" if state is None else "m3scan_bwd_state")
    return o


@_placed
def m3scan_decode(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ssm_state,
                  conv_state, *, gated=None, y_dbg=None, want_y=False, stream=None):
    """Forward of a short window (x [B, T, D], typically T = 1) from the
    carried state, updating ``ssm_state`` [B, N, D] (f32) and ``conv_state``
    [B, 3, D] (activation dtype) in place.  Returns (gated, y_dbg or None)."""
    torch = _torch()
    act = x.dtype
    dev = x.device
    for n, t in (("x", x), ("delta_raw", delta_raw), ("z", z), ("B", Bm), ("C", Cm),
                 ("conv_state", conv_state)):
        _check(t, n, act, dev)
    for n, t in (("conv_w", conv_w), ("conv_b", conv_b), ("dt_bias", dt_bias),
                 ("a_log", a_log), ("D", D), ("ssm_state", ssm_state)):
        _check(t, n, torch.float32, dev)
    Bsz, T, Dn = x.shape
    dims = make_dims(Bsz, T, Dn, d_state=Bm.shape[-1], d_conv=conv_w.shape[-1])
    if gated is None:
        gated = torch.empty_like(x)
    if want_y and y_dbg is None:
        y_dbg = torch.empty_like(x)
    st = raw_decode(dims, _act_code(x), _ptr(x), _ptr(delta_raw), _ptr(z), _ptr(Bm), _ptr(Cm),
                    _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), _ptr(a_log), _ptr(D),
                    _ptr(ssm_state), _ptr(conv_state), _ptr(gated), _ptr(y_dbg),
                    _stream_handle(stream))
    if st != 0:
        raise M3Error(st, "m3scan_decode")
    return gated, y_dbg


@_placed
def m3scan_bwd_two_phase(x, delta_raw, z, Bm, Cm, conv_w, conv_b, dt_bias, a_log, D, ckpt,
                         d_gated, du_extra_fn=None, *, conv_state=None, d_ssm_state_out=None,
                         d_conv_state_out=None, chunk=0, segments=0, bc_stride=0, dbc_stride=0,
                         dB=None, dC=None, accumulate_param_grads=False, stream=None,
                         threads_per_channel=0, deterministic=False):
    """The two-phase backward: m3scan_bwd_scan, then ``du_extra_fn(grads)``
    (the caller's x_proj/dt_proj GEMMs, given the scan's gradients; may
    return None), then m3scan_conv_bwd.  ``Bm``/``Cm`` may be column views
    of one x_proj output (``bc_stride`` its row length), ``dB``/``dC``
    column views of its gradient (``dbc_stride``).  Returns the gradient
    dict (with ``du`` and, when states are involved, ``d_ssm_state`` and
    ``d_conv_state``)."""
    torch = _torch()
    act = x.dtype
    dev = x.device
    Bsz, T, Dn = x.shape
    N, W = Bm.shape[-1], conv_w.shape[-1]
    dims = make_dims(Bsz, T, Dn, d_state=N, d_conv=W, chunk=chunk, segments=segments,
                     accumulate_param_grads=accumulate_param_grads, bc_stride=bc_stride,
                     dbc_stride=dbc_stride, threads_per_channel=threads_per_channel,
                     deterministic=deterministic)
    code = _act_code(x)
    pl = m3scan_plan(dims, code)
    ws = Workspace(pl.workspace_bytes, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    o = {"du": torch.empty_like(x), "d_delta_raw": torch.empty_like(x), "dz": torch.empty_like(x),
         "dB": dB if dB is not None else torch.empty((Bsz, T, N), **f32),
         "dC": dC if dC is not None else torch.empty((Bsz, T, N), **f32),
         "d_dt_bias": torch.zeros((Dn,), **f32), "d_a_log": torch.zeros((Dn, N), **f32),
         "dD": torch.zeros((Dn,), **f32), "d_x": torch.empty_like(x),
         "d_conv_w": torch.zeros((Dn, W), **f32), "d_conv_b": torch.zeros((Dn,), **f32),
         "d_ssm_state": torch.empty((Bsz, N, Dn), **f32),
         "d_conv_state": torch.empty((Bsz, W - 1, Dn), dtype=act, device=dev)}
    st = M3BwdState(_ptr(conv_state), _ptr(d_ssm_state_out), _ptr(d_conv_state_out),
                    _ptr(o["d_ssm_state"]), _ptr(o["d_conv_state"]))
    h = _stream_handle(stream)
    r = raw_bwd_scan(dims, code, _ptr(x), _ptr(delta_raw), _ptr(z), _ptr(Bm), _ptr(Cm),
                     _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), _ptr(a_log), _ptr(D), _ptr(ckpt),
                     _ptr(d_gated), _ptr(o["du"]), _ptr(o["d_delta_raw"]), _ptr(o["dz"]),
                     o["dB"].data_ptr(), o["dC"].data_ptr(), _ptr(o["d_dt_bias"]),
                     _ptr(o["d_a_log"]), _ptr(o["dD"]), st, ws.ptr, ws.nbytes, h)
    if r != 0:
        raise M3Error(r, "m3scan_bwd_scan")
    du_extra = du_extra_fn(o) if du_extra_fn is not None else None
    if du_extra is not None:
        _check(du_extra, "du_extra", act, dev)
    r = raw_conv_bwd(dims, code, _ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(o["du"]),
                     _ptr(du_extra), _ptr(o["d_x"]), _ptr(o["d_conv_w"]), _ptr(o["d_conv_b"]),
                     st, ws.ptr, ws.nbytes, h)
    if r != 0:
        raise M3Error(r, "m3scan_conv_bwd")
    return o


# ---------------------------------------------------------------------------
# block operators: layer norm and the gated delta rule
# ---------------------------------------------------------------------------
# Single tokens and small rows take a few microseconds on the GPU, so these
# wrappers keep the host's share small: one pass of cheap checks per tensor
# (the slow ones only name what is wrong), and the plan of a set of sizes is
# made once.

def m3scan_norm_plan(dims: M3NormDims, act: int) -> M3NormPlan:
    out = M3NormPlan()
    st = _lib_handle().m3scan_norm_plan(ctypes.byref(dims), int(act), ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_norm_plan")
    return out


def m3scan_delta_plan(dims: M3DeltaDims, act: int) -> M3DeltaPlan:
    out = M3DeltaPlan()
    st = _lib_handle().m3scan_delta_plan(ctypes.byref(dims), int(act), ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_delta_plan")
    return out


def _shape(t, name, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need(t, name, dtype, index, shape):
    """``t`` (or None), which must be a dense tensor of that dtype and shape
    on CUDA device ``index``."""
    if t is None or (t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous()):
        return t
    _shape(t, name, shape)
    _check(t, name, dtype, _torch().device("cuda", index))
    return t


def _scratch(workspace, nbytes, torch, dev):
    """(address, bytes) of the caller's workspace or of a new one, the current
    stream's (whose status block nobody can query, so it need not start at
    zero), and what must stay alive until the call is enqueued."""
    if workspace is not None:
        return workspace.ptr, workspace.nbytes, workspace
    if nbytes == 0:
        return None, 0, None
    buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return buf.data_ptr(), nbytes, buf


@functools.lru_cache(maxsize=1024)
def _norm_sizes(rows, dim, eps, accumulate, code):
    dims = M3NormDims(rows, dim, eps, accumulate)
    return ctypes.byref(dims), m3scan_norm_plan(dims, code).workspace_bytes


@_placed
def m3scan_norm_fwd(x, weight, bias=None, *, residual=None, eps=1e-5, y=None, residual_out=None,
                    mean=None, rstd=None, want_stats=True, stream=None):
    """Layer norm over the last dimension of ``x`` [..., dim], of x + residual
    when the f32 ``residual`` stream is given.  Returns (y, residual_out,
    mean, rstd): ``residual_out`` (f32) is x + residual, None without a
    residual unless a tensor for it is passed; ``mean`` and ``rstd`` (f32
    [...]) are None when ``want_stats`` is False."""
    torch = _TORCH or _torch()
    code = _act_code(x)
    dev, shape, f32, index = x.device, x.shape, torch.float32, x.get_device()
    if index < 0 or not x.is_contiguous():
        _check(x, "x")
    dim, rshape = shape[-1], shape[:-1]
    _need(weight, "weight", f32, index, (dim,))
    _need(bias, "bias", f32, index, (dim,))
    _need(residual, "residual", f32, index, shape)
    y = torch.empty_like(x) if y is None else _need(y, "y", x.dtype, index, shape)
    if residual_out is not None:
        _need(residual_out, "residual_out", f32, index, shape)
    elif residual is not None:
        residual_out = torch.empty_like(residual)
    if mean is not None:
        _need(mean, "mean", f32, index, rshape)
    elif want_stats:
        mean = torch.empty(rshape, dtype=f32, device=dev)
    if rstd is not None:
        _need(rstd, "rstd", f32, index, rshape)
    elif want_stats:
        rstd = torch.empty(rshape, dtype=f32, device=dev)
    dims, _ = _norm_sizes(x.numel() // dim if dim else 0, dim, float(eps), 0, code)
    st = _LIB.m3scan_norm_fwd(dims, code, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias), y.data_ptr(),
                              _ptr(residual_out), _ptr(mean), _ptr(rstd), _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_norm_fwd")
    return y, residual_out, mean, rstd


@_placed
def m3scan_norm_bwd(dy, normed, weight, mean, rstd, *, d_residual_out=None, want_bias=True,
                    accumulate_param_grads=False, out=None, workspace=None, stream=None):
    """Backward of ``m3scan_norm_fwd``.  ``normed`` is its ``residual_out``
    (f32), or x when it had no residual; ``d_residual_out`` (f32) is the
    gradient reaching the residual stream past the norm.  Returns a dict:
    ``dx`` (dtype of dy), ``d_residual`` (f32; None without
    ``d_residual_out`` unless passed in ``out``), ``d_weight``, ``d_bias``."""
    torch = _torch()
    code, ncode = _act_code(dy), _act_code(normed)
    dev, shape, f32, index = dy.device, dy.shape, torch.float32, dy.get_device()
    if index < 0 or not dy.is_contiguous():
        _check(dy, "dy")
    dim, rshape = shape[-1], shape[:-1]
    o = dict(out) if out else {}
    dx, d_res, d_w, d_b = o.get("dx"), o.get("d_residual"), o.get("d_weight"), o.get("d_bias")
    new = torch.zeros if accumulate_param_grads else torch.empty
    _need(normed, "normed", normed.dtype, index, shape)
    _need(weight, "weight", f32, index, (dim,))
    _need(mean, "mean", f32, index, rshape)
    _need(rstd, "rstd", f32, index, rshape)
    _need(d_residual_out, "d_residual_out", f32, index, shape)
    dx = torch.empty_like(dy) if dx is None else _need(dx, "dx", dy.dtype, index, shape)
    if d_res is not None:
        _need(d_res, "d_residual", f32, index, shape)
    elif d_residual_out is not None:
        d_res = torch.empty_like(d_residual_out)
    d_w = new(dim, dtype=f32, device=dev) if d_w is None else _need(d_w, "d_weight", f32, index, (dim,))
    if d_b is not None:
        _need(d_b, "d_bias", f32, index, (dim,))
    elif want_bias:
        d_b = new(dim, dtype=f32, device=dev)
    dims, nbytes = _norm_sizes(dy.numel() // dim if dim else 0, dim, 0.0, int(bool(accumulate_param_grads)), code)
    ws, nbytes, _keep = _scratch(workspace, nbytes, torch, dev)
    st = _LIB.m3scan_norm_bwd(dims, code, dy.data_ptr(), normed.data_ptr(), ncode, weight.data_ptr(), mean.data_ptr(),
                              rstd.data_ptr(), _ptr(d_residual_out), dx.data_ptr(), _ptr(d_res), d_w.data_ptr(),
                              _ptr(d_b), ws, nbytes, _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_norm_bwd")
    o.update(dx=dx, d_residual=d_res, d_weight=d_w, d_bias=d_b)
    return o


def _stream_of(stream, index):
    if stream is not None:
        return stream.cuda_stream
    try:
        return _TORCH._C._cuda_getCurrentRawStream(index)  # 20 times cheaper than the Stream object
    except AttributeError:
        return _TORCH.cuda.current_stream(index).cuda_stream


def _token_stride(t, name, dtype, index, shape):
    """Elements between tokens of a [B, T, H, D] tensor whose heads are dense
    and whose batch rows follow each other at that stride (a column view of a
    projection's output); 0 = dense."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _shape(t, name, shape)
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.is_contiguous():
        return 0
    B, T, H, D = shape
    sb, stk, sh, sd = t.stride()
    if T <= 1:
        stk = sb if B > 1 else H * D
    if stk < H * D:  # a broadcast view (0 would be taken as dense), or tokens that overlap
        raise ValueError(f"{name}: tokens must be at least {H * D} elements apart, got strides {t.stride()}")
    if (D > 1 and sd != 1) or (H > 1 and sh != D) or (B > 1 and T > 0 and sb != T * stk):
        raise ValueError(f"{name}: heads must be dense and batch rows T token strides apart, got strides {t.stride()}")
    return stk


@functools.lru_cache(maxsize=1024)
def _delta_sizes(code, kshape, vshape, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, scale, qk_l2norm):
    """(dims, state shape, checkpoint floats, (forward, any) workspace bytes)
    for those shapes."""
    if len(kshape) != 4 or len(vshape) != 4 or tuple(kshape[:2]) != tuple(vshape[:2]):
        raise ValueError(f"k and v must be [batch, seq_len, heads, head size], got {tuple(kshape)}, {tuple(vshape)}")
    B, T, Hv, dv = vshape
    Hk, dk = kshape[2:]
    dims = M3DeltaDims(B, T, Hk, Hv, dk, dv, q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride, float(scale),
                       int(bool(qk_l2norm)))
    pl = m3scan_delta_plan(dims, code)
    return ctypes.byref(dims), (B, Hv, dk, dv), pl.ckpt_bytes // 4, (pl.fwd_workspace_bytes, pl.workspace_bytes)


def _delta_inputs(q, k, v, g, beta):
    """Checks the inputs; returns (dtype code, device index, k's and v's
    shapes, token strides of q, k, v)."""
    dt, index = v.dtype, v.get_device()
    code = _act_code(v)
    kshape, vshape, gshape = k.shape, v.shape, v.shape[:3]
    if index < 0:
        _check(v, "v")
    _need(g, "g", dt, index, gshape)
    _need(beta, "beta", dt, index, gshape)
    if (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and q.dtype is dt and k.dtype is dt
            and q.shape == kshape and q.get_device() == index and k.get_device() == index):
        return code, index, kshape, vshape, 0, 0, 0
    if len(kshape) != 4 or len(vshape) != 4:
        raise ValueError(f"k and v must be [batch, seq_len, heads, head size], got {tuple(kshape)}, {tuple(vshape)}")
    kwant = (*vshape[:2], *kshape[2:])
    return (code, index, kshape, vshape, _token_stride(q, "q", dt, index, kwant), _token_stride(k, "k", dt, index, kwant),
            _token_stride(v, "v", dt, index, vshape))


@_placed
def m3scan_delta_fwd(q, k, v, g, beta, *, state=None, scale=0.0, qk_l2norm=False, want_state=True,
                     want_ckpt=False, o=None, state_out=None, ckpt=None, workspace=None, stream=None):
    """Gated delta rule over a sequence.  q, k [B, T, Hk, dk], v [B, T, Hv,
    dv] (column views of a projection's output are fine), g (log decay) and
    beta [B, T, Hv], all bf16 or f32; ``state`` [B, Hv, dk, dv] f32 or None
    (zero).  Returns (o, state_out or None, ckpt or None); the backward needs
    ``want_ckpt=True``."""
    torch = _torch()
    dev, f32 = v.device, torch.float32
    code, index, kshape, vshape, sq, sk, sv = _delta_inputs(q, k, v, g, beta)
    dims, sshape, n_ckpt, nbytes = _delta_sizes(code, kshape, vshape, sq, sk, sv, 0, 0, 0, scale, qk_l2norm)
    _need(state, "state", f32, index, sshape)
    o = torch.empty(vshape, dtype=v.dtype, device=dev) if o is None else _need(o, "o", v.dtype, index, vshape)
    if state_out is not None:
        _need(state_out, "state_out", f32, index, sshape)
    elif want_state:
        state_out = torch.empty(sshape, dtype=f32, device=dev)
    if ckpt is not None:
        _need(ckpt, "ckpt", f32, index, (n_ckpt,))
    elif want_ckpt:
        ckpt = torch.empty(n_ckpt, dtype=f32, device=dev)
    ws, nbytes, _keep = _scratch(workspace, nbytes[0], torch, dev)
    st = _LIB.m3scan_delta_fwd(dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                               _ptr(state), o.data_ptr(), _ptr(state_out), _ptr(ckpt), ws, nbytes,
                               _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_delta_fwd")
    return o, state_out, ckpt


@_placed
def m3scan_delta_bwd(q, k, v, g, beta, ckpt, d_o, *, d_state_out=None, want_d_state=False, scale=0.0,
                     qk_l2norm=False, out=None, workspace=None, stream=None):
    """Backward of ``m3scan_delta_fwd`` (same q, k, v, g, beta, scale and
    qk_l2norm, its ``ckpt``).  Returns a dict: dq, dk, dv, dg, dbeta
    (activation dtype) and d_state (f32, None unless wanted).  dq, dk and dv
    in ``out`` may be column views of a projection's gradient."""
    torch = _torch()
    dev, dt, f32 = v.device, v.dtype, torch.float32
    code, index, kshape, vshape, sq, sk, sv = _delta_inputs(q, k, v, g, beta)
    r = dict(out) if out else {}
    for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
        if r.get(n) is None:
            r[n] = torch.empty(t.shape, dtype=dt, device=dev)
    _need(r["dg"], "dg", dt, index, g.shape)
    _need(r["dbeta"], "dbeta", dt, index, g.shape)
    strides = [_token_stride(r[n], n, dt, index, t.shape) for n, t in (("dq", q), ("dk", k), ("dv", v))]
    dims, sshape, n_ckpt, nbytes = _delta_sizes(code, kshape, vshape, sq, sk, sv, *strides, scale, qk_l2norm)
    if r.get("d_state") is None:
        r["d_state"] = torch.empty(sshape, dtype=f32, device=dev) if want_d_state else None
    _need(d_state_out, "d_state_out", f32, index, sshape)
    _need(r["d_state"], "d_state", f32, index, sshape)
    _need(d_o, "d_o", dt, index, v.shape)
    _need(ckpt, "ckpt", f32, index, (n_ckpt,))
    ws, nbytes, _keep = _scratch(workspace, nbytes[1], torch, dev)
    st = _LIB.m3scan_delta_bwd(dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                               ckpt.data_ptr(), d_o.data_ptr(), _ptr(d_state_out), r["dq"].data_ptr(),
                               r["dk"].data_ptr(), r["dv"].data_ptr(), r["dg"].data_ptr(), r["dbeta"].data_ptr(),
                               _ptr(r["d_state"]), ws, nbytes, _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_delta_bwd")
    return r


@_placed
def m3scan_delta_decode(q, k, v, g, beta, state, *, scale=0.0, qk_l2norm=False, o=None, stream=None):
    """A short window (typically one token: T = 1) from the carried ``state``
    [B, Hv, dk, dv] (f32), which is updated in place.  Returns o."""
    torch = _torch()
    code, index, kshape, vshape, sq, sk, sv = _delta_inputs(q, k, v, g, beta)
    dims, sshape, _, _ = _delta_sizes(code, kshape, vshape, sq, sk, sv, 0, 0, 0, scale, qk_l2norm)
    o = torch.empty(vshape, dtype=v.dtype, device=v.device) if o is None else _need(o, "o", v.dtype, index, vshape)
    _need(state, "state", torch.float32, index, sshape)
    st = _LIB.m3scan_delta_decode(dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                  state.data_ptr(), o.data_ptr(), _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_delta_decode")
    return o


# ---------------------------------------------------------------------------
# norm and rotation of queries and keys
# ---------------------------------------------------------------------------

def m3scan_qkrot_plan(dims: M3QkrotDims, act: int) -> M3QkrotPlan:
    out = M3QkrotPlan()
    st = _lib_handle().m3scan_qkrot_plan(ctypes.byref(dims), int(act), ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_qkrot_plan")
    return out


@functools.lru_cache(maxsize=1024)
def _qkrot_sizes(code, qshape, kshape, rot, strides, position_stride, eps, interleaved, accumulate):
    if len(qshape) != 4 or len(kshape) != 4 or qshape[:2] != kshape[:2] or qshape[3] != kshape[3]:
        raise ValueError(f"q and k must be [batch, seq_len, heads, head size], got {tuple(qshape)}, {tuple(kshape)}")
    B, T, Hq, D = qshape
    dims = M3QkrotDims(B, T, Hq, kshape[2], D, rot, *strides, position_stride, float(eps), int(bool(interleaved)),
                       int(bool(accumulate)), 0)
    return ctypes.byref(dims), m3scan_qkrot_plan(dims, code).workspace_bytes


def _qkrot_positions(positions, B, T, index, torch):
    """(address, elements between batch rows) of int64 positions [B, T] or [T]."""
    if positions is None:
        return None, 0
    if positions.dtype is not torch.int64:
        raise TypeError(f"positions must be {torch.int64}, got {positions.dtype}")
    if positions.get_device() != index:
        raise ValueError(f"positions is on {positions.device}, expected cuda:{index}")
    shape = positions.shape
    if shape == (B, T) and positions.is_contiguous():
        return positions.data_ptr(), T if B > 1 else 0
    if shape == (T,):
        batch = 0
    elif shape == (B, T):
        batch = positions.stride(0) if B > 1 else 0
        if B > 1 and 0 < batch < T or batch < 0:
            raise ValueError(f"positions: batch rows overlap, strides {positions.stride()}")
    else:
        raise ValueError(f"positions must have shape {(B, T)} or {(T,)}, got {tuple(shape)}")
    if T > 1 and positions.stride(-1) != 1:
        raise ValueError(f"positions must be dense in time, got strides {positions.stride()}")
    return positions.data_ptr(), batch


def _tokens_of(t, name, dtype, index, shape):
    """``_token_stride``, at once for the dense tensors that most are."""
    if t.is_contiguous() and t.dtype is dtype and t.shape == shape and t.get_device() == index:
        return 0
    return _token_stride(t, name, dtype, index, shape)


def _qkrot_inputs(q, k, q_weight, k_weight, positions, inv_freq, torch):
    """Checks the inputs; returns (dtype code, device index, q's and k's
    shapes, token strides of q and k, address and batch stride of the
    positions, rotated size)."""
    dt, index, qshape, kshape = q.dtype, q.get_device(), q.shape, k.shape
    code = _act_code(q)
    if index < 0:
        _check(q, "q")
    if len(qshape) != 4 or len(kshape) != 4:
        raise ValueError(f"q and k must be [batch, seq_len, heads, head size], got {tuple(qshape)}, {tuple(kshape)}")
    B, T, _, D = qshape
    sq = _tokens_of(q, "q", dt, index, qshape)
    sk = _tokens_of(k, "k", dt, index, (B, T, kshape[2], D))
    f32 = torch.float32
    _need(q_weight, "q_weight", f32, index, (D,))
    _need(k_weight, "k_weight", f32, index, (D,))
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _need(inv_freq, "inv_freq", f32, index, (rot // 2,))
        if rot and positions is None:
            raise ValueError("positions are needed where inv_freq is given")
    pos, pos_stride = _qkrot_positions(positions, B, T, index, torch)
    return code, index, qshape, kshape, sq, sk, pos, pos_stride, rot


@_placed
def m3scan_qkrot_fwd(q, k, q_weight, k_weight, positions, inv_freq, *, eps=1e-6, interleaved=False,
                     q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every head of q [B, T, Hq, D] and k [B, T, Hk,
    D] (column views of a projection's output are fine) with weights [D] (f32;
    None = ones), and their rotation by ``positions`` (int64 [B, T] or [T]) and
    ``inv_freq`` (f32 [R], 2 R <= D; None = no rotation).  Pairs are (i, i + R),
    or neighbours with ``interleaved``.  Returns (q_out, k_out), which may be q
    and k themselves."""
    torch = _TORCH or _torch()
    code, index, qshape, kshape, sq, sk, pos, pos_stride, rot = _qkrot_inputs(q, k, q_weight, k_weight, positions, inv_freq, torch)
    dt, sqo, sko = q.dtype, 0, 0
    if q_out is None:
        q_out = torch.empty(qshape, dtype=dt, device=q.device)
    else:
        sqo = _tokens_of(q_out, "q_out", dt, index, qshape)
    if k_out is None:
        k_out = torch.empty(kshape, dtype=dt, device=q.device)
    else:
        sko = _tokens_of(k_out, "k_out", dt, index, kshape)
    dims, _ = _qkrot_sizes(code, qshape, kshape, rot, (sq, sk, sqo, sko, 0, 0, 0, 0), pos_stride, eps, interleaved, False)
    st = _LIB.m3scan_qkrot_fwd(dims, code, q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), pos,
                               _ptr(inv_freq), q_out.data_ptr(), k_out.data_ptr(), _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_qkrot_fwd")
    return q_out, k_out


@_placed
def m3scan_qkrot_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, *, eps=1e-6,
                     interleaved=False, accumulate_param_grads=False, out=None, workspace=None, stream=None):
    """Backward of ``m3scan_qkrot_fwd`` (the same q, k, weights, positions,
    inv_freq, eps and interleaved).  Returns a dict: dq, dk (activation dtype;
    in ``out`` they may be column views of a projection's gradient, or dq_out
    and dk_out themselves) and d_q_weight, d_k_weight (f32 [D]; None for a
    weight that is None)."""
    torch = _TORCH or _torch()
    code, index, qshape, kshape, sq, sk, pos, pos_stride, rot = _qkrot_inputs(q, k, q_weight, k_weight, positions, inv_freq, torch)
    dt, dev, f32, D = q.dtype, q.device, torch.float32, qshape[3]
    o = dict(out) if out else {}
    dq, dk, dwq, dwk = o.get("dq"), o.get("dk"), o.get("d_q_weight"), o.get("d_k_weight")
    sdq = sdk = 0
    if dq is None:
        dq = torch.empty(qshape, dtype=dt, device=dev)
    else:
        sdq = _tokens_of(dq, "dq", dt, index, qshape)
    if dk is None:
        dk = torch.empty(kshape, dtype=dt, device=dev)
    else:
        sdk = _tokens_of(dk, "dk", dt, index, kshape)
    new = torch.zeros if accumulate_param_grads else torch.empty
    if dwq is not None:
        _need(dwq, "d_q_weight", f32, index, (D,))
    elif q_weight is not None:
        dwq = new(D, dtype=f32, device=dev)
    if dwk is not None:
        _need(dwk, "d_k_weight", f32, index, (D,))
    elif k_weight is not None:
        dwk = new(D, dtype=f32, device=dev)
    strides = (sq, sk, 0, 0, sdq, sdk, _tokens_of(dq_out, "dq_out", dt, index, qshape), _tokens_of(dk_out, "dk_out", dt, index, kshape))
    dims, nbytes = _qkrot_sizes(code, qshape, kshape, rot, strides, pos_stride, eps, interleaved, accumulate_param_grads)
    ws, nbytes, _keep = _scratch(workspace, nbytes, torch, dev)
    st = _LIB.m3scan_qkrot_bwd(dims, code, dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(),
                               _ptr(q_weight), _ptr(k_weight), pos, _ptr(inv_freq), dq.data_ptr(), dk.data_ptr(),
                               _ptr(dwq), _ptr(dwk), ws, nbytes, _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_qkrot_bwd")
    o.update(dq=dq, dk=dk, d_q_weight=dwq, d_k_weight=dwk)
    return o


# ---------------------------------------------------------------------------
# linear attention with a decay for each head
# ---------------------------------------------------------------------------

def m3scan_linattn_plan(dims: M3LinattnDims, act: int) -> M3LinattnPlan:
    out = M3LinattnPlan()
    st = _lib_handle().m3scan_linattn_plan(ctypes.byref(dims), int(act), ctypes.byref(out))
    if st != 0:
        raise M3Error(st, "m3scan_linattn_plan")
    return out


@functools.lru_cache(maxsize=1024)
def _linattn_sizes(code, kshape, vshape, strides, scale):
    """(dims, state shape, (forward, any) workspace bytes) for those shapes."""
    if len(kshape) != 4 or len(vshape) != 4 or tuple(kshape[:2]) != tuple(vshape[:2]):
        raise ValueError(f"k and v must be [batch, seq_len, heads, head size], got {tuple(kshape)}, {tuple(vshape)}")
    B, T, Hv, dv = vshape
    Hk, dk = kshape[2:]
    dims = M3LinattnDims(B, T, Hk, Hv, dk, dv, *strides, float(scale), 0)
    pl = m3scan_linattn_plan(dims, code)
    return ctypes.byref(dims), (B, Hv, dk, dv), (pl.fwd_workspace_bytes, pl.workspace_bytes)


def _linattn_inputs(q, k, v, log_decay, torch):
    """Checks the inputs; returns (dtype code, device index, k's and v's
    shapes, token strides of q, k, v)."""
    dt, index = v.dtype, v.get_device()
    code = _act_code(v)
    kshape, vshape = k.shape, v.shape
    if index < 0:
        _check(v, "v")
    if len(kshape) != 4 or len(vshape) != 4:
        raise ValueError(f"k and v must be [batch, seq_len, heads, head size], got {tuple(kshape)}, {tuple(vshape)}")
    _need(log_decay, "log_decay", torch.float32, index, vshape[2:3])
    if (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and q.dtype is dt and k.dtype is dt
            and q.shape == kshape and q.get_device() == index and k.get_device() == index):
        return code, index, kshape, vshape, 0, 0, 0
    kwant = (*vshape[:2], *kshape[2:])
    return (code, index, kshape, vshape, _tokens_of(q, "q", dt, index, kwant), _tokens_of(k, "k", dt, index, kwant),
            _tokens_of(v, "v", dt, index, vshape))


@_placed
def m3scan_linattn_fwd(q, k, v, log_decay, *, state=None, scale=0.0, want_state=True, o=None, state_out=None,
                       workspace=None, stream=None):
    """Linear attention with a decay per head over a sequence.  q, k [B, T, Hk,
    dk], v [B, T, Hv, dv] (column views of a projection's output are fine), bf16
    or f32; ``log_decay`` [Hv] f32; ``state`` [B, Hv, dk, dv] f32 or None
    (zero).  Returns (o, state_out or None)."""
    torch = _TORCH or _torch()
    dev, f32 = v.device, torch.float32
    code, index, kshape, vshape, sq, sk, sv = _linattn_inputs(q, k, v, log_decay, torch)
    dims, sshape, nbytes = _linattn_sizes(code, kshape, vshape, (sq, sk, sv, 0, 0, 0), scale)
    _need(state, "state", f32, index, sshape)
    o = torch.empty(vshape, dtype=v.dtype, device=dev) if o is None else _need(o, "o", v.dtype, index, vshape)
    if state_out is not None:
        _need(state_out, "state_out", f32, index, sshape)
    elif want_state:
        state_out = torch.empty(sshape, dtype=f32, device=dev)
    ws, nbytes, _keep = _scratch(workspace, nbytes[0], torch, dev)
    st = _LIB.m3scan_linattn_fwd(dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(state),
                                 o.data_ptr(), _ptr(state_out), ws, nbytes, _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_linattn_fwd")
    return o, state_out


@_placed
def m3scan_linattn_bwd(q, k, v, log_decay, d_o, *, state=None, d_state_out=None, want_d_state=False, scale=0.0,
                       out=None, workspace=None, stream=None):
    """Backward of ``m3scan_linattn_fwd`` (same q, k, v, log_decay, ``state``
    and scale; no checkpoints).  Returns a dict: dq, dk, dv (activation dtype)
    and d_state (f32, None unless wanted).  dq, dk and dv in ``out`` may be
    column views of a projection's gradient."""
    torch = _TORCH or _torch()
    dev, dt, f32 = v.device, v.dtype, torch.float32
    code, index, kshape, vshape, sq, sk, sv = _linattn_inputs(q, k, v, log_decay, torch)
    r = dict(out) if out else {}
    dq, dk, d_v, d_state = r.get("dq"), r.get("dk"), r.get("dv"), r.get("d_state")
    sdq = sdk = sdv = 0
    if dq is None:
        dq = torch.empty(kshape, dtype=dt, device=dev)
    else:
        sdq = _tokens_of(dq, "dq", dt, index, kshape)
    if dk is None:
        dk = torch.empty(kshape, dtype=dt, device=dev)
    else:
        sdk = _tokens_of(dk, "dk", dt, index, kshape)
    if d_v is None:
        d_v = torch.empty(vshape, dtype=dt, device=dev)
    else:
        sdv = _tokens_of(d_v, "dv", dt, index, vshape)
    dims, sshape, nbytes = _linattn_sizes(code, kshape, vshape, (sq, sk, sv, sdq, sdk, sdv), scale)
    if d_state is not None:
        _need(d_state, "d_state", f32, index, sshape)
    elif want_d_state:
        d_state = torch.empty(sshape, dtype=f32, device=dev)
    _need(state, "state", f32, index, sshape)
    _need(d_state_out, "d_state_out", f32, index, sshape)
    _need(d_o, "d_o", dt, index, vshape)
    ws, nbytes, _keep = _scratch(workspace, nbytes[1], torch, dev)
    st = _LIB.m3scan_linattn_bwd(dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(state),
                                 d_o.data_ptr(), _ptr(d_state_out), dq.data_ptr(), dk.data_ptr(), d_v.data_ptr(),
                                 _ptr(d_state), ws, nbytes, _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_linattn_bwd")
    r.update(dq=dq, dk=dk, dv=d_v, d_state=d_state)
    return r


@_placed
def m3scan_linattn_decode(q, k, v, log_decay, state, *, scale=0.0, o=None, stream=None):
    """A short window (typically one token: T = 1) from the carried ``state``
    [B, Hv, dk, dv] (f32), which is updated in place.  Returns o."""
    torch = _TORCH or _torch()
    code, index, kshape, vshape, sq, sk, sv = _linattn_inputs(q, k, v, log_decay, torch)
    dims, sshape, _ = _linattn_sizes(code, kshape, vshape, (sq, sk, sv, 0, 0, 0), scale)
    o = torch.empty(vshape, dtype=v.dtype, device=v.device) if o is None else _need(o, "o", v.dtype, index, vshape)
    _need(state, "state", torch.float32, index, sshape)
    st = _LIB.m3scan_linattn_decode(dims, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                    state.data_ptr(), o.data_ptr(), _stream_of(stream, index))
    if st:
        raise M3Error(st, "m3scan_linattn_decode")
    return o
