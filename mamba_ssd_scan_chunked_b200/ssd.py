"""Thin Python binding of libssd (include/ssd.h).

Argument marshalling only: every step of the SSD computation runs in the CUDA
kernels of ``libssd.so``.  PyTorch serves as the allocator of device memory and
the source of streams.  There is no fallback: if ``libssd.so`` is missing the
first call raises.

Raw names mirror the C ABI (``ssd_chunk_scan_fwd``, ``ssd_state_update``, ...)
and take integer device pointers; ``chunk_scan_fwd`` and ``state_update`` are
the tensor-level conveniences (shape checks, output and workspace allocation),
as are those of the operators around the scan (``conv1d_fwd``, ``conv1d_update``,
``conv1d_bwd``, ``selective_scan_fwd``, ``selective_state_update``,
``selective_scan_bwd``, ``group_norm_fwd``, ``group_norm_bwd``).  These work on
the device of their tensors and, unless ``stream`` is given, on its current
stream; outputs and workspaces that they allocate belong to the launching stream.
A given ``stream`` first waits for the current one, so that tensors made there may
be passed, and dropped after the call; to leave the two apart make it the current
one (``torch.cuda.stream``).  What a call wrote is read elsewhere after the caller's
own wait for that stream.  Where a graph captures one of the two streams alone there
is no wait, and the tensors are the caller's to keep.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libssd.so")

SSD_F32 = 0
SSD_BF16 = 1

STATUS = {0: "SSD_OK", 1: "SSD_ERR_INVALID_ARG", 2: "SSD_ERR_UNSUPPORTED", 3: "SSD_ERR_ALIGNMENT",
          4: "SSD_ERR_WORKSPACE", 5: "SSD_ERR_CUDA", 6: "SSD_ERR_DEVICE_TIMEOUT"}

# every symbol include/ssd.h declares
EXPORTS = ("ssd_version", "ssd_status_string", "ssd_chunk_scan_workspace_size", "ssd_chunk_scan_path",
           "ssd_chunk_scan_fwd", "ssd_chunk_scan_fwd_varlen", "ssd_chunk_scan_fwd_noalloc",
           "ssd_chunk_scan_bwd", "ssd_chunk_scan_bwd_workspace_size", "ssd_chunk_scan_bwd_launches",
           "ssd_chunk_scan_fwd_mamba3", "ssd_chunk_scan_mamba3_workspace_size", "ssd_chunk_scan_mamba3_launches",
           "ssd_state_update", "ssd_state_update_mimo", "ssd_state_update_mamba3",
           "ssd_replay_buffer_size",
           "ssd_replay_step", "ssd_get_device_error", "ssd_debug_inject",
           "ssd_conv1d_fwd", "ssd_conv1d_update", "ssd_conv1d_bwd", "ssd_conv1d_bwd_workspace_size",
           "ssd_selective_scan_fwd", "ssd_selective_scan_workspace_size", "ssd_selective_state_update",
           "ssd_selective_scan_bwd", "ssd_selective_scan_bwd_workspace_size",
           "ssd_group_norm_fwd", "ssd_group_norm_bwd", "ssd_group_norm_bwd_workspace_size")

# fault-injection bits of ssd_debug_inject
SSD_FAULT_DROP_RUN_PUBLISH = 0x1

# scratch size of ssd_chunk_scan_fwd_noalloc (SSD_NOALLOC_WORKSPACE_BYTES)
NOALLOC_WORKSPACE_BYTES = 32 << 20


class SsdError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class PrefillDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32)]


class DecodeDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class MimoDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("rank", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class ReplayDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("capacity", ctypes.c_int32)]


class Conv1dDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("width", ctypes.c_int64), ("x_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64),
                ("split1", ctypes.c_int64), ("split2", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class SelectiveDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class GroupNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("z_stride", ctypes.c_int64), ("eps", ctypes.c_float), ("x_dtype", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("center", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


# ssd_norm_activation_t
SSD_NORM_NONE, SSD_NORM_SILU, SSD_NORM_GATE_AFTER, SSD_NORM_GATE_BEFORE = 0, 1, 2, 3

_lock = threading.Lock()
_lib = None
_VP = ctypes.c_void_p


def lib():
    """The loaded libssd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m mamba_ssd_scan_chunked_b200.build` (there is no fallback path)")
            L = ctypes.CDLL(LIB_PATH)
            L.ssd_version.restype = ctypes.c_int
            L.ssd_version.argtypes = []
            L.ssd_status_string.restype = ctypes.c_char_p
            L.ssd_status_string.argtypes = [ctypes.c_int]
            L.ssd_chunk_scan_workspace_size.restype = ctypes.c_int
            L.ssd_chunk_scan_workspace_size.argtypes = [ctypes.POINTER(PrefillDesc), ctypes.POINTER(ctypes.c_size_t)]
            L.ssd_chunk_scan_path.restype = ctypes.c_int
            L.ssd_chunk_scan_path.argtypes = [ctypes.POINTER(PrefillDesc), ctypes.POINTER(ctypes.c_int32)]
            L.ssd_chunk_scan_fwd.restype = ctypes.c_int
            L.ssd_chunk_scan_fwd.argtypes = [ctypes.POINTER(PrefillDesc)] + [_VP] * 10 + [_VP, ctypes.c_size_t, _VP]
            L.ssd_chunk_scan_fwd_varlen.restype = ctypes.c_int
            L.ssd_chunk_scan_fwd_varlen.argtypes = [ctypes.POINTER(PrefillDesc)] + [_VP] * 11 + [_VP, ctypes.c_size_t, _VP]
            L.ssd_chunk_scan_fwd_noalloc.restype = ctypes.c_int
            L.ssd_chunk_scan_fwd_noalloc.argtypes = [ctypes.POINTER(PrefillDesc)] + [_VP] * 11
            L.ssd_chunk_scan_bwd.restype = ctypes.c_int
            L.ssd_chunk_scan_bwd.argtypes = [ctypes.POINTER(PrefillDesc)] + [_VP] * 19 + [ctypes.c_size_t, _VP]
            L.ssd_chunk_scan_bwd_workspace_size.restype = ctypes.c_int
            L.ssd_chunk_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(PrefillDesc),
                                                            ctypes.POINTER(ctypes.c_size_t)]
            L.ssd_chunk_scan_bwd_launches.restype = ctypes.c_int
            L.ssd_chunk_scan_bwd_launches.argtypes = [ctypes.POINTER(PrefillDesc), ctypes.c_int32,
                                                      ctypes.POINTER(ctypes.c_int32)]
            L.ssd_chunk_scan_fwd_mamba3.restype = ctypes.c_int
            L.ssd_chunk_scan_fwd_mamba3.argtypes = [ctypes.POINTER(PrefillDesc)] + [_VP] * 13 + [ctypes.c_size_t, _VP]
            L.ssd_chunk_scan_mamba3_workspace_size.restype = ctypes.c_int
            L.ssd_chunk_scan_mamba3_workspace_size.argtypes = [ctypes.POINTER(PrefillDesc),
                                                               ctypes.POINTER(ctypes.c_size_t)]
            L.ssd_chunk_scan_mamba3_launches.restype = ctypes.c_int
            L.ssd_chunk_scan_mamba3_launches.argtypes = [ctypes.POINTER(PrefillDesc)] + [ctypes.c_int32] * 3 + \
                [ctypes.POINTER(ctypes.c_int32)]
            L.ssd_state_update.restype = ctypes.c_int
            L.ssd_state_update.argtypes = [ctypes.POINTER(DecodeDesc)] + [_VP] * 10
            L.ssd_state_update_mimo.restype = ctypes.c_int
            L.ssd_state_update_mimo.argtypes = [ctypes.POINTER(MimoDesc)] + [_VP] * 10
            L.ssd_state_update_mamba3.restype = ctypes.c_int
            L.ssd_state_update_mamba3.argtypes = [ctypes.POINTER(DecodeDesc)] + [_VP] * 14
            L.ssd_replay_buffer_size.restype = ctypes.c_int
            L.ssd_replay_buffer_size.argtypes = [ctypes.POINTER(ReplayDesc), ctypes.POINTER(ctypes.c_size_t)]
            L.ssd_replay_step.restype = ctypes.c_int
            L.ssd_replay_step.argtypes = [ctypes.POINTER(ReplayDesc), _VP, _VP, ctypes.c_int32] + [_VP] * 9
            L.ssd_get_device_error.restype = ctypes.c_int
            L.ssd_get_device_error.argtypes = [_VP, ctypes.POINTER(ctypes.c_uint32)]
            L.ssd_debug_inject.restype = ctypes.c_int
            L.ssd_debug_inject.argtypes = [ctypes.c_uint32]
            size = [ctypes.POINTER(ctypes.c_size_t)]
            for name, desc, args in (
                    ("ssd_conv1d_fwd", Conv1dDesc, [_VP] * 10), ("ssd_conv1d_update", Conv1dDesc, [_VP] * 8),
                    ("ssd_conv1d_bwd", Conv1dDesc, [_VP] * 13 + [ctypes.c_size_t, _VP]),
                    ("ssd_conv1d_bwd_workspace_size", Conv1dDesc, size),
                    ("ssd_selective_scan_fwd", SelectiveDesc, [_VP] * 13 + [ctypes.c_size_t, _VP]),
                    ("ssd_selective_scan_workspace_size", SelectiveDesc, size),
                    ("ssd_selective_state_update", SelectiveDesc, [_VP] * 11),
                    ("ssd_selective_scan_bwd", SelectiveDesc, [_VP] * 21 + [ctypes.c_size_t, _VP]),
                    ("ssd_selective_scan_bwd_workspace_size", SelectiveDesc, size),
                    ("ssd_group_norm_fwd", GroupNormDesc, [_VP] * 6),
                    ("ssd_group_norm_bwd", GroupNormDesc, [_VP] * 10 + [ctypes.c_size_t, _VP]),
                    ("ssd_group_norm_bwd_workspace_size", GroupNormDesc, size)):
                getattr(L, name).restype = ctypes.c_int
                getattr(L, name).argtypes = [ctypes.POINTER(desc)] + args
            _lib = L
    return _lib


# --------------------------------------------------------------------------
# raw C-ABI calls (integer device pointers; 0 = NULL)
# --------------------------------------------------------------------------
def ssd_version() -> int:
    return lib().ssd_version()


def ssd_status_string(status: int) -> str:
    return lib().ssd_status_string(status).decode()


def ssd_chunk_scan_workspace_size(desc: PrefillDesc) -> int:
    n = ctypes.c_size_t(0)
    st = lib().ssd_chunk_scan_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st:
        raise SsdError(st, "ssd_chunk_scan_workspace_size")
    return n.value


def ssd_chunk_scan_path(desc: PrefillDesc) -> int:
    p = ctypes.c_int32(-1)
    st = lib().ssd_chunk_scan_path(ctypes.byref(desc), ctypes.byref(p))
    if st:
        raise SsdError(st, "ssd_chunk_scan_path")
    return p.value


def ssd_chunk_scan_fwd(desc, x, dt_raw, dt_bias, A, B, C, D, init_state, y, final_state,
                       workspace, workspace_bytes, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_chunk_scan_fwd(ctypes.byref(desc), x or None, dt_raw or None, dt_bias or None, A or None,
                                     B or None, C or None, D or None, init_state or None, y or None,
                                     final_state or None, workspace or None, int(workspace_bytes), stream or None)


def ssd_chunk_scan_fwd_varlen(desc, x, dt_raw, dt_bias, A, B, C, D, init_state, pad_left, y, final_state,
                              workspace, workspace_bytes, stream) -> int:
    """Raw call of the left-padded variable-length variant; returns the status code."""
    return lib().ssd_chunk_scan_fwd_varlen(ctypes.byref(desc), x or None, dt_raw or None, dt_bias or None, A or None,
                                           B or None, C or None, D or None, init_state or None, pad_left or None,
                                           y or None, final_state or None, workspace or None, int(workspace_bytes),
                                           stream or None)


def ssd_chunk_scan_bwd(desc, x, dt_raw, dt_bias, A, B, C, D, init_state, dy, dfinal_state, dx, ddt_raw, ddt_bias, dA,
                       dB, dC, dD, dinit_state, workspace, workspace_bytes, stream) -> int:
    """Raw call of the backward pass; returns the status code (0 = enqueued)."""
    ptrs = (x, dt_raw, dt_bias, A, B, C, D, init_state, dy, dfinal_state, dx, ddt_raw, ddt_bias, dA, dB, dC, dD,
            dinit_state, workspace)
    return lib().ssd_chunk_scan_bwd(ctypes.byref(desc), *(p or None for p in ptrs), int(workspace_bytes),
                                     stream or None)


def ssd_chunk_scan_fwd_mamba3(desc, x, dt_raw, dt_bias, A, B, C, D, lam, theta, init_state, y, final_state,
                              workspace, workspace_bytes, stream) -> int:
    """Raw call of the Mamba-3 prefill; returns the status code (0 = enqueued)."""
    ptrs = (x, dt_raw, dt_bias, A, B, C, D, lam, theta, init_state, y, final_state, workspace)
    return lib().ssd_chunk_scan_fwd_mamba3(ctypes.byref(desc), *(p or None for p in ptrs), int(workspace_bytes),
                                            stream or None)


def ssd_chunk_scan_mamba3_workspace_size(desc: PrefillDesc) -> int:
    n = ctypes.c_size_t(0)
    st = lib().ssd_chunk_scan_mamba3_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st:
        raise SsdError(st, "ssd_chunk_scan_mamba3_workspace_size")
    return int(n.value)


def ssd_chunk_scan_mamba3_launches(desc: PrefillDesc, has_lam: bool, has_theta: bool, has_final: bool) -> int:
    n = ctypes.c_int32(0)
    st = lib().ssd_chunk_scan_mamba3_launches(ctypes.byref(desc), int(bool(has_lam)), int(bool(has_theta)),
                                              int(bool(has_final)), ctypes.byref(n))
    if st:
        raise SsdError(st, "ssd_chunk_scan_mamba3_launches")
    return int(n.value)


def ssd_chunk_scan_bwd_workspace_size(desc: PrefillDesc) -> int:
    n = ctypes.c_size_t(0)
    st = lib().ssd_chunk_scan_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(n))
    if st:
        raise SsdError(st, "ssd_chunk_scan_bwd_workspace_size")
    return int(n.value)


def ssd_chunk_scan_bwd_launches(desc: PrefillDesc, has_states: bool) -> int:
    n = ctypes.c_int32(0)
    st = lib().ssd_chunk_scan_bwd_launches(ctypes.byref(desc), int(bool(has_states)), ctypes.byref(n))
    if st:
        raise SsdError(st, "ssd_chunk_scan_bwd_launches")
    return int(n.value)


def ssd_chunk_scan_fwd_noalloc(desc, x, dt_raw, dt_bias, A, B, C, D, init_state, y, final_state, stream) -> int:
    """Raw call of the variant without a caller workspace; returns the status code."""
    return lib().ssd_chunk_scan_fwd_noalloc(ctypes.byref(desc), x or None, dt_raw or None, dt_bias or None, A or None,
                                            B or None, C or None, D or None, init_state or None, y or None,
                                            final_state or None, stream or None)


def ssd_state_update(desc, state, x, dt_raw, dt_bias, A, B, C, D, y, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_state_update(ctypes.byref(desc), state or None, x or None, dt_raw or None, dt_bias or None,
                                  A or None, B or None, C or None, D or None, y or None, stream or None)


def ssd_state_update_mimo(desc, state, x, dt_raw, dt_bias, A, B, C, D, y, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_state_update_mimo(ctypes.byref(desc), state or None, x or None, dt_raw or None, dt_bias or None,
                                       A or None, B or None, C or None, D or None, y or None, stream or None)


def ssd_state_update_mamba3(desc, state, x, x_prev, dt_raw, dt_bias, A, B, B_prev, C, D, lam, theta, y,
                            stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_state_update_mamba3(ctypes.byref(desc), state or None, x or None, x_prev or None, dt_raw or None,
                                         dt_bias or None, A or None, B or None, B_prev or None, C or None, D or None,
                                         lam or None, theta or None, y or None, stream or None)


def ssd_replay_buffer_size(desc: ReplayDesc) -> int:
    n = ctypes.c_size_t(0)
    st = lib().ssd_replay_buffer_size(ctypes.byref(desc), ctypes.byref(n))
    if st:
        raise SsdError(st, "ssd_replay_buffer_size")
    return n.value


def ssd_replay_step(desc, checkpoint, buffer, fill, x, dt_raw, dt_bias, A, B, C, D, y, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_replay_step(ctypes.byref(desc), checkpoint or None, buffer or None, int(fill), x or None,
                                 dt_raw or None, dt_bias or None, A or None, B or None, C or None, D or None,
                                 y or None, stream or None)


def ssd_get_device_error(stream=None):
    """Synchronise ``stream`` and return (status, detail bits) of the device error word."""
    d = ctypes.c_uint32(0)
    st = lib().ssd_get_device_error(stream or None, ctypes.byref(d))
    return st, d.value


def ssd_debug_inject(faults: int) -> int:
    """Test hook: fault bits injected into every following launch (0 clears)."""
    return lib().ssd_debug_inject(int(faults))


def ssd_conv1d_fwd(desc, x, weight, bias, init_state, pad_left, y0, y1, y2, final_state, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_conv1d_fwd(desc, x, weight, bias, init_state, pad_left, y0, y1, y2, final_state, stream)


def ssd_conv1d_update(desc, state, x, weight, bias, y0, y1, y2, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_conv1d_update(desc, state, x, weight, bias, y0, y1, y2, stream)


def ssd_conv1d_bwd(desc, x, weight, bias, init_state, dy0, dy1, dy2, dfinal_state, dx, dweight, dbias, dinit_state,
                   workspace, workspace_bytes, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_conv1d_bwd(desc, x, weight, bias, init_state, dy0, dy1, dy2, dfinal_state, dx, dweight, dbias,
                                dinit_state, workspace, workspace_bytes, stream)


def ssd_selective_scan_fwd(desc, x, dt_raw, dt_bias, A, B, C, D, z, init_state, pad_left, y, final_state, workspace,
                           workspace_bytes, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_selective_scan_fwd(desc, x, dt_raw, dt_bias, A, B, C, D, z, init_state, pad_left, y, final_state,
                                        workspace, workspace_bytes, stream)


def ssd_selective_state_update(desc, state, x, dt_raw, dt_bias, A, B, C, D, z, y, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_selective_state_update(desc, state, x, dt_raw, dt_bias, A, B, C, D, z, y, stream)


def ssd_selective_scan_bwd(desc, x, dt_raw, dt_bias, A, B, C, D, z, init_state, dy, dfinal_state, dx, ddt_raw,
                           ddt_bias, dA, dB, dC, dD, dz, dinit_state, workspace, workspace_bytes, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_selective_scan_bwd(desc, x, dt_raw, dt_bias, A, B, C, D, z, init_state, dy, dfinal_state, dx,
                                        ddt_raw, ddt_bias, dA, dB, dC, dD, dz, dinit_state, workspace, workspace_bytes,
                                        stream)


def ssd_group_norm_fwd(desc, x, z, weight, bias, y, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_group_norm_fwd(desc, x, z, weight, bias, y, stream)


def ssd_group_norm_bwd(desc, x, z, weight, bias, dy, dx, dz, dweight, dbias, workspace, workspace_bytes, stream) -> int:
    """Raw call; returns the status code (0 = enqueued)."""
    return lib().ssd_group_norm_bwd(desc, x, z, weight, bias, dy, dx, dz, dweight, dbias, workspace, workspace_bytes,
                                    stream)


def _size_of(name, desc) -> int:
    n = ctypes.c_size_t(0)
    st = getattr(lib(), name)(desc, n)
    if st:
        raise SsdError(st, name)
    return n.value


def ssd_conv1d_bwd_workspace_size(desc: Conv1dDesc) -> int:
    return _size_of("ssd_conv1d_bwd_workspace_size", desc)


def ssd_selective_scan_workspace_size(desc: SelectiveDesc) -> int:
    return _size_of("ssd_selective_scan_workspace_size", desc)


def ssd_selective_scan_bwd_workspace_size(desc: SelectiveDesc) -> int:
    return _size_of("ssd_selective_scan_bwd_workspace_size", desc)


def ssd_group_norm_bwd_workspace_size(desc: GroupNormDesc) -> int:
    return _size_of("ssd_group_norm_bwd_workspace_size", desc)


# --------------------------------------------------------------------------
# tensor-level conveniences
# --------------------------------------------------------------------------
def _dtype_code(t) -> int:
    import torch
    if t == torch.float32:
        return SSD_F32
    if t == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"unsupported dtype {t}; libssd takes float32 or bfloat16")


def _torch_dtype(code: int):
    import torch
    return torch.bfloat16 if code == SSD_BF16 else torch.float32


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _expect(t, shape, name, dtype=None):
    """The C ABI takes bare pointers and sizes from the descriptor, so a tensor of
    another shape or dtype than the descriptor implies would be read or written
    out of bounds: refuse it here (None passes: optional arguments)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def prefill_desc(x, B, chunk, y_dtype=None, state_dtype=None) -> PrefillDesc:
    import torch
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    io = _dtype_code(x.dtype)
    return PrefillDesc(b, L, H, P, N, G, int(chunk), io,
                       _dtype_code(y_dtype) if y_dtype is not None else io,
                       _dtype_code(state_dtype) if state_dtype is not None else SSD_F32)


def workspace_bytes(x, B, chunk, y_dtype=None, state_dtype=None) -> int:
    return ssd_chunk_scan_workspace_size(prefill_desc(x, B, chunk, y_dtype, state_dtype))


def _check_prefill_args(desc, x, dt_raw, dt_bias, A, B, C, D, init_state):
    import torch
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _expect(dt_raw, (b, L, H), "dt_raw", x.dtype)
    _expect(B, (b, L, G, N), "B", x.dtype)
    _expect(C, (b, L, G, N), "C", x.dtype)
    for name, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _expect(t, (H,), name, torch.float32)
    _expect(init_state, (b, H, N, P), "init_state", _torch_dtype(desc.state_dtype))


def chunk_scan_fwd(x, dt_raw, dt_bias, A, B, C, D, chunk, init_state=None, *, y=None, final_state=None,
                   y_dtype=None, state_dtype=None, want_final_state=True, workspace=None, pad_left=None, stream=None):
    """Chunked prefill scan.  Shapes: x [b,L,H,P], dt_raw [b,L,H], B/C [b,L,G,N], dt_bias/A/D [H] (fp32);
    ``pad_left`` (int32 [b], CUDA) marks left-padded variable-length sequences.

    Returns (y, final_state).  Outputs and workspace are allocated with torch
    when not given; ``state_dtype`` defaults to init_state's dtype, else fp32.
    """
    import torch
    if y_dtype is None and y is not None:
        y_dtype = y.dtype
    if state_dtype is None:
        state_dtype = (init_state.dtype if init_state is not None else
                       final_state.dtype if final_state is not None else torch.float32)
    desc = prefill_desc(x, B, chunk, y_dtype, state_dtype)
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _check_prefill_args(desc, x, dt_raw, dt_bias, A, B, C, D, init_state)
    _expect(y, (b, L, H, P), "y", _torch_dtype(desc.y_dtype))
    _expect(final_state, (b, H, N, P), "final_state", _torch_dtype(desc.state_dtype))
    _expect(pad_left, (b,), "pad_left")
    for t in (x, dt_raw, B, C, dt_bias, A, D, init_state, y, final_state):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    if y is None:
        y = torch.empty((b, L, H, P), dtype=_torch_dtype(desc.y_dtype), device=x.device)
    if final_state is None and want_final_state:
        final_state = torch.empty((b, H, N, P), dtype=_torch_dtype(desc.state_dtype), device=x.device)
    need = ssd_chunk_scan_workspace_size(desc)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if pad_left is None:
        st = ssd_chunk_scan_fwd(desc, _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                _ptr(init_state), _ptr(y), _ptr(final_state), _ptr(workspace), workspace.numel(),
                                _stream(stream))
    else:
        if pad_left.dtype != torch.int32 or not pad_left.is_cuda or not pad_left.is_contiguous():
            raise ValueError("pad_left must be a contiguous int32 CUDA tensor [batch]")
        st = ssd_chunk_scan_fwd_varlen(desc, _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
                                       _ptr(D), _ptr(init_state), _ptr(pad_left), _ptr(y), _ptr(final_state),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    if st:
        raise SsdError(st, "ssd_chunk_scan_fwd")
    return y, final_state


def chunk_scan_fwd_mamba3(x, dt_raw, dt_bias, A, B, C, D, chunk, lam=None, theta=None, init_state=None, *,
                          y_dtype=None, state_dtype=None, want_final_state=True, workspace=None, stream=None):
    """Mamba-3 prefill (trapezoidal input mix ``lam`` [b,L,H] fp32, rotation
    angles ``theta`` [b,L,G,N/2] fp32; either may be None).  Returns (y, final_state)."""
    import torch
    if state_dtype is None:
        state_dtype = init_state.dtype if init_state is not None else torch.float32
    desc = prefill_desc(x, B, chunk, y_dtype, state_dtype)
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _check_prefill_args(desc, x, dt_raw, dt_bias, A, B, C, D, init_state)
    _expect(lam, (b, L, H), "lam")
    _expect(theta, (b, L, G, N // 2), "theta")
    for t in (x, dt_raw, B, C, dt_bias, A, D, lam, theta, init_state):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    for t in (lam, theta):
        if t is not None and t.dtype != torch.float32:
            raise ValueError("lam and theta are fp32")
    y = torch.empty((b, L, H, P), dtype=_torch_dtype(desc.y_dtype), device=x.device)
    final_state = (torch.empty((b, H, N, P), dtype=_torch_dtype(desc.state_dtype), device=x.device)
                   if want_final_state else None)
    need = ssd_chunk_scan_mamba3_workspace_size(desc)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    st = ssd_chunk_scan_fwd_mamba3(desc, _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                   _ptr(lam), _ptr(theta), _ptr(init_state), _ptr(y), _ptr(final_state),
                                   _ptr(workspace), workspace.numel(), _stream(stream))
    if st:
        raise SsdError(st, "ssd_chunk_scan_fwd_mamba3")
    return y, final_state


def chunk_scan_bwd(x, dt_raw, dt_bias, A, B, C, D, chunk, dy, init_state=None, dfinal_state=None, *,
                   grad_dtype=None, state_dtype=None, want_dinit=True, workspace=None, stream=None):
    """Backward pass of ``chunk_scan_fwd``: gradients of sum<dy, y> + <dfinal_state, final_state>.

    Returns a dict of CUDA tensors: dx, ddt_raw, dB, dC (``grad_dtype``, default
    x's dtype), dA, ddt_bias, dD (fp32 [H]) and dinit_state (state dtype, or
    None when ``want_dinit`` is false).
    """
    import torch
    if state_dtype is None:
        src = init_state if init_state is not None else dfinal_state
        state_dtype = src.dtype if src is not None else torch.float32
    desc = prefill_desc(x, B, chunk, grad_dtype, state_dtype)
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _check_prefill_args(desc, x, dt_raw, dt_bias, A, B, C, D, init_state)
    _expect(dy, (b, L, H, P), "dy", x.dtype)
    _expect(dfinal_state, (b, H, N, P), "dfinal_state", _torch_dtype(desc.state_dtype))
    for t in (x, dt_raw, B, C, dt_bias, A, D, init_state, dy, dfinal_state):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    gd, dev = _torch_dtype(desc.y_dtype), x.device
    out = {"dx": torch.empty((b, L, H, P), dtype=gd, device=dev),
           "ddt_raw": torch.empty((b, L, H), dtype=gd, device=dev),
           "dB": torch.empty((b, L, G, N), dtype=gd, device=dev),
           "dC": torch.empty((b, L, G, N), dtype=gd, device=dev),
           "dA": torch.empty(H, dtype=torch.float32, device=dev),
           "ddt_bias": torch.empty(H, dtype=torch.float32, device=dev),
           "dD": torch.empty(H, dtype=torch.float32, device=dev),
           "dinit_state": (torch.empty((b, H, N, P), dtype=_torch_dtype(desc.state_dtype), device=dev)
                           if want_dinit else None)}
    need = ssd_chunk_scan_bwd_workspace_size(desc)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    st = ssd_chunk_scan_bwd(desc, _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                            _ptr(init_state), _ptr(dy), _ptr(dfinal_state), _ptr(out["dx"]), _ptr(out["ddt_raw"]),
                            _ptr(out["ddt_bias"]), _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]),
                            _ptr(out["dD"]), _ptr(out["dinit_state"]), _ptr(workspace), workspace.numel(),
                            _stream(stream))
    if st:
        raise SsdError(st, "ssd_chunk_scan_bwd")
    return out


def _check_decode_args(state, x, dt_raw, dt_bias, A, B, C, D, y, y_dtype, bshape=None):
    import torch
    b, H = x.shape[0], x.shape[1]
    P = x.shape[-1]
    G, N = B.shape[1], B.shape[-1]
    _expect(state, (b, H, N, P), "state")
    _expect(dt_raw, (b, H), "dt_raw", x.dtype)
    _expect(B, bshape or (b, G, N), "B", x.dtype)
    _expect(C, bshape or (b, G, N), "C", x.dtype)
    for name, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _expect(t, (H,), name, torch.float32)
    _expect(y, tuple(x.shape), "y", y_dtype)


def state_update(state, x, dt_raw, dt_bias, A, B, C, D, *, y=None, y_dtype=None, stream=None):
    """Decode step in place on ``state`` [b,H,N,P].  x [b,H,P], dt_raw [b,H], B/C [b,G,N].  Returns y."""
    import torch
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    if y_dtype is None and y is not None:
        y_dtype = y.dtype
    _check_decode_args(state, x, dt_raw, dt_bias, A, B, C, D, y, y_dtype)
    io = _dtype_code(x.dtype)
    desc = DecodeDesc(b, H, P, N, G, io, _dtype_code(y_dtype) if y_dtype is not None else io,
                      _dtype_code(state.dtype))
    for t in (state, x, dt_raw, B, C, dt_bias, A, D, y):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    if y is None:
        y = torch.empty((b, H, P), dtype=_torch_dtype(desc.y_dtype), device=x.device)
    st = ssd_state_update(desc, _ptr(state), _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
                          _ptr(D), _ptr(y), _stream(stream))
    if st:
        raise SsdError(st, "ssd_state_update")
    return y


def state_update_mamba3(state, x, dt_raw, dt_bias, A, B, C, D, *, x_prev=None, B_prev=None, lam=None, theta=None,
                        y=None, y_dtype=None, stream=None):
    """Mamba-3 decode step in place on ``state`` [b,H,N,P]: x, x_prev [b,H,P], dt_raw [b,H],
    B, B_prev, C [b,G,N], lam [b,H] (fp32), theta [b,G,N/2] (fp32).  x_prev and B_prev
    are the previous token's x and B (None before the first token).  Returns y."""
    import torch
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    if y_dtype is None and y is not None:
        y_dtype = y.dtype
    _check_decode_args(state, x, dt_raw, dt_bias, A, B, C, D, y, y_dtype)
    _expect(x_prev, (b, H, P), "x_prev", x.dtype)
    _expect(B_prev, (b, G, N), "B_prev", x.dtype)
    _expect(lam, (b, H), "lam")
    _expect(theta, (b, G, N // 2), "theta")
    io = _dtype_code(x.dtype)
    desc = DecodeDesc(b, H, P, N, G, io, _dtype_code(y_dtype) if y_dtype is not None else io,
                      _dtype_code(state.dtype))
    for t in (state, x, x_prev, dt_raw, B, B_prev, C, dt_bias, A, D, lam, theta, y):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    if y is None:
        y = torch.empty((b, H, P), dtype=_torch_dtype(desc.y_dtype), device=x.device)
    st = ssd_state_update_mamba3(desc, _ptr(state), _ptr(x), _ptr(x_prev), _ptr(dt_raw), _ptr(dt_bias), _ptr(A),
                                 _ptr(B), _ptr(B_prev), _ptr(C), _ptr(D), _ptr(lam), _ptr(theta), _ptr(y),
                                 _stream(stream))
    if st:
        raise SsdError(st, "ssd_state_update_mamba3")
    return y


def replay_desc(checkpoint, x, B, capacity, y_dtype=None) -> ReplayDesc:
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    io = _dtype_code(x.dtype)
    return ReplayDesc(b, H, P, N, G, io, _dtype_code(y_dtype) if y_dtype is not None else io,
                      _dtype_code(checkpoint.dtype), int(capacity))


def replay_buffer(checkpoint, x, B, capacity):
    """A device buffer of the size ssd_replay_step needs (uint8, 256-byte aligned by the allocator)."""
    import torch
    n = ssd_replay_buffer_size(replay_desc(checkpoint, x, B, capacity))
    return torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)


def replay_step(checkpoint, buffer, fill, capacity, x, dt_raw, dt_bias, A, B, C, D, *, y=None, y_dtype=None,
                stream=None):
    """Replayed decode step: checkpoint [b,H,N,P] + buffer (``replay_buffer``) holding ``fill``
    tokens; x [b,H,P], dt_raw [b,H], B/C [b,G,N].  Returns (y, next fill)."""
    import torch
    if y_dtype is None and y is not None:
        y_dtype = y.dtype
    _check_decode_args(checkpoint, x, dt_raw, dt_bias, A, B, C, D, y, y_dtype)
    desc = replay_desc(checkpoint, x, B, capacity, y_dtype)
    if buffer is not None and buffer.numel() * buffer.element_size() < ssd_replay_buffer_size(desc):
        raise ValueError("buffer: smaller than ssd_replay_buffer_size")
    for t in (checkpoint, buffer, x, dt_raw, B, C, dt_bias, A, D, y):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    b, H, P = x.shape
    if y is None:
        y = torch.empty((b, H, P), dtype=_torch_dtype(desc.y_dtype), device=x.device)
    st = ssd_replay_step(desc, _ptr(checkpoint), _ptr(buffer), fill, _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A),
                         _ptr(B), _ptr(C), _ptr(D), _ptr(y), _stream(stream))
    if st:
        raise SsdError(st, "ssd_replay_step")
    return y, (fill + 1) % int(capacity)


def state_update_mimo(state, x, dt_raw, dt_bias, A, B, C, D, *, y=None, y_dtype=None, stream=None):
    """MIMO decode step in place on ``state`` [b,H,N,P].  x [b,H,R,P], dt_raw [b,H], B/C [b,G,R,N].  Returns y."""
    import torch
    b, H, R, P = x.shape
    G, N = B.shape[1], B.shape[3]
    if y_dtype is None and y is not None:
        y_dtype = y.dtype
    _check_decode_args(state, x, dt_raw, dt_bias, A, B, C, D, y, y_dtype, bshape=(b, G, R, N))
    io = _dtype_code(x.dtype)
    desc = MimoDesc(b, H, P, N, G, R, io, _dtype_code(y_dtype) if y_dtype is not None else io,
                    _dtype_code(state.dtype))
    for t in (state, x, dt_raw, B, C, dt_bias, A, D, y):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libssd takes contiguous CUDA tensors")
    if y is None:
        y = torch.empty((b, H, R, P), dtype=_torch_dtype(desc.y_dtype), device=x.device)
    st = ssd_state_update_mimo(desc, _ptr(state), _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(D), _ptr(y), _stream(stream))
    if st:
        raise SsdError(st, "ssd_state_update_mimo")
    return y


# --------------------------------------------------------------------------
# the operators around the scan
# --------------------------------------------------------------------------
# A token's calls take a few microseconds on the device, so these wrappers read
# each property of a tensor once.
def _code(dtype) -> int:
    c = _CODES.get(dtype)
    if c is None:
        c = _CODES[dtype] = _dtype_code(dtype)
    return c


_CODES = {}


def _check(t, shape, name, dtype=None):
    """As ``_expect``."""
    if t is not None and (t.shape != shape or (dtype is not None and t.dtype != dtype)):
        _expect(t, shape, name, dtype)


def _row_stride(t, name, lead, width, dtype):
    """Elements from a row of ``t`` (shape ``lead + (width,)``, possibly columns cut out of wider
    rows) to the next one; the rows follow each other at one distance."""
    _check(t, lead + (width,), name, dtype)
    if t.is_contiguous():
        return width
    strides = t.stride()
    if strides[-1] != 1 and width > 1:
        raise ValueError(f"{name}: the channels have to be neighbours in memory")
    stride, rows = None, 1
    for n, st in zip(reversed(lead), reversed(strides[:-1])):
        if n != 1:
            if stride is None:
                stride = st
            elif st != stride * rows:
                raise ValueError(f"{name}: rows at one distance expected, strides {strides}")
        rows *= n
    if stride is None:
        return width
    if stride < width:
        raise ValueError(f"{name}: overlapping rows, strides {strides}")
    return stride


def _one_device(dense, rows=()) -> int:
    """The index of the CUDA device of all the tensors (None passes); the ``dense`` ones have to be contiguous."""
    index = None
    for t in dense:
        if t is not None:
            i = t.get_device()
            if i != index:
                if i < 0:
                    raise ValueError("libssd takes contiguous CUDA tensors")
                if index is not None:
                    raise ValueError(f"tensors on devices {index} and {i}: libssd takes them on one device")
                index = i
            if not t.is_contiguous():
                raise ValueError("libssd takes contiguous CUDA tensors")
    for t in rows:
        if t is not None and t.get_device() != index:
            if t.get_device() < 0:
                raise ValueError("libssd takes contiguous CUDA tensors")
            if index is not None:
                raise ValueError(f"tensors on devices {index} and {t.get_device()}: libssd takes them on one device")
            index = t.get_device()
    return index


def _launch_on(index, stream, call, tensors=()):
    """``call(handle)`` with device ``index`` the current one and ``stream`` (None: the device's current
    stream) the one that outputs and workspaces are allocated for and the call is enqueued on.  A stream
    other than the current one waits for the current one first, and ``tensors`` (the caller's; None passes)
    keep their memory until it has used them."""
    import torch
    if stream is None:
        if index == torch.cuda.current_device():
            return call(torch._C._cuda_getCurrentRawStream(index))   # the handle alone, 3 us less than the object
        with torch.cuda.device(index):
            return call(torch._C._cuda_getCurrentRawStream(index))
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    if stream.device.index != index:
        raise ValueError(f"stream on device {stream.device.index}, tensors on device {index}")
    with torch.cuda.device(index):
        current = torch.cuda.current_stream(index)
        captured = torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(stream):
            # a graph that captures one of the two streams alone cannot hold the wait
            if stream.cuda_stream != current.cuda_stream and torch.cuda.is_current_stream_capturing() == captured:
                stream.wait_stream(current)
                for t in tensors:
                    if t is not None:
                        t.record_stream(stream)
            return call(stream.cuda_stream)


def _workspace(workspace, need, x):
    """The address and size of the caller's workspace when it is large enough, else of one of this call's
    own beside x, and the tensor."""
    if workspace is not None:
        nbytes = workspace.numel() * workspace.element_size()
        if nbytes >= need:
            return workspace.data_ptr(), nbytes, workspace
    if need == 0:
        return 0, 0, None
    import torch
    workspace = x.new_empty(need, dtype=torch.uint8)
    return workspace.data_ptr(), need, workspace


def _silu_flag(activation) -> int:
    if activation is None:
        return 0
    if activation != "silu":
        raise ValueError(f"activation: {activation!r}, expected None or 'silu'")
    return 1


def _split_widths(split, channels):
    if split is None:
        return (channels,)
    widths = tuple(split)
    if not 1 <= len(widths) <= 3 or min(widths) < 1 or sum(widths) != channels:
        raise ValueError(f"split: {split}, expected one to three widths that add up to {channels} channels")
    return widths


def _conv_outputs(y, widths, lead, dtype, one):
    """The given outputs, checked."""
    y = [y] if one and hasattr(y, "shape") else list(y)
    if len(y) != len(widths):
        raise ValueError(f"y: {len(y)} tensors, expected {len(widths)}")
    for t, n in zip(y, widths):
        _check(t, lead + (n,), "y", dtype)
    return y


def _three(tensors):
    """The addresses of up to three tensors, 0 for those that are not there."""
    n = len(tensors)
    return (tensors[0].data_ptr(), tensors[1].data_ptr() if n > 1 else 0, tensors[2].data_ptr() if n > 2 else 0)


def _conv_desc(b, L, D, W, xs, dxs, widths, io, y, state, activation) -> Conv1dDesc:
    n = len(widths)
    return Conv1dDesc(b, L, D, W, xs, dxs, widths[1] if n > 1 else 0, widths[2] if n > 2 else 0, _code(io), _code(y),
                      _code(state), _silu_flag(activation))


def conv1d_fwd(x, weight, bias=None, init_state=None, *, split=None, activation="silu", pad_left=None, y=None,
               final_state=None, y_dtype=None, state_dtype=None, want_final_state=True, stream=None):
    """Short causal convolution: x [b,L,D] (columns of wider rows are taken), weight [D,W] and bias [D] fp32,
    W = 2, 3 or 4; the W - 1 inputs before the first token are init_state [b,W-1,D]'s.

    ``split``: widths of up to three dense output tensors (as the scan takes x, B and C); None gives one.
    ``pad_left`` (int32 [b], CUDA): leading tokens that are absent; y is 0 there.
    Returns (y, final_state): a tensor, with ``split`` a tuple of them, and the kept inputs [b,W-1,D]
    (None without ``want_final_state``); state_dtype defaults to init_state's dtype, else fp32.
    """
    import torch
    b, L, D = x.shape
    W = weight.shape[1]
    widths = _split_widths(split, D)
    xs = _row_stride(x, "x", (b, L), D, None)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else (y if hasattr(y, "dtype") else y[0]).dtype
    if state_dtype is None:
        state_dtype = (init_state.dtype if init_state is not None else
                       final_state.dtype if final_state is not None else torch.float32)
    kept = (b, W - 1, D)
    _check(weight, (D, W), "weight", torch.float32)
    _check(bias, (D,), "bias", torch.float32)
    _check(init_state, kept, "init_state", state_dtype)
    _check(final_state, kept, "final_state", state_dtype)
    _check(pad_left, (b,), "pad_left", torch.int32)
    out = _conv_outputs(y, widths, (b, L), y_dtype, split is None) if y is not None else ()
    desc = _conv_desc(b, L, D, W, xs, D, widths, x.dtype, y_dtype, state_dtype, activation)
    dense, rows = (weight, bias, init_state, pad_left, final_state, *out), (x,)
    device = _one_device(dense, rows)

    def call(handle):
        ys = out if y is not None else [x.new_empty((b, L, n), dtype=y_dtype) for n in widths]
        final = final_state
        if final is None and want_final_state:
            final = x.new_empty(kept, dtype=state_dtype)
        st = ssd_conv1d_fwd(desc, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(init_state), _ptr(pad_left),
                            *_three(ys), _ptr(final), handle)
        if st:
            raise SsdError(st, "ssd_conv1d_fwd")
        return (ys[0] if split is None else tuple(ys)), final

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def conv1d_update(state, x, weight, bias=None, *, split=None, activation="silu", y=None, y_dtype=None, stream=None):
    """One token of ``conv1d_fwd``, in place on the kept inputs ``state`` [b,W-1,D]: x [b,D] (columns of wider
    rows are taken).  Returns y [b,D], with ``split`` a tuple of tensors."""
    import torch
    b, D = x.shape
    W = weight.shape[1]
    widths = _split_widths(split, D)
    xs = _row_stride(x, "x", (b,), D, None)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else (y if hasattr(y, "dtype") else y[0]).dtype
    _check(weight, (D, W), "weight", torch.float32)
    _check(bias, (D,), "bias", torch.float32)
    _check(state, (b, W - 1, D), "state")
    out = _conv_outputs(y, widths, (b,), y_dtype, split is None) if y is not None else ()
    desc = _conv_desc(b, 1, D, W, xs, D, widths, x.dtype, y_dtype, state.dtype, activation)
    dense, rows = (state, weight, bias, *out), (x,)
    device = _one_device(dense, rows)

    def call(handle):
        ys = out if y is not None else [x.new_empty((b, n), dtype=y_dtype) for n in widths]
        st = ssd_conv1d_update(desc, state.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), *_three(ys), handle)
        if st:
            raise SsdError(st, "ssd_conv1d_update")
        return ys[0] if split is None else tuple(ys)

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def conv1d_bwd(x, weight, bias, dy, init_state=None, dfinal_state=None, *, activation="silu", dx=None,
               grad_dtype=None, state_dtype=None, want_dinit=True, workspace=None, stream=None):
    """Backward pass of ``conv1d_fwd`` (without padding): gradients of sum<dy, y> + <dfinal_state, final_state>.

    ``dy``: a tensor [b,L,D] or the tuple of the split outputs' gradients, in x's dtype.  ``dx`` may be given,
    as columns of wider rows too (the other columns are left as they were); else it is allocated dense, in
    ``grad_dtype`` (default x's dtype).  Returns a dict: dx, dweight [D,W] and dbias [D] fp32 (None without
    bias), dinit_state [b,W-1,D] (None without ``want_dinit``).
    """
    import torch
    b, L, D = x.shape
    W = weight.shape[1]
    dys = [dy] if hasattr(dy, "shape") else list(dy)
    widths = _split_widths([t.shape[-1] for t in dys], D)
    xs = _row_stride(x, "x", (b, L), D, None)
    if grad_dtype is None:
        grad_dtype = dx.dtype if dx is not None else x.dtype
    dxs = D if dx is None else _row_stride(dx, "dx", (b, L), D, grad_dtype)
    if state_dtype is None:
        src = init_state if init_state is not None else dfinal_state
        state_dtype = src.dtype if src is not None else torch.float32
    kept = (b, W - 1, D)
    _check(weight, (D, W), "weight", torch.float32)
    _check(bias, (D,), "bias", torch.float32)
    _check(init_state, kept, "init_state", state_dtype)
    _check(dfinal_state, kept, "dfinal_state", state_dtype)
    for t, n in zip(dys, widths):
        _check(t, (b, L, n), "dy", x.dtype)
    desc = _conv_desc(b, L, D, W, xs, dxs, widths, x.dtype, grad_dtype, state_dtype, activation)
    dense, rows = (weight, bias, init_state, dfinal_state, workspace, *dys), (x, dx)
    device = _one_device(dense, rows)
    need = ssd_conv1d_bwd_workspace_size(desc)

    def call(handle):
        f32, empty = torch.float32, x.new_empty
        out = {"dx": empty((b, L, D), dtype=grad_dtype) if dx is None else dx,
               "dweight": empty((D, W), dtype=f32),
               "dbias": empty(D, dtype=f32) if bias is not None else None,
               "dinit_state": empty(kept, dtype=state_dtype) if want_dinit else None}
        ws, nbytes, keep = _workspace(workspace, need, x)
        st = ssd_conv1d_bwd(desc, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(init_state), *_three(dys),
                            _ptr(dfinal_state), out["dx"].data_ptr(), out["dweight"].data_ptr(), _ptr(out["dbias"]),
                            _ptr(out["dinit_state"]), ws, nbytes, handle)
        if st:
            raise SsdError(st, "ssd_conv1d_bwd")
        return out

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def _selective_args(lead, x, dt_raw, dt_bias, A, B, C, D, z, y_dtype, state_dtype) -> SelectiveDesc:
    """The arguments that the calls of the selective scan share, checked, as its descriptor."""
    import torch
    f32, ch, dtype = torch.float32, x.shape[-1], x.dtype
    G, N = B.shape[-2:]
    bc = lead + (G, N)
    _check(dt_raw, lead + (ch,), "dt_raw", dtype)
    _check(B, bc, "B", dtype)
    _check(C, bc, "C", dtype)
    _check(A, (ch, N), "A", f32)
    _check(dt_bias, (ch,), "dt_bias", f32)
    _check(D, (ch,), "D", f32)
    zs = ch if z is None else _row_stride(z, "z", lead, ch, dtype)
    return SelectiveDesc(lead[0], lead[1] if len(lead) > 1 else 1, ch, N, G, zs, _code(dtype), _code(y_dtype),
                         _code(state_dtype))


def selective_scan_fwd(x, dt_raw, dt_bias, A, B, C, D, z=None, init_state=None, *, y=None, final_state=None,
                       y_dtype=None, state_dtype=None, want_final_state=True, pad_left=None, workspace=None,
                       stream=None):
    """Selective scan (a decay per channel and state): x, dt_raw [b,L,D], dt_bias and D [D] fp32 (may be None),
    A [D,N] fp32, B, C [b,L,G,N], gate z [b,L,D] (columns of wider rows are taken; may be None), states [b,D,N].
    ``pad_left`` (int32 [b], CUDA): leading tokens that are absent; y is 0 there.

    Returns (y, final_state) (None without ``want_final_state``); state_dtype defaults to init_state's dtype,
    else fp32.
    """
    import torch
    b, L, ch = x.shape
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    if state_dtype is None:
        state_dtype = (init_state.dtype if init_state is not None else
                       final_state.dtype if final_state is not None else torch.float32)
    desc = _selective_args((b, L), x, dt_raw, dt_bias, A, B, C, D, z, y_dtype, state_dtype)
    states = (b, ch, B.shape[-1])
    _check(init_state, states, "init_state", state_dtype)
    _check(final_state, states, "final_state", state_dtype)
    _check(y, (b, L, ch), "y", y_dtype)
    _check(pad_left, (b,), "pad_left", torch.int32)
    dense, rows = (x, dt_raw, dt_bias, A, B, C, D, init_state, pad_left, y, final_state, workspace), (z,)
    device = _one_device(dense, rows)
    need = ssd_selective_scan_workspace_size(desc)

    def call(handle):
        out = x.new_empty((b, L, ch), dtype=y_dtype) if y is None else y
        final = final_state
        if final is None and want_final_state:
            final = x.new_empty(states, dtype=state_dtype)
        ws, nbytes, keep = _workspace(workspace, need, x)
        st = ssd_selective_scan_fwd(desc, x.data_ptr(), dt_raw.data_ptr(), _ptr(dt_bias), A.data_ptr(), B.data_ptr(),
                                    C.data_ptr(), _ptr(D), _ptr(z), _ptr(init_state), _ptr(pad_left), out.data_ptr(),
                                    _ptr(final), ws, nbytes, handle)
        if st:
            raise SsdError(st, "ssd_selective_scan_fwd")
        return out, final

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def selective_state_update(state, x, dt_raw, dt_bias, A, B, C, D, z=None, *, y=None, y_dtype=None, stream=None):
    """One token of ``selective_scan_fwd``, in place on ``state`` [b,D,N]: x, dt_raw [b,D], B, C [b,G,N],
    z [b,D] (columns of wider rows are taken).  Returns y [b,D]."""
    import torch
    b, ch = x.shape
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    desc = _selective_args((b,), x, dt_raw, dt_bias, A, B, C, D, z, y_dtype, state.dtype)
    _check(state, (b, ch, B.shape[-1]), "state")
    _check(y, (b, ch), "y", y_dtype)
    dense, rows = (state, x, dt_raw, dt_bias, A, B, C, D, y), (z,)
    device = _one_device(dense, rows)

    def call(handle):
        out = x.new_empty((b, ch), dtype=y_dtype) if y is None else y
        st = ssd_selective_state_update(desc, state.data_ptr(), x.data_ptr(), dt_raw.data_ptr(), _ptr(dt_bias),
                                        A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), out.data_ptr(),
                                        handle)
        if st:
            raise SsdError(st, "ssd_selective_state_update")
        return out

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def selective_scan_bwd(x, dt_raw, dt_bias, A, B, C, D, dy, z=None, init_state=None, dfinal_state=None, *,
                       grad_dtype=None, state_dtype=None, want_dinit=True, workspace=None, stream=None):
    """Backward pass of ``selective_scan_fwd`` (without padding): gradients of sum<dy, y> + <dfinal_state,
    final_state>; dy [b,L,D] in x's dtype.

    Returns a dict: dx, ddt_raw, dz [b,L,D], dB, dC [b,L,G,N] (``grad_dtype``, default x's dtype), dA [D,N],
    ddt_bias, dD [D] (fp32), dinit_state [b,D,N] (None without ``want_dinit``); dz, ddt_bias and dD are None
    where z, dt_bias and D are.
    """
    import torch
    b, L, ch = x.shape
    if grad_dtype is None:
        grad_dtype = x.dtype
    if state_dtype is None:
        src = init_state if init_state is not None else dfinal_state
        state_dtype = src.dtype if src is not None else torch.float32
    desc = _selective_args((b, L), x, dt_raw, dt_bias, A, B, C, D, z, grad_dtype, state_dtype)
    states = (b, ch, B.shape[-1])
    _check(dy, (b, L, ch), "dy", x.dtype)
    _check(init_state, states, "init_state", state_dtype)
    _check(dfinal_state, states, "dfinal_state", state_dtype)
    dense, rows = (x, dt_raw, dt_bias, A, B, C, D, dy, init_state, dfinal_state, workspace), (z,)
    device = _one_device(dense, rows)
    need = ssd_selective_scan_bwd_workspace_size(desc)

    def call(handle):
        f32, empty = torch.float32, x.new_empty
        out = {"dx": empty((b, L, ch), dtype=grad_dtype),
               "ddt_raw": empty((b, L, ch), dtype=grad_dtype),
               "dz": empty((b, L, ch), dtype=grad_dtype) if z is not None else None,
               "dB": empty(B.shape, dtype=grad_dtype), "dC": empty(B.shape, dtype=grad_dtype),
               "dA": empty(A.shape, dtype=f32),
               "ddt_bias": empty(ch, dtype=f32) if dt_bias is not None else None,
               "dD": empty(ch, dtype=f32) if D is not None else None,
               "dinit_state": empty(states, dtype=state_dtype) if want_dinit else None}
        ws, nbytes, keep = _workspace(workspace, need, x)
        st = ssd_selective_scan_bwd(desc, x.data_ptr(), dt_raw.data_ptr(), _ptr(dt_bias), A.data_ptr(), B.data_ptr(),
                                    C.data_ptr(), _ptr(D), _ptr(z), _ptr(init_state), dy.data_ptr(),
                                    _ptr(dfinal_state), out["dx"].data_ptr(), out["ddt_raw"].data_ptr(),
                                    _ptr(out["ddt_bias"]), out["dA"].data_ptr(), out["dB"].data_ptr(),
                                    out["dC"].data_ptr(), _ptr(out["dD"]), _ptr(out["dz"]), _ptr(out["dinit_state"]),
                                    ws, nbytes, handle)
        if st:
            raise SsdError(st, "ssd_selective_scan_bwd")
        return out

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def _norm_desc(x, z, weight, bias, ngroups, eps, center, gate_first, activation, io_dtype, y_dtype) -> GroupNormDesc:
    *lead, C = x.shape
    act, zs, rows = _silu_flag(activation), C, 1
    for n in lead:
        rows *= n
    if weight is not None or bias is not None:
        import torch
        _check(weight, (C,), "weight", torch.float32)
        _check(bias, (C,), "bias", torch.float32)
    if z is not None:
        if act:
            raise ValueError("activation: the gate z has its own SiLU")
        zs = _row_stride(z, "z", tuple(lead), C, io_dtype)
        act = SSD_NORM_GATE_BEFORE if gate_first else SSD_NORM_GATE_AFTER
    return GroupNormDesc(rows, C, ngroups, zs, eps, _code(x.dtype), _code(io_dtype), _code(y_dtype),
                         1 if center else 0, act)


def group_norm_fwd(x, weight=None, bias=None, z=None, *, ngroups=1, eps=1e-5, center=False, gate_first=True,
                   activation=None, y=None, y_dtype=None, stream=None):
    """Group normalisation of x [..., C] over the C / ngroups channels of a group in each row (the root mean
    square form; ``center`` subtracts the mean first), weight and bias [C] fp32 (may be None).

    With a gate z [..., C] (columns of wider rows are taken) x silu(z) is normalised, without ``gate_first``
    the result is multiplied by silu(z); without one ``activation`` may be "silu".  Returns y [..., C]
    (``y_dtype``, default z's dtype, else x's).
    """
    io_dtype = z.dtype if z is not None else x.dtype
    if y_dtype is None:
        y_dtype = y.dtype if y is not None else io_dtype
    desc = _norm_desc(x, z, weight, bias, ngroups, eps, center, gate_first, activation, io_dtype, y_dtype)
    _check(y, x.shape, "y", y_dtype)
    dense, rows = (x, weight, bias, y), (z,)
    device = _one_device(dense, rows)

    def call(handle):
        out = x.new_empty(x.shape, dtype=y_dtype) if y is None else y
        st = ssd_group_norm_fwd(desc, x.data_ptr(), _ptr(z), _ptr(weight), _ptr(bias), out.data_ptr(), handle)
        if st:
            raise SsdError(st, "ssd_group_norm_fwd")
        return out

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))


def group_norm_bwd(x, weight, bias, dy, z=None, *, ngroups=1, eps=1e-5, center=False, gate_first=True,
                   activation=None, grad_dtype=None, workspace=None, stream=None):
    """Backward pass of ``group_norm_fwd``; dy [..., C] (and z) in one dtype.  Returns a dict: dx, dz [..., C]
    (``grad_dtype``, default dy's dtype), dweight, dbias [C] fp32; None where z, weight, bias are."""
    import torch
    if grad_dtype is None:
        grad_dtype = dy.dtype
    desc = _norm_desc(x, z, weight, bias, ngroups, eps, center, gate_first, activation, dy.dtype, grad_dtype)
    _check(dy, x.shape, "dy")
    dense, rows = (x, weight, bias, dy, workspace), (z,)
    device = _one_device(dense, rows)
    need = ssd_group_norm_bwd_workspace_size(desc)

    def call(handle):
        f32, empty, C = torch.float32, x.new_empty, x.shape[-1]
        out = {"dx": empty(x.shape, dtype=grad_dtype),
               "dz": empty(x.shape, dtype=grad_dtype) if z is not None else None,
               "dweight": empty(C, dtype=f32) if weight is not None else None,
               "dbias": empty(C, dtype=f32) if bias is not None else None}
        ws, nbytes, keep = _workspace(workspace, need, x)
        st = ssd_group_norm_bwd(desc, x.data_ptr(), _ptr(z), _ptr(weight), _ptr(bias), dy.data_ptr(),
                                out["dx"].data_ptr(), _ptr(out["dz"]), _ptr(out["dweight"]), _ptr(out["dbias"]), ws,
                                nbytes, handle)
        if st:
            raise SsdError(st, "ssd_group_norm_bwd")
        return out

    return _launch_on(device, stream, call, () if stream is None else (*dense, *rows))
