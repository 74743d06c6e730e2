"""ctypes binding of ``libkda.so`` (C ABI in ``include/kda.h``).

Argument marshalling only: tensors are checked for dtype, device, shape and
contiguity and turned into raw pointers; every step of the computation runs
in the library's CUDA kernels. There is no fallback: if the library is
missing or fails to load, these functions raise. (``_native.so``, where it is
built, does the same for some plain calls in less host time.)
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

from . import build as _build

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3
KDA_ERR_GATE_RANGE = 4
KDA_ERR_BAD_SEQLENS = 5
KDA_ERR_TIMEOUT = 6
KDA_ERR_VALUE_RANGE = 7
KDA_ERR_SCRATCH_TOO_SMALL = 8
KDA_ERR_BOUNDS = 9
KDA_ERR_BAD_SLOT = 10
KDA_DEBUG_WITHHOLD_READY = 1
KDA_DEBUG_WY_PRODUCER = 2  # the producer CTAs form the WY product
KDA_DEBUG_WY_CONSUMER = 4  # the consumer CTAs form it
KDA_DEBUG_SPLIT_COLUMNS = 8  # a chain's value columns over two consumer CTAs
KDA_DEBUG_WHOLE_COLUMNS = 16  # one consumer CTA per chain's columns

HEAD_DIM = 128
EXPORTED = ("kda_chunk_fwd", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd_static_scratch",
            "kda_chunk_fwd_debug", "kda_chunk_fwd_raw_gates", "kda_chunk_fwd_gated_norm", "kda_chunk_fwd_split",
            "kda_chunk_fwd_split_plan", "kda_chunk_fwd_split_workspace_size", "kda_chunk_fwd_host", "kda_chunk_fwd_plan",
            "kda_chunk_fwd_host_buffer_size", "kda_decode_fwd",
            "kda_chunk_fwd_launches", "kda_linear_chunk_fwd", "kda_linear_chunk_fwd_debug", "kda_linear_chunk_fwd_workspace_size",
            "kda_linear_decode_fwd", "kda_state_store", "kda_state_load", "kda_add_rms_norm",
            "kda_gated_delta_chunk_fwd", "kda_gated_delta_chunk_fwd_debug", "kda_gated_delta_chunk_fwd_workspace_size", "kda_gated_delta_decode_fwd",
            "kda_gated_rms_norm", "kda_scaled_matmul", "kda_scaled_matmul_debug",
            "kda_status_string", "kda_version")
DECODE_MAX_TOKENS = 64
NORM_MAX_WIDTH = 32768

_lock = threading.Lock()
_lib = None
_native = None  # the plain calls as native code, once the library is loaded and if they are built


class KdaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} (code {code})")
        self.code = code


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load ``libkda.so``; raises ``OSError`` if it is absent (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"{path} not found: build it with kda_chunked_prefill_gb300.build.build()")
            _build.build()
        lib = ctypes.CDLL(path)
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        lib.kda_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, f32, f32,
                                      vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.kda_chunk_fwd.restype = ctypes.c_int
        lib.kda_chunk_fwd_debug.argtypes = lib.kda_chunk_fwd.argtypes + [ctypes.c_uint32]
        lib.kda_chunk_fwd_debug.restype = ctypes.c_int
        lib.kda_chunk_fwd_raw_gates.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, f32, f32,
                                                vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.kda_chunk_fwd_raw_gates.restype = ctypes.c_int
        lib.kda_chunk_fwd_gated_norm.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, f32, f32,
                                                 vp, vp, f32, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.kda_chunk_fwd_gated_norm.restype = ctypes.c_int
        lib.kda_chunk_fwd_split.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, f32, f32, i32,
                                            vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.kda_chunk_fwd_split.restype = ctypes.c_int
        lib.kda_chunk_fwd_split_plan.argtypes = [vp, i32, i32, i32]
        lib.kda_chunk_fwd_split_plan.restype = ctypes.c_int32
        lib.kda_chunk_fwd_plan.argtypes = [i32, i64, i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                           ctypes.POINTER(i32)]
        lib.kda_chunk_fwd_plan.restype = ctypes.c_int
        lib.kda_chunk_fwd_split_workspace_size.argtypes = [vp, i32, i32, i32]
        lib.kda_chunk_fwd_split_workspace_size.restype = ctypes.c_size_t
        lib.kda_chunk_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, f32, f32, vp, vp, vp,
                                           vp, ctypes.c_size_t, i32, vp, vp, vp]
        lib.kda_chunk_fwd_host.restype = ctypes.c_int
        lib.kda_chunk_fwd_host_buffer_size.argtypes = [vp, i32, i32, i32, i32, i32]
        lib.kda_chunk_fwd_host_buffer_size.restype = ctypes.c_size_t
        lib.kda_decode_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, f32, f32, vp, vp, vp, vp]
        lib.kda_decode_fwd.restype = ctypes.c_int
        lib.kda_linear_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i64, i64, i64, i32, vp,
                                             f32, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.kda_linear_chunk_fwd.restype = ctypes.c_int
        lib.kda_linear_chunk_fwd_debug.argtypes = lib.kda_linear_chunk_fwd.argtypes + [i32, i32]
        lib.kda_linear_chunk_fwd_debug.restype = ctypes.c_int
        lib.kda_linear_chunk_fwd_workspace_size.argtypes = [i32, i64, i32]
        lib.kda_linear_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_linear_decode_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i64, i64, i32, vp, f32,
                                              vp, vp, vp, vp]
        lib.kda_linear_decode_fwd.restype = ctypes.c_int
        lib.kda_state_store.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        lib.kda_state_store.restype = ctypes.c_int
        lib.kda_state_load.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
        lib.kda_state_load.restype = ctypes.c_int
        lib.kda_add_rms_norm.argtypes = [vp, vp, vp, i64, i32, f32, i32, vp, vp, vp, vp]
        lib.kda_add_rms_norm.restype = ctypes.c_int
        lib.kda_gated_delta_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i64, i64, i64, vp,
                                                  f32, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.kda_gated_delta_chunk_fwd.restype = ctypes.c_int
        lib.kda_gated_delta_chunk_fwd_debug.argtypes = lib.kda_gated_delta_chunk_fwd.argtypes + [i32]
        lib.kda_gated_delta_chunk_fwd_debug.restype = ctypes.c_int
        lib.kda_gated_delta_chunk_fwd_workspace_size.argtypes = [i32, i64, i32]
        lib.kda_gated_delta_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_gated_delta_decode_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, i64, i64, vp, f32,
                                                   vp, vp, vp, vp]
        lib.kda_gated_delta_decode_fwd.restype = ctypes.c_int
        lib.kda_gated_rms_norm.argtypes = [vp, vp, i64, vp, i64, i32, i32, f32, i32, i32, vp, vp, vp]
        lib.kda_gated_rms_norm.restype = ctypes.c_int
        lib.kda_scaled_matmul.argtypes = [vp, vp, i32, vp, vp, i64, i32, i32, vp, vp, vp]
        lib.kda_scaled_matmul.restype = ctypes.c_int
        lib.kda_scaled_matmul_debug.argtypes = lib.kda_scaled_matmul.argtypes + [i32]
        lib.kda_scaled_matmul_debug.restype = ctypes.c_int
        lib.kda_chunk_fwd_workspace_size.argtypes = [i32, i32]
        lib.kda_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        lib.kda_chunk_fwd_launches.argtypes = [i32, i64, i32]
        lib.kda_chunk_fwd_launches.restype = i32
        lib.kda_status_string.argtypes = [i32]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_version.argtypes = []
        lib.kda_version.restype = i32
        _load_native(lib)
        _lib = lib
        return lib


def _load_native(lib):
    global _native
    try:
        from . import _native as native
    except ImportError:  # not built: every call takes its general path
        return
    if getattr(native, "torch_version", None) != torch.__version__:  # (built against another torch: it would misread tensors)
        return
    native.set_entry(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.kda_gated_rms_norm, lib.kda_scaled_matmul, lib.kda_gated_delta_decode_fwd, lib.kda_gated_delta_chunk_fwd,
        lib.kda_gated_delta_chunk_fwd_workspace_size)))
    _native = native


def _done(result, what):
    """What a native call returned: an error code, or the outputs."""
    if type(result) is int:
        raise KdaError(result, what)
    return result


def status_string(code: int) -> str:
    return load_library().kda_status_string(int(code)).decode()


def version() -> int:
    return int(load_library().kda_version())


def workspace_size(num_seqs: int, num_heads: int) -> int:
    """Workspace bytes ``kda_chunk_fwd`` needs on the current CUDA device."""
    return int(load_library().kda_chunk_fwd_workspace_size(int(num_seqs), int(num_heads)))


_ws_cache = {}


def workspace_for(num_seqs: int, num_heads: int, device) -> torch.Tensor:
    """A cached workspace buffer for calls on ``device``'s current stream.
    Calls that may overlap on the GPU need buffers of their own."""
    need = workspace_size(num_seqs, num_heads)
    key = torch.device(device)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.empty(max(need, 1), dtype=torch.uint8, device=key)
        _ws_cache[key] = buf
    return buf


def chunk_fwd_launches(num_seqs: int, total_tokens: int, num_heads: int) -> int:
    return int(load_library().kda_chunk_fwd_launches(int(num_seqs), int(total_tokens), int(num_heads)))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def kda_chunk_fwd(q, k, v, g, beta, cu_seqlens, initial_state, scale: float, lower_bound: float,
                  o, final_state, status=None, stream=None, workspace=None, debug_flags: int = 0,
                  raw_gates: bool = False, A_log=None, dt_bias=None, norm_gate=None, norm_weight=None,
                  norm_eps: float = 1e-5) -> int:
    """Call the C entry point ``kda_chunk_fwd`` with caller-allocated outputs.

    q, k, v: bf16 [T,H,128]; o: fp32 [T,H,128]; g: fp32 [T,H,128]; beta: fp32 [T,H];
    cu_seqlens: int32 [N+1]; initial_state / final_state: fp32 [N,H,128,128]
    or None; status: int32 [1] or None; workspace: uint8 tensor of at least
    ``workspace_size(N, H)`` bytes (default: a cached per-device buffer). All on
    one CUDA device. ``stream`` is a ``torch.cuda.Stream`` (default: the current
    stream). Raises ``KdaError`` on a host-side error; returns ``KDA_OK`` once
    the work is queued. A nonzero ``debug_flags`` calls ``kda_chunk_fwd_debug``
    (failure-detection testing; see include/kda.h). ``raw_gates=True`` calls
    ``kda_chunk_fwd_raw_gates``: ``g`` and ``beta`` are then the raw gate and
    beta projections, activated inside the kernel with the optional per-head
    ``A_log`` (fp32 [H]) and ``dt_bias`` (fp32 [H,128]). Given ``norm_gate``
    (bf16 [T,H,128]) and ``norm_weight`` (fp32 [128]), ``kda_chunk_fwd_gated_norm``
    writes ``o`` as the gated RMSNorm of the output (``norm_eps`` inside the root).
    """
    T, H, D = q.shape
    N = cu_seqlens.shape[0] - 1
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(q, "q", torch.bfloat16, (T, H, D), dev)
    _check(k, "k", torch.bfloat16, (T, H, D), dev)
    _check(v, "v", torch.bfloat16, (T, H, v.shape[2]), dev)
    _check(g, "g", torch.float32, (T, H, D), dev)
    _check(beta, "beta", torch.float32, (T, H), dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    _check(o, "o", torch.float32, tuple(v.shape), dev)
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (N, H, D, v.shape[2]), dev)
    if final_state is not None:
        _check(final_state, "final_state", torch.float32, (N, H, D, v.shape[2]), dev)
    if status is not None:
        _check(status, "status", torch.int32, (1,), dev)
    if not raw_gates and (A_log is not None or dt_bias is not None):
        raise ValueError("A_log and dt_bias apply only with raw_gates=True")
    if A_log is not None:
        _check(A_log, "A_log", torch.float32, (H,), dev)
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", torch.float32, (H, D), dev)
    norm = norm_gate is not None or norm_weight is not None
    if norm:
        if norm_gate is None or norm_weight is None:
            raise ValueError("norm_gate and norm_weight go together")
        _check(norm_gate, "norm_gate", torch.bfloat16, tuple(v.shape), dev)
        _check(norm_weight, "norm_weight", torch.float32, (v.shape[2],), dev)
        if raw_gates or debug_flags:
            raise ValueError("the gated norm combines with neither raw_gates nor debug_flags")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    if workspace is None:
        workspace = workspace_for(N, H, dev)
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N, T, H, D, v.shape[2],
            _ptr(initial_state), float(scale), float(lower_bound), _ptr(o), _ptr(final_state),
            _ptr(status), _ptr(workspace), workspace.numel(), ctypes.c_void_p(stream.cuda_stream))
    lib = load_library()
    if norm:
        rc = lib.kda_chunk_fwd_gated_norm(*args[:14], _ptr(norm_gate), _ptr(norm_weight), float(norm_eps), *args[14:])
        what = "kda_chunk_fwd_gated_norm"
    elif raw_gates:
        if debug_flags:
            raise ValueError("debug_flags and raw_gates cannot be combined")
        rc = lib.kda_chunk_fwd_raw_gates(*args[:5], _ptr(A_log), _ptr(dt_bias), *args[5:])
        what = "kda_chunk_fwd_raw_gates"
    else:
        rc = lib.kda_chunk_fwd_debug(*args, int(debug_flags)) if debug_flags else lib.kda_chunk_fwd(*args)
        what = "kda_chunk_fwd"
    if rc != KDA_OK:
        raise KdaError(rc, what)
    return rc


def chunk_fwd(q, k, v, g, beta, cu_seqlens, initial_state=None, scale: Optional[float] = None,
              lower_bound: float = -5.0, output_final_state: bool = True, check: bool = False,
              stream=None, raw_gates: bool = False, A_log=None, dt_bias=None, norm_gate=None,
              norm_weight=None, norm_eps: float = 1e-5):
    """Allocate ``o`` (and ``final_state``) and run ``kda_chunk_fwd``.

    Returns ``(o, final_state)``; ``final_state`` is None when not requested.
    With ``check=True`` the device status word is read back (a synchronising
    copy) and a device-detected error raises ``KdaError``. ``raw_gates``,
    ``A_log``, ``dt_bias`` and the gated-norm arguments are passed to
    ``kda_chunk_fwd``.
    """
    T, H, D = q.shape
    N = cu_seqlens.shape[0] - 1
    if scale is None:
        scale = D ** -0.5
    o = torch.empty((T, H, v.shape[2]), dtype=torch.float32, device=q.device)
    fs = (torch.empty((N, H, D, v.shape[2]), dtype=torch.float32, device=q.device)
          if output_final_state else None)
    status = torch.zeros(1, dtype=torch.int32, device=q.device) if check else None
    kda_chunk_fwd(q, k, v, g, beta, cu_seqlens, initial_state, scale, lower_bound, o, fs, status, stream,
                  raw_gates=raw_gates, A_log=A_log, dt_bias=dt_bias, norm_gate=norm_gate,
                  norm_weight=norm_weight, norm_eps=norm_eps)
    if check:
        code = int(status.item())
        if code != KDA_OK:
            raise KdaError(code, "kda_chunk_fwd (device)")
    return o, fs


def _host_cu(cu_seqlens_host):
    cu = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).cpu().contiguous()
    return cu, ctypes.c_void_p(cu.data_ptr())


def split_plan(cu_seqlens_host, num_heads: int, num_sms: int = 0) -> int:
    """Segment length (in 64-token chunks) ``kda_chunk_fwd_split`` would pick
    for these sequence lengths (0: no split). ``num_sms`` 0 = the current device."""
    cu, ptr = _host_cu(cu_seqlens_host)
    return int(load_library().kda_chunk_fwd_split_plan(ptr, cu.numel() - 1, int(num_heads), int(num_sms)))


def chunk_fwd_plan(num_seqs: int, total_tokens: int, num_heads: int, num_sms: int = 0,
                   plain_device_o: bool = True) -> Tuple[int, bool, bool]:
    """``kda_chunk_fwd_plan``: (consumers, whether the consumers form the WY
    product, whether each consumer is two CTAs with half the value columns each)
    for a call of this shape. ``num_sms`` 0 = the current device."""
    c, w, sp = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
    rc = load_library().kda_chunk_fwd_plan(int(num_seqs), int(total_tokens), int(num_heads), int(num_sms),
                                           1 if plain_device_o else 0, ctypes.byref(c), ctypes.byref(w),
                                           ctypes.byref(sp))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_plan")
    return int(c.value), bool(w.value), bool(sp.value)


def split_workspace_size(cu_seqlens_host, num_heads: int, segment_chunks: int = 0) -> int:
    cu, ptr = _host_cu(cu_seqlens_host)
    return int(load_library().kda_chunk_fwd_split_workspace_size(ptr, cu.numel() - 1, int(num_heads),
                                                                  int(segment_chunks)))


def kda_chunk_fwd_split(q, k, v, g, beta, cu_seqlens, cu_seqlens_host, initial_state, scale: float,
                        lower_bound: float, o, final_state, status=None, stream=None, segment_chunks: int = 0,
                        workspace=None) -> int:
    """Call ``kda_chunk_fwd_split`` (the split-sequence scan; see include/kda.h).
    Arguments as ``kda_chunk_fwd`` plus ``cu_seqlens_host`` (the same offsets on
    the host: a CPU tensor, array or list) and ``segment_chunks`` (0: planned).
    ``workspace`` defaults to a fresh uint8 tensor of the needed size."""
    T, H, D = q.shape
    dev = q.device
    cu, cu_ptr = _host_cu(cu_seqlens_host)
    N = cu.numel() - 1
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(q, "q", torch.bfloat16, (T, H, D), dev)
    _check(k, "k", torch.bfloat16, (T, H, D), dev)
    _check(v, "v", torch.bfloat16, (T, H, v.shape[2]), dev)
    _check(g, "g", torch.float32, (T, H, D), dev)
    _check(beta, "beta", torch.float32, (T, H), dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    _check(o, "o", torch.float32, tuple(v.shape), dev)
    for t, name in ((initial_state, "initial_state"), (final_state, "final_state")):
        if t is not None:
            _check(t, name, torch.float32, (N, H, D, v.shape[2]), dev)
    if status is not None:
        _check(status, "status", torch.int32, (1,), dev)
    lib = load_library()
    if workspace is None:
        nbytes = lib.kda_chunk_fwd_split_workspace_size(cu_ptr, N, H, int(segment_chunks))
        if nbytes == 0:
            raise KdaError(KDA_ERR_INVALID_ARG, "kda_chunk_fwd_split_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    rc = lib.kda_chunk_fwd_split(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), cu_ptr, N, T, H,
                                 D, v.shape[2], _ptr(initial_state), float(scale), float(lower_bound),
                                 int(segment_chunks), _ptr(o), _ptr(final_state), _ptr(status), _ptr(workspace),
                                 workspace.numel(), ctypes.c_void_p(stream.cuda_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_split")
    return rc


def chunk_fwd_split(q, k, v, g, beta, cu_seqlens, cu_seqlens_host=None, initial_state=None,
                    scale: Optional[float] = None, lower_bound: float = -5.0, output_final_state: bool = True,
                    check: bool = False, stream=None, segment_chunks: int = 0):
    """Allocate ``o`` (and ``final_state``) and run ``kda_chunk_fwd_split``.
    ``cu_seqlens_host`` defaults to a copy of ``cu_seqlens`` (a synchronising
    device-to-host read)."""
    T, H, D = q.shape
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.cpu()
    N = cu_seqlens.shape[0] - 1
    if scale is None:
        scale = D ** -0.5
    o = torch.empty((T, H, v.shape[2]), dtype=torch.float32, device=q.device)
    fs = (torch.empty((N, H, D, v.shape[2]), dtype=torch.float32, device=q.device)
          if output_final_state else None)
    status = torch.zeros(1, dtype=torch.int32, device=q.device) if check else None
    kda_chunk_fwd_split(q, k, v, g, beta, cu_seqlens, cu_seqlens_host, initial_state, scale, lower_bound, o, fs,
                        status, stream, segment_chunks=segment_chunks)
    if check:
        code = int(status.item())
        if code != KDA_OK:
            raise KdaError(code, "kda_chunk_fwd_split (device)")
    return o, fs


def host_buffer_size(cu_seqlens_host, num_heads: int, with_initial_state: bool, with_final_state: bool = True,
                     groups: int = 0) -> int:
    cu, ptr = _host_cu(cu_seqlens_host)
    return int(load_library().kda_chunk_fwd_host_buffer_size(ptr, cu.numel() - 1, int(num_heads),
                                                              int(bool(with_initial_state)),
                                                              int(bool(with_final_state)), int(groups)))


def kda_chunk_fwd_host(q, k, v, g, beta, cu_seqlens_host, initial_state, scale: float, lower_bound: float, o,
                       final_state, device_buffer, status=None, groups: int = 0, stream=None, h2d_stream=None,
                       d2h_stream=None) -> int:
    """Call ``kda_chunk_fwd_host``: q .. beta, initial_state, o and final_state
    are CPU tensors (layouts as ``kda_chunk_fwd``), ``device_buffer`` a CUDA uint8
    tensor of ``host_buffer_size(...)`` bytes. With ``groups=0`` and page-locked
    tensors (``pin_memory()``) the kernel reads and writes them in place; else
    the copies of groups of sequences overlap the computation. The results are
    in ``o`` / ``final_state`` once ``stream`` is synchronised."""
    T, H, D = q.shape
    cu, cu_ptr = _host_cu(cu_seqlens_host)
    N = cu.numel() - 1
    cpu = torch.device("cpu")
    _check(q, "q", torch.bfloat16, (T, H, D), cpu)
    _check(k, "k", torch.bfloat16, (T, H, D), cpu)
    _check(v, "v", torch.bfloat16, (T, H, v.shape[2]), cpu)
    _check(g, "g", torch.float32, (T, H, D), cpu)
    _check(beta, "beta", torch.float32, (T, H), cpu)
    _check(o, "o", torch.float32, tuple(v.shape), cpu)
    for t, name in ((initial_state, "initial_state"), (final_state, "final_state")):
        if t is not None:
            _check(t, name, torch.float32, (N, H, D, v.shape[2]), cpu)
    dev = device_buffer.device
    if dev.type != "cuda" or device_buffer.dtype != torch.uint8 or not device_buffer.is_contiguous():
        raise ValueError("device_buffer must be a contiguous CUDA uint8 tensor")
    if status is not None:
        _check(status, "status", torch.int32, (1,), dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    sp = lambda s_: None if s_ is None else ctypes.c_void_p(s_.cuda_stream)
    rc = load_library().kda_chunk_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), cu_ptr, N, T, H, D,
                                           v.shape[2], _ptr(initial_state), float(scale), float(lower_bound), _ptr(o),
                                           _ptr(final_state), _ptr(status), _ptr(device_buffer), device_buffer.numel(),
                                           int(groups), sp(stream), sp(h2d_stream), sp(d2h_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_host")
    return rc


def kda_decode_fwd(q, k, v, g, beta, num_seqs: int, initial_state, scale: float, lower_bound: float,
                   o, final_state, status=None, stream=None) -> int:
    """Call the C entry point ``kda_decode_fwd`` with caller-allocated outputs.

    q, k, v: bf16 [N*Tn, H, 128] (sequence n's Tn tokens at rows n*Tn..); g:
    fp32 [N*Tn, H, 128]; beta: fp32 [N*Tn, H]; o: fp32 [N*Tn, H, 128];
    initial_state / final_state: fp32 [N, H, 128, 128] or None (they may be
    the same tensor). Raises ``KdaError`` on a host-side error.
    """
    T, H, D = q.shape
    N = int(num_seqs)
    if N < 0 or (N == 0 and T != 0) or (N > 0 and T % N != 0):
        raise ValueError("q must hold the same number of tokens for every sequence")
    Tn = T // N if N > 0 else 0
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    _check(q, "q", torch.bfloat16, (T, H, D), dev)
    _check(k, "k", torch.bfloat16, (T, H, D), dev)
    _check(v, "v", torch.bfloat16, (T, H, v.shape[2]), dev)
    _check(g, "g", torch.float32, (T, H, D), dev)
    _check(beta, "beta", torch.float32, (T, H), dev)
    _check(o, "o", torch.float32, tuple(v.shape), dev)
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (N, H, D, v.shape[2]), dev)
    if final_state is not None:
        _check(final_state, "final_state", torch.float32, (N, H, D, v.shape[2]), dev)
    if status is not None:
        _check(status, "status", torch.int32, (1,), dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    rc = load_library().kda_decode_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), N, Tn, H, D, v.shape[2], _ptr(initial_state),
        float(scale), float(lower_bound), _ptr(o), _ptr(final_state), _ptr(status), ctypes.c_void_p(stream.cuda_stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_fwd")
    return rc


def decode_fwd(q, k, v, g, beta, num_seqs: int, state=None, scale: Optional[float] = None,
               lower_bound: float = -5.0, in_place: bool = False, check: bool = False, stream=None):
    """Run ``kda_decode_fwd``; returns ``(o, final_state)``. With ``in_place``
    the given ``state`` tensor is updated and returned as ``final_state``."""
    T, H, D = q.shape
    N = int(num_seqs)
    if scale is None:
        scale = D ** -0.5
    o = torch.empty((T, H, v.shape[2]), dtype=torch.float32, device=q.device)
    if in_place:
        if state is None:
            raise ValueError("in_place needs a state tensor")
        fs = state
    else:
        fs = torch.empty((N, H, D, v.shape[2]), dtype=torch.float32, device=q.device)
    status = torch.zeros(1, dtype=torch.int32, device=q.device) if check else None
    kda_decode_fwd(q, k, v, g, beta, N, state, scale, lower_bound, o, fs, status, stream)
    if check:
        code = int(status.item())
        if code != KDA_OK:
            raise KdaError(code, "kda_decode_fwd (device)")
    return o, fs


# ------------------------------------------------------------------ what the calls below share
# A call's host time counts where its kernel takes a few microseconds: each tensor is checked by one expression (the detailed
# message is made only when it fails), the current stream is read as a handle, and the device is switched only if it has to be.
_BF16, _F32, _I32, _I8, _F8, _U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.float8_e4m3fn, torch.uint8)
# (None on a torch without CUDA, which can import this module and make no call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _need(t, name, dtype, shape, index):
    """``t`` is a contiguous tensor of this dtype and shape on CUDA device ``index``."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _check(t, name, dtype, shape, torch.device("cuda", index))


def _device_of(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("inputs must be CUDA tensors")
    return index


def _call(f, what, index, args, stream):
    """Call a C entry point whose last argument is the stream, on device ``index``."""
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = f(*args, handle)
    if rc != KDA_OK:
        raise KdaError(rc, what)
    return rc


def _on(stream):
    """Where a call's own tensors are allocated: on its stream."""
    return _here if stream is None else torch.cuda.stream(stream)


_here = contextlib.nullcontext()


def _raise_device(status, stream, what):
    if stream is not None:
        stream.synchronize()
    code = int(status.item())
    if code != KDA_OK:
        raise KdaError(code, f"{what} (device)")


def _status(check, device):
    return torch.empty(1, dtype=_I32, device=device) if check else None


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ linear attention with one decay per head
def _heads_view(t, name, tokens, index):
    """Check a [T, heads, 128] bf16 tensor whose tokens may be strided (a slice
    of a wider projection); returns its token stride in elements."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != tokens:
        raise ValueError(f"{name} must have shape ({tokens}, heads, head_dim), got {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on CUDA device {index}, got {t.device}")
    width = shape[1] * shape[2]
    if tokens == 0 or t.is_contiguous():
        return width
    st, sh, sd = t.stride()
    if sd != 1 or (sh != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must hold its heads and channels contiguously within a token")
    if tokens == 1:
        return width
    if st < width or st % 8:
        raise ValueError(f"{name}'s tokens must not overlap and lie a multiple of 8 elements apart")
    return st


def _linear_args(q, k, v, g, o, initial_state, final_state, num_seqs, status):
    """The checks kda_linear_chunk_fwd and kda_linear_decode_fwd share."""
    index = _device_of(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must have shape (tokens, heads, head_dim)")
    T, Hk, D = q.shape
    H, V = v.shape[1], v.shape[2]
    qs, ks, vs = _heads_view(q, "q", T, index), _heads_view(k, "k", T, index), _heads_view(v, "v", T, index)
    if k.shape != q.shape:
        raise ValueError(f"k must have q's shape {tuple(q.shape)}, got {tuple(k.shape)}")
    if Hk < 1 or H % Hk:
        raise ValueError(f"the number of value heads ({H}) must be a multiple of the query/key heads ({Hk})")
    per_token = g.dim() == 2
    _need(g, "g", _F32, (T, H) if per_token else (H,), index)
    _need(o, "o", _BF16, (T, H, V), index)
    if initial_state is not None:
        _need(initial_state, "initial_state", _F32, (num_seqs, H, D, V), index)
    if final_state is not None:
        _need(final_state, "final_state", _F32, (num_seqs, H, D, V), index)
    if status is not None:
        _need(status, "status", _I32, (1,), index)
    return index, T, H, Hk, D, V, qs, ks, vs, int(per_token)


def linear_workspace_size(num_seqs: int, total_tokens: int, num_heads: int) -> int:
    """Workspace bytes ``kda_linear_chunk_fwd`` needs on the current CUDA device (0: none)."""
    return int(load_library().kda_linear_chunk_fwd_workspace_size(int(num_seqs), int(total_tokens), int(num_heads)))


def kda_linear_chunk_fwd(q, k, v, g, cu_seqlens, initial_state, scale: float, o, final_state, status=None, stream=None,
                         workspace=None, withhold: Optional[Tuple[int, int]] = None) -> int:
    """Call the C entry point ``kda_linear_chunk_fwd`` with caller-allocated outputs.

    q, k: bf16 [T,Hk,128]; v: bf16 [T,H,128], H a multiple of Hk (tokens may be
    strided); g: fp32 log decay [T,H], or [H] for one decay per head; cu_seqlens:
    int32 [N+1]; initial_state / final_state: fp32 [N,H,128,128] or None (may be
    the same tensor); o: bf16 [T,H,128]; status: int32 [1] or None; workspace:
    uint8 tensor of ``linear_workspace_size(N, T, H)`` bytes (default: a new one
    from torch's allocator for the call's stream). All on one CUDA device.
    ``withhold`` calls ``kda_linear_chunk_fwd_debug`` with these two numbers.
    Raises ``KdaError`` on a host-side error; returns ``KDA_OK`` once queued.
    """
    N = cu_seqlens.shape[0] - 1
    index, T, H, Hk, D, V, qs, ks, vs, per_token = _linear_args(q, k, v, g, o, initial_state, final_state, N, status)
    _need(cu_seqlens, "cu_seqlens", _I32, (N + 1,), index)
    lib = load_library()
    if workspace is None:
        with torch.cuda.device(index) if _current_device() != index else _here:
            need = lib.kda_linear_chunk_fwd_workspace_size(N, T, H)
        if need:
            with _on(stream):
                workspace = torch.empty(need, dtype=_U8, device=q.device)
    elif workspace.get_device() != index or workspace.dtype is not _U8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), cu_seqlens.data_ptr(), N, T, H, Hk, D, V, qs, ks,
            vs, per_token, _p(initial_state), scale, o.data_ptr(), _p(final_state), _p(status), _p(workspace),
            0 if workspace is None else workspace.numel())
    if withhold is not None:
        debug = lib.kda_linear_chunk_fwd_debug
        return _call(lambda *a: debug(*a, *withhold), "kda_linear_chunk_fwd_debug", index, args, stream)
    return _call(lib.kda_linear_chunk_fwd, "kda_linear_chunk_fwd", index, args, stream)


def linear_chunk_fwd(q, k, v, g, cu_seqlens, initial_state=None, scale: Optional[float] = None,
                     output_final_state: bool = True, check: bool = False, stream=None):
    """Allocate ``o`` (and ``final_state``) and run ``kda_linear_chunk_fwd``.

    Returns ``(o, final_state)``; ``final_state`` is None when not requested. With
    ``check=True`` the device status word is read back (a synchronising copy)
    and a device-detected error raises ``KdaError``. Rows of ``o`` behind the last
    sequence are not written.
    """
    dev, shape = q.device, v.shape
    if scale is None:
        scale = q.shape[2] ** -0.5
    with _on(stream):
        o = torch.empty(shape, dtype=_BF16, device=dev)
        fs = (torch.empty((cu_seqlens.shape[0] - 1, shape[1], q.shape[2], shape[2]), dtype=_F32, device=dev)
              if output_final_state else None)
        status = _status(check, dev)
    kda_linear_chunk_fwd(q, k, v, g, cu_seqlens, initial_state, scale, o, fs, status, stream)
    if check:
        _raise_device(status, stream, "kda_linear_chunk_fwd")
    return o, fs


def kda_linear_decode_fwd(q, k, v, g, num_seqs: int, initial_state, scale: float, o, final_state, status=None,
                          stream=None) -> int:
    """Call the C entry point ``kda_linear_decode_fwd`` with caller-allocated
    outputs: sequence n's tokens are rows n*Tn .. n*Tn+Tn-1 of q, k, v, g and o;
    tensors as in ``kda_linear_chunk_fwd``."""
    N = int(num_seqs)
    T = q.shape[0]
    if N < 0 or (N == 0 and T != 0) or (N > 0 and T % N != 0):
        raise ValueError("q must hold the same number of tokens for every sequence")
    index, T, H, Hk, D, V, qs, ks, vs, per_token = _linear_args(q, k, v, g, o, initial_state, final_state, N, status)
    return _call(load_library().kda_linear_decode_fwd, "kda_linear_decode_fwd", index,
                 (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), N, T // N if N else 0, H, Hk, D, V, qs, ks, vs,
                  per_token, _p(initial_state), scale, o.data_ptr(), _p(final_state), _p(status)), stream)


def linear_decode_fwd(q, k, v, g, num_seqs: int, state=None, scale: Optional[float] = None, in_place: bool = False,
                      check: bool = False, stream=None):
    """Run ``kda_linear_decode_fwd``; returns ``(o, final_state)``. With
    ``in_place`` the given ``state`` tensor is updated and returned as ``final_state``."""
    dev, shape = q.device, v.shape
    if scale is None:
        scale = q.shape[2] ** -0.5
    if in_place and state is None:
        raise ValueError("in_place needs a state tensor")
    with _on(stream):
        o = torch.empty(shape, dtype=_BF16, device=dev)
        fs = state if in_place else torch.empty((int(num_seqs), shape[1], q.shape[2], shape[2]), dtype=_F32, device=dev)
        status = _status(check, dev)
    kda_linear_decode_fwd(q, k, v, g, num_seqs, state, scale, o, fs, status, stream)
    if check:
        _raise_device(status, stream, "kda_linear_decode_fwd")
    return o, fs


# ------------------------------------------------------------------ the int8 cache of states
def _cache_args(state, slots, codes, scales, status):
    index = _device_of(state)
    shape = state.shape
    if len(shape) != 4:
        raise ValueError("state must have shape (rows, heads, 128, 128)")
    M, H, K, V = shape
    S = codes.shape[0]
    _need(state, "state", _F32, shape, index)
    _need(slots, "slots", _I32, (M,), index)
    _need(codes, "codes", _I8, (S, H, K, V), index)
    _need(scales, "scales", _F32, (S, H, K), index)
    if status is not None:
        _need(status, "status", _I32, (1,), index)
    return index, M, H, K, V, S


def kda_state_store(state, slots, codes, scales, status=None, stream=None) -> int:
    """Call the C entry point ``kda_state_store``: quantise state (fp32
    [M,H,128,128]) into the slots (int32 [M], -1: none) of the cache codes (int8
    [S,H,128,128]) and scales (fp32 [S,H,128])."""
    index, M, H, K, V, S = _cache_args(state, slots, codes, scales, status)
    return _call(load_library().kda_state_store, "kda_state_store", index,
                 (state.data_ptr(), slots.data_ptr(), M, H, K, V, S, codes.data_ptr(), scales.data_ptr(), _p(status)), stream)


def kda_state_load(codes, scales, slots, state, status=None, stream=None) -> int:
    """Call the C entry point ``kda_state_load``: read the slots of the cache
    back into ``state`` (a row with slot -1 becomes zeros)."""
    index, M, H, K, V, S = _cache_args(state, slots, codes, scales, status)
    return _call(load_library().kda_state_load, "kda_state_load", index,
                 (codes.data_ptr(), scales.data_ptr(), slots.data_ptr(), M, H, K, V, S, state.data_ptr(), _p(status)), stream)


def state_store(state, slots, codes, scales, check: bool = False, stream=None) -> None:
    """Run ``kda_state_store``; with ``check`` a bad slot raises ``KdaError``."""
    with _on(stream):
        status = _status(check, state.device)
    kda_state_store(state, slots, codes, scales, status, stream)
    if check:
        _raise_device(status, stream, "kda_state_store")


def state_load(codes, scales, slots, check: bool = False, stream=None):
    """Allocate the states fp32 [M,H,128,128] and run ``kda_state_load``."""
    dev = codes.device
    with _on(stream):
        state = torch.empty((slots.shape[0], *codes.shape[1:]), dtype=_F32, device=dev)
        status = _status(check, dev)
    kda_state_load(codes, scales, slots, state, status, stream)
    if check:
        _raise_device(status, stream, "kda_state_load")
    return state


# ------------------------------------------------------------------ residual addition, RMS norm, e4m3 output
def kda_add_rms_norm(x, residual, weight, eps: float, residual_out, y, y_scale, stream=None) -> int:
    """Call the C entry point ``kda_add_rms_norm``: x bf16 [..., d]; residual and
    residual_out (may be the same tensor) bf16 or fp32 like x; weight fp32 [d];
    y float8_e4m3fn like x; y_scale fp32 [...]."""
    index, shape = _device_of(x), x.shape
    if len(shape) < 1:
        raise ValueError("x must have at least one dimension")
    kind = residual.dtype
    if kind is not _BF16 and kind is not _F32:
        raise TypeError(f"residual must be {_BF16} or {_F32}, got {kind}")
    _need(x, "x", _BF16, shape, index)
    _need(residual, "residual", kind, shape, index)
    _need(residual_out, "residual_out", kind, shape, index)
    _need(weight, "weight", _F32, shape[-1:], index)
    _need(y, "y", _F8, shape, index)
    _need(y_scale, "y_scale", _F32, shape[:-1], index)
    return _call(load_library().kda_add_rms_norm, "kda_add_rms_norm", index,
                 (x.data_ptr(), residual.data_ptr(), weight.data_ptr(), y_scale.numel(), shape[-1], eps,
                  1 if kind is _F32 else 0, residual_out.data_ptr(), y.data_ptr(), y_scale.data_ptr()), stream)


def add_rms_norm(x, residual, weight, eps: float = 1e-6, in_place: bool = False, stream=None):
    """Run ``kda_add_rms_norm``; returns ``(y, y_scale, residual_out)``. With
    ``in_place`` the given ``residual`` is updated and returned."""
    dev, shape = x.device, x.shape
    with _on(stream):
        y = torch.empty(shape, dtype=_F8, device=dev)
        y_scale = torch.empty(shape[:-1], dtype=_F32, device=dev)
        res = residual if in_place else torch.empty_like(residual)
    kda_add_rms_norm(x, residual, weight, eps, res, y, y_scale, stream)
    return y, y_scale, res


# ------------------------------------------------------------------ the delta rule with one decay per head
# (Of the calls from here on, those that allocate their outputs do not check them, and the plain ones, without a stream or a check, are
# one native call: a small call's host time is its time. What that does not take, a refused argument among it, goes the general way.)
def _delta_inputs(q, k, v, g, beta, initial_state, num_seqs):
    """The checks of what kda_gated_delta_chunk_fwd and kda_gated_delta_decode_fwd read, and what they pass on."""
    index = _device_of(q)
    shape = q.shape
    if len(shape) != 3 or v.dim() != 3:
        raise ValueError("q, k and v must have shape (tokens, heads, head_dim)")
    T, Hk, D = shape
    _, H, V = v.shape
    qs, ks, vs = _heads_view(q, "q", T, index), _heads_view(k, "k", T, index), _heads_view(v, "v", T, index)
    if k.shape != shape:
        raise ValueError(f"k must have q's shape {tuple(shape)}, got {tuple(k.shape)}")
    if Hk < 1 or H % Hk:
        raise ValueError(f"the number of value heads ({H}) must be a multiple of the query/key heads ({Hk})")
    if g.dim() != 2:
        raise ValueError(f"g must have shape (tokens, heads), got {tuple(g.shape)}")
    _need(g, "g", _F32, (T, H), index)
    _need(beta, "beta", _F32, (T, H), index)
    if initial_state is not None:
        _need(initial_state, "initial_state", _F32, (num_seqs, H, D, V), index)
    return index, T, H, Hk, D, V, qs, ks, vs


def _delta_outputs(inputs, o, final_state, status, num_seqs):
    index, T, H, _, D, V = inputs[:6]
    _need(o, "o", _BF16, (T, H, V), index)
    if final_state is not None:
        _need(final_state, "final_state", _F32, (num_seqs, H, D, V), index)
    if status is not None:
        _need(status, "status", _I32, (1,), index)


def gated_delta_workspace_size(num_seqs: int, total_tokens: int, num_heads: int) -> int:
    """Workspace bytes ``kda_gated_delta_chunk_fwd`` needs on the current CUDA device (0: none)."""
    return int(load_library().kda_gated_delta_chunk_fwd_workspace_size(int(num_seqs), int(total_tokens), int(num_heads)))


def _delta_chunk(inputs, q, k, v, g, beta, cu_seqlens, initial_state, scale, o, final_state, status, stream, workspace,
                 withhold=None):
    index, T, H, Hk, D, V, qs, ks, vs = inputs
    N = cu_seqlens.shape[0] - 1
    _need(cu_seqlens, "cu_seqlens", _I32, (N + 1,), index)
    lib = load_library()
    if workspace is None:
        if _current_device() == index:
            need = lib.kda_gated_delta_chunk_fwd_workspace_size(N, T, H)
        else:
            with torch.cuda.device(index):
                need = lib.kda_gated_delta_chunk_fwd_workspace_size(N, T, H)
        if need:
            with _on(stream):
                workspace = torch.empty(need, dtype=_U8, device=q.device)
    elif workspace.get_device() != index or workspace.dtype is not _U8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), cu_seqlens.data_ptr(), N, T, H, Hk,
            D, V, qs, ks, vs, _p(initial_state), scale, o.data_ptr(), _p(final_state), _p(status), _p(workspace),
            0 if workspace is None else workspace.numel())
    if withhold is not None:
        debug = lib.kda_gated_delta_chunk_fwd_debug
        return _call(lambda *a: debug(*a, withhold), "kda_gated_delta_chunk_fwd_debug", index, args, stream)
    return _call(lib.kda_gated_delta_chunk_fwd, "kda_gated_delta_chunk_fwd", index, args, stream)


def kda_gated_delta_chunk_fwd(q, k, v, g, beta, cu_seqlens, initial_state, scale: float, o, final_state, status=None,
                              stream=None, workspace=None, withhold: Optional[int] = None) -> int:
    """Call the C entry point ``kda_gated_delta_chunk_fwd`` with caller-allocated outputs.

    q, k: bf16 [T,Hk,128]; v: bf16 [T,H,128], H a multiple of Hk (tokens may be
    strided); g, beta: fp32 [T,H]; cu_seqlens: int32 [N+1]; initial_state /
    final_state: fp32 [N,H,128,128] or None (may be the same tensor); o: bf16
    [T,H,128]; status: int32 [1] or None; workspace: uint8 tensor of
    ``gated_delta_workspace_size(N, T, H)`` bytes (default: a new one from torch's
    allocator for the call's stream). All on one CUDA device. ``withhold`` calls
    ``kda_gated_delta_chunk_fwd_debug`` with this number. Raises ``KdaError`` on a
    host-side error; returns ``KDA_OK`` once queued.
    """
    N = cu_seqlens.shape[0] - 1
    inputs = _delta_inputs(q, k, v, g, beta, initial_state, N)
    _delta_outputs(inputs, o, final_state, status, N)
    return _delta_chunk(inputs, q, k, v, g, beta, cu_seqlens, initial_state, scale, o, final_state, status, stream, workspace,
                        withhold)


def gated_delta_chunk_fwd(q, k, v, g, beta, cu_seqlens, initial_state=None, scale: Optional[float] = None,
                          output_final_state: bool = True, check: bool = False, stream=None):
    """Allocate ``o`` (and ``final_state``) and run ``kda_gated_delta_chunk_fwd``.

    Returns ``(o, final_state)``; ``final_state`` is None when not requested. With
    ``check=True`` the device status word is read back (a synchronising copy)
    and a device-detected error raises ``KdaError``. Rows of ``o`` behind the last
    sequence are not written.
    """
    if stream is None and not check and _native is not None:
        r = _native.gated_delta_chunk(q, k, v, g, beta, cu_seqlens, initial_state, scale, True if output_final_state else False)
        if r is not None:
            return _done(r, "kda_gated_delta_chunk_fwd")
    N = cu_seqlens.shape[0] - 1
    inputs = _delta_inputs(q, k, v, g, beta, initial_state, N)
    _, T, H, _, D, V = inputs[:6]
    dev = q.device
    with _on(stream):
        o = torch.empty((T, H, V), dtype=_BF16, device=dev)
        fs = torch.empty((N, H, D, V), dtype=_F32, device=dev) if output_final_state else None
        status = _status(check, dev)
    _delta_chunk(inputs, q, k, v, g, beta, cu_seqlens, initial_state, D ** -0.5 if scale is None else scale, o, fs, status, stream,
                 None)
    if check:
        _raise_device(status, stream, "kda_gated_delta_chunk_fwd")
    return o, fs


def _steps(q, num_seqs):
    N, T = int(num_seqs), q.shape[0]
    if N < 0 or (N == 0 and T != 0) or (N > 0 and T % N != 0):
        raise ValueError("q must hold the same number of tokens for every sequence")
    return N, T // N if N else 0


def _delta_decode(inputs, q, k, v, g, beta, N, steps, initial_state, scale, o, final_state, status, stream):
    index, _, H, Hk, D, V, qs, ks, vs = inputs
    return _call(load_library().kda_gated_delta_decode_fwd, "kda_gated_delta_decode_fwd", index,
                 (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), N, steps, H, Hk, D, V, qs, ks, vs,
                  _p(initial_state), scale, o.data_ptr(), _p(final_state), _p(status)), stream)


def kda_gated_delta_decode_fwd(q, k, v, g, beta, num_seqs: int, initial_state, scale: float, o, final_state, status=None,
                               stream=None) -> int:
    """Call the C entry point ``kda_gated_delta_decode_fwd`` with caller-allocated
    outputs: sequence n's tokens are rows n*Tn .. n*Tn+Tn-1 of q, k, v, g, beta and
    o; tensors as in ``kda_gated_delta_chunk_fwd``."""
    N, steps = _steps(q, num_seqs)
    inputs = _delta_inputs(q, k, v, g, beta, initial_state, N)
    _delta_outputs(inputs, o, final_state, status, N)
    return _delta_decode(inputs, q, k, v, g, beta, N, steps, initial_state, scale, o, final_state, status, stream)


def gated_delta_decode_fwd(q, k, v, g, beta, num_seqs: int, state=None, scale: Optional[float] = None,
                           in_place: bool = False, check: bool = False, stream=None):
    """Run ``kda_gated_delta_decode_fwd``; returns ``(o, final_state)``. With
    ``in_place`` the given ``state`` tensor is updated and returned as ``final_state``."""
    if stream is None and not check and _native is not None:
        r = _native.gated_delta_decode(q, k, v, g, beta, num_seqs, state, scale, True if in_place else False)
        if r is not None:
            return _done(r, "kda_gated_delta_decode_fwd")
    N, steps = _steps(q, num_seqs)
    inputs = _delta_inputs(q, k, v, g, beta, state, N)
    _, T, H, _, D, V = inputs[:6]
    if in_place and state is None:
        raise ValueError("in_place needs a state tensor")
    dev = q.device
    with _on(stream):
        o = torch.empty((T, H, V), dtype=_BF16, device=dev)
        fs = state if in_place else torch.empty((N, H, D, V), dtype=_F32, device=dev)
        status = _status(check, dev)
    _delta_decode(inputs, q, k, v, g, beta, N, steps, state, D ** -0.5 if scale is None else scale, o, fs, status, stream)
    if check:
        _raise_device(status, stream, "kda_gated_delta_decode_fwd")
    return o, fs


# ------------------------------------------------------------------ gated RMS norm of the heads' outputs, e4m3 output
_ACTIVATIONS = {"sigmoid": 0, "silu": 1}


def _gate_inputs(x, gate, weight, activation):
    index, shape, kind = _device_of(x), x.shape, x.dtype
    if len(shape) != 3:
        raise ValueError(f"x must have shape (tokens, heads, head_dim), got {tuple(shape)}")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(_ACTIVATIONS)}, got {activation!r}")
    if kind is not _BF16 and kind is not _F32:
        raise TypeError(f"x must be {_BF16} or {_F32}, got {kind}")
    T, H, D = shape
    _need(x, "x", kind, shape, index)
    gs = _heads_view(gate, "gate", T, index)
    if gate.shape != shape:
        raise ValueError(f"gate must have x's shape {tuple(shape)}, got {tuple(gate.shape)}")
    _need(weight, "weight", _F32, (D,), index)
    return index, T, H, D, gs, 1 if kind is _F32 else 0, _ACTIVATIONS[activation]


def _gate_call(inputs, x, gate, weight, eps, y, y_scale, stream):
    index, T, H, D, gs, fp32, silu = inputs
    return _call(load_library().kda_gated_rms_norm, "kda_gated_rms_norm", index,
                 (x.data_ptr(), gate.data_ptr(), gs, weight.data_ptr(), T, H, D, eps, fp32, silu, y.data_ptr(), y_scale.data_ptr()),
                 stream)


def kda_gated_rms_norm(x, gate, weight, eps: float, y, y_scale, activation: str = "sigmoid", stream=None) -> int:
    """Call the C entry point ``kda_gated_rms_norm``: x bf16 or fp32 [T,H,128];
    gate bf16 [T,H,128] (tokens may be strided); weight fp32 [128]; y
    float8_e4m3fn [T,H*128]; y_scale fp32 [T,H]; activation "sigmoid" or "silu"."""
    inputs = _gate_inputs(x, gate, weight, activation)
    index, T, H, D = inputs[:4]
    _need(y, "y", _F8, (T, H * D), index)
    _need(y_scale, "y_scale", _F32, (T, H), index)
    return _gate_call(inputs, x, gate, weight, eps, y, y_scale, stream)


def gated_rms_norm(x, gate, weight, eps: float = 1e-5, activation: str = "sigmoid", stream=None):
    """Run ``kda_gated_rms_norm`` on an attention output x [T,H,128]; returns
    ``(y, y_scale)``, float8_e4m3fn [T,H*128] and fp32 [T,H]."""
    if stream is None and _native is not None and activation in _ACTIVATIONS:
        r = _native.gated_rms_norm(x, gate, weight, eps, _ACTIVATIONS[activation])
        if r is not None:
            return _done(r, "kda_gated_rms_norm")
    inputs = _gate_inputs(x, gate, weight, activation)
    _, T, H, D = inputs[:4]
    dev = x.device
    with _on(stream):
        y = torch.empty((T, H * D), dtype=_F8, device=dev)
        y_scale = torch.empty((T, H), dtype=_F32, device=dev)
    _gate_call(inputs, x, gate, weight, eps, y, y_scale, stream)
    return y, y_scale


# ------------------------------------------------------------------ e4m3 product with scales
def _product_inputs(x, x_scale, weight, weight_scale):
    index, shape = _device_of(x), x.shape
    if len(shape) < 1 or weight.dim() != 2:
        raise ValueError("x must have shape (..., width) and weight (outs, width)")
    N, K = weight.shape
    lead = shape[:-1]
    blocks = (K + 127) // 128
    per_block = x_scale.dim() == len(shape)
    _need(x, "x", _F8, (*lead, K), index)
    _need(weight, "weight", _F8, (N, K), index)
    _need(x_scale, "x_scale", _F32, (*lead, blocks) if per_block else lead, index)
    _need(weight_scale, "weight_scale", _F32, ((N + 127) // 128, blocks), index)
    return index, lead, K, N, int(per_block)


def _product_call(inputs, x, x_scale, weight, weight_scale, y, status, stream, withhold=None):
    index, lead, K, N, per_block = inputs
    lib = load_library()
    args = (x.data_ptr(), x_scale.data_ptr(), per_block, weight.data_ptr(), weight_scale.data_ptr(), lead.numel(), K, N,
            y.data_ptr(), _p(status))
    if withhold is not None:
        return _call(lambda *a: lib.kda_scaled_matmul_debug(*a, withhold), "kda_scaled_matmul_debug", index, args, stream)
    return _call(lib.kda_scaled_matmul, "kda_scaled_matmul", index, args, stream)


def kda_scaled_matmul(x, x_scale, weight, weight_scale, y, status=None, stream=None, withhold: Optional[int] = None) -> int:
    """Call the C entry point ``kda_scaled_matmul``: x float8_e4m3fn [..., K] with
    x_scale fp32 [...] or [..., ceil(K/128)]; weight float8_e4m3fn [N,K] with
    weight_scale fp32 [ceil(N/128), ceil(K/128)]; y bf16 [..., N]; status: int32 [1] or
    None. ``withhold`` calls ``kda_scaled_matmul_debug`` with this number."""
    inputs = _product_inputs(x, x_scale, weight, weight_scale)
    index, lead, _, N, _ = inputs
    _need(y, "y", _BF16, (*lead, N), index)
    if status is not None:
        _need(status, "status", _I32, (1,), index)
    return _product_call(inputs, x, x_scale, weight, weight_scale, y, status, stream, withhold)


def scaled_matmul(x, x_scale, weight, weight_scale, check: bool = False, stream=None):
    """Run ``kda_scaled_matmul``; returns y bf16 [..., N]. With ``check=True`` the
    device status word is read back (a synchronising copy)."""
    if stream is None and not check and _native is not None:
        r = _native.scaled_matmul(x, x_scale, weight, weight_scale)
        if r is not None:
            return _done(r, "kda_scaled_matmul")
    inputs = _product_inputs(x, x_scale, weight, weight_scale)
    dev = x.device
    with _on(stream):
        y = torch.empty((*inputs[1], inputs[3]), dtype=_BF16, device=dev)
        status = _status(check, dev)
    _product_call(inputs, x, x_scale, weight, weight_scale, y, status, stream)
    if check:
        _raise_device(status, stream, "kda_scaled_matmul")
    return y
