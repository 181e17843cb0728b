"""Thin ctypes binding of liblla.so (include/lla.h) for torch tensors.

Argument marshalling only: every step of the operator runs in the library's
CUDA kernels. torch supplies device memory and the current stream. The
library must exist (built by ``log_linear_attention_gb300.build``); there is
no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblla.so")

LLA_OK = 0
LLA_ERR_INVALID_ARG = -1
LLA_ERR_UNSUPPORTED = -2
LLA_ERR_CUDA = -3
LLA_ERR_TIMEOUT = -4
LLA_ERR_NOMEM = -5
LLA_ERR_DEVICE = -6
LLA_BF16 = 0
LLA_F32 = 1

_lock = threading.Lock()
_lib = None


class LLAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load() -> ctypes.CDLL:
    """Load liblla.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with log_linear_attention_gb300.build.build()")
            lib = ctypes.CDLL(LIB_PATH)
            vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.lla_status_string.argtypes = [i]
            lib.lla_status_string.restype = ctypes.c_char_p
            lib.lla_num_levels.argtypes = [ctypes.c_int64]
            lib.lla_num_levels.restype = i
            lib.lla_forward.argtypes = [vp, vp, vp, fp, fp, vp] + [i] * 6 + [vp, i]
            lib.lla_forward.restype = i
            lib.lla_forward_workspace_size.argtypes = [i] * 7
            lib.lla_forward_workspace_size.restype = sz
            lib.lla_forward_host.argtypes = [vp, vp, vp, fp, fp, vp] + [i] * 6 + [vp, i]
            lib.lla_forward_host.restype = i
            lib.lla_forward_ws.argtypes = [vp, vp, vp, fp, fp, vp] + [i] * 6 + [vp, i, vp, sz]
            lib.lla_forward_ws.restype = i
            lib.lla_forward_noalloc.argtypes = [vp, vp, vp, fp, fp, vp] + [i] * 6 + [vp, i]
            lib.lla_forward_noalloc.restype = i
            lib.lla_forward_profile.argtypes = [vp, vp, vp, fp, fp, vp] + [i] * 6 + [vp, i, vp, vp, i]
            lib.lla_forward_profile.restype = i
            lib.lla_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, vp] + [i] * 6
            lib.lla_decode_step.restype = i
            lib.lla_prefill_state.argtypes = [vp, vp, fp, fp] + [i] * 6 + [vp, i]
            lib.lla_prefill_state.restype = i
            lib.lla_device_error.argtypes = [vp]
            lib.lla_device_error.restype = i
            lib.lla_gdn_forward.argtypes = [vp, vp, vp, fp, fp, fp, vp] + [i] * 6 + [vp, i]
            lib.lla_gdn_forward.restype = i
            lib.lla_gdn_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, vp, vp] + [i] * 6
            lib.lla_gdn_decode_step.restype = i
            lib.lla_gdn_forward_profile.argtypes = [vp, vp, vp, fp, fp, fp, vp] + [i] * 6 + [vp, i, vp, vp, i]
            lib.lla_gdn_forward_profile.restype = i
            lib.lla_debug_set_waits.argtypes = [ctypes.c_int64, i]
            lib.lla_debug_set_waits.restype = i
            lib.lla_backward.argtypes = [vp, vp, vp, fp, fp, vp, vp, vp, vp, fp, fp] + [i] * 6 + [vp, i]
            lib.lla_backward.restype = i
            lib.lla_forward_varlen.argtypes = [vp, vp, vp, fp, fp, vp, vp] + [i] * 7 + [vp, i]
            lib.lla_forward_varlen.restype = i
            lib.lla_prefill_state_varlen.argtypes = [vp, vp, fp, vp, fp] + [i] * 7 + [vp, i]
            lib.lla_prefill_state_varlen.restype = i
            lib.lla_linear_forward.argtypes = [vp, vp, vp, fp, fp, vp, fp] + [i] * 6 + [vp, i]
            lib.lla_linear_forward.restype = i
            lib.lla_linear_forward_varlen.argtypes = [vp, vp, vp, fp, fp, vp, fp, vp] + [i] * 7 + [vp, i]
            lib.lla_linear_forward_varlen.restype = i
            lib.lla_linear_backward.argtypes = [vp, vp, vp, fp, fp, vp, fp, vp, vp, vp, fp] + [i] * 6 + [vp, i]
            lib.lla_linear_backward.restype = i
            lib.lla_linear_decode_step.argtypes = [vp, vp, vp, fp, fp, vp, vp] + [i] * 5
            lib.lla_linear_decode_step.restype = i
            lib.lla_decode_step_shared.argtypes = ([vp, vp, vp, fp, fp, fp, ctypes.c_int64, i, fp, fp, vp, vp, vp]
                                                   + [i] * 6)
            lib.lla_decode_step_shared.restype = i
            for name, types in {
                "lla_gated_forward": [vp, vp, fp, vp, fp] + [i] * 4 + [vp, i, i],
                "lla_gated_forward_varlen": [vp, vp, fp, vp, fp, vp] + [i] * 4 + [vp, i, i],
                "lla_gated_backward": [vp, vp, fp, vp, fp, vp, vp, fp] + [i] * 4 + [vp, i, i],
                "lla_gated_backward_varlen": [vp, vp, fp, vp, fp, vp, vp, fp, vp] + [i] * 4 + [vp, i, i],
                "lla_gated_decode_step": [vp, vp, fp, vp, vp] + [i] * 4,
                "lla_gated_decode_tree": [vp, vp, fp, vp, vp, vp] + [i] * 6,
                "lla_gated_decode_commit": [vp, vp, fp, vp, vp, vp] + [i] * 6,
                "lla_decode_tree": [vp, vp, vp, fp, fp, fp, vp, vp, vp, vp] + [i] * 8,
                "lla_decode_commit": [vp, vp, fp, fp, vp, vp, vp, vp] + [i] * 8,
                "lla_linear_decode_tree": [vp, vp, vp, fp, fp, vp, vp, vp] + [i] * 7,
                "lla_linear_decode_commit": [vp, vp, fp, fp, vp, vp, vp] + [i] * 7,
            }.items():
                getattr(lib, name).argtypes = types
                getattr(lib, name).restype = i
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().lla_status_string(int(status)).decode()


def num_levels(T: int) -> int:
    return int(load().lla_num_levels(int(T)))


_torch_module = None
_current_device = _raw_stream = None  # the current device's index; the handle of a device's current stream


def _cuda_calls(torch):
    """(current device, current stream's handle), as torch's own bindings give them without building objects, or through
    torch.cuda where a torch has no such bindings."""
    device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return device, stream or (lambda index: int(torch.cuda.current_stream(index).cuda_stream))


def _torch():
    global _torch_module, _current_device, _raw_stream
    if _torch_module is None:
        import torch
        _current_device, _raw_stream = _cuda_calls(torch)
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return LLA_BF16
    if t.dtype == torch.float32:
        return LLA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _stream_handle(stream) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _check(t, name, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _call(status: int, where: str):
    if status != LLA_OK:
        raise LLAError(status, where)


def forward(q, k, v, log_a, lam, chunk: int, out=None, stream=None, workspace=None):
    """Chunk-parallel prefill, lla_forward / lla_forward_ws.

    q, k [B,H,T,dk]; v [B,H,T,dv] (bf16 or fp32, same dtype); log_a [B,H,T] fp32;
    lam [B,H,T,L] fp32 with L = num_levels(T). Host (CPU) inputs go through
    lla_forward_host (pipelined copies in and out) and the result comes back in host memory.
    ``workspace``: optional uint8 CUDA tensor of at least workspace_size(...) bytes.
    """
    torch = _torch()
    if not q.is_cuda:
        return _forward_host(q, k, v, log_a, lam, chunk, out, stream)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda")):
        _check(t_, n, q.device)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    if log_a.dtype != torch.float32 or lam.dtype != torch.float32:
        raise TypeError("log_a and lambda must be float32")
    if k.shape != q.shape or v.shape[:3] != (B, H, T) or log_a.shape != (B, H, T) or lam.shape[:3] != (B, H, T):
        raise ValueError("shape mismatch between q, k, v, log_a and lambda")
    if lam.shape[3] != num_levels(T):
        raise ValueError(f"lambda needs {num_levels(T)} levels for T={T}, got {lam.shape[3]}")
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", q.device)
    code = _dtype_code(q)
    lib = load()
    sh = _stream_handle(stream)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(), out.data_ptr(),
            B, H, T, dk, dv, int(chunk), sh, code)
    if workspace is None:
        _call(lib.lla_forward(*args), "lla_forward")
    else:
        _check(workspace, "workspace", q.device)
        _call(lib.lla_forward_ws(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size()),
              "lla_forward_ws")
    return out


def _forward_host(q, k, v, log_a, lam, chunk, out=None, stream=None):
    """lla_forward_host: every tensor in host memory (pinned for full copy bandwidth). The
    library copies head groups in, runs them and copies them out with the copies of one group
    overlapping the kernels of the next; returns the host output (pinned unless given)."""
    torch = _torch()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda")):
        if t_.is_cuda or not t_.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor")
    if k.dtype != q.dtype or v.dtype != q.dtype or log_a.dtype != torch.float32 or lam.dtype != torch.float32:
        raise TypeError("q, k, v share one dtype; log_a and lambda are float32")
    if k.shape != q.shape or v.shape[:3] != (B, H, T) or log_a.shape != (B, H, T) or lam.shape != (B, H, T, num_levels(T)):
        raise ValueError("shape mismatch between q, k, v, log_a and lambda")
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, pin_memory=True)
    if out.is_cuda or not out.is_contiguous() or out.shape != (B, H, T, dv) or out.dtype != q.dtype:
        raise ValueError("out must be a contiguous host tensor [B,H,T,dv] of q's dtype")
    _call(load().lla_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                  out.data_ptr(), B, H, T, dk, dv, int(chunk), _stream_handle(stream),
                                  _dtype_code(q)), "lla_forward_host")
    return out


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def forward_noalloc(q, k, v, log_a, lam, chunk: int, out, stream=None):
    """lla_forward_noalloc: the prefill with its scratch in the library's fixed device
    array (no allocation at all). ``out`` must be preallocated by the caller. Raises
    LLAError(LLA_ERR_NOMEM) when the sizes need more than NOALLOC_SCRATCH_BYTES."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda"), (out, "out")):
        _check(t_, n, q.device)
    _call(load().lla_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                     out.data_ptr(), B, H, T, dk, dv, int(chunk), _stream_handle(stream),
                                     _dtype_code(q)), "lla_forward_noalloc")
    return out


def forward_profile(q, k, v, log_a, lam, chunk: int, out, stream=None):
    """lla_forward_profile: one synchronous forward call; returns [(kernel_name, ms), ...]
    in launch order, timed with CUDA events on the launch stream."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    cap = 32
    ms = (ctypes.c_float * cap)()
    names = (ctypes.c_char_p * cap)()
    n = load().lla_forward_profile(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                   out.data_ptr(), B, H, T, dk, dv, int(chunk), _stream_handle(stream),
                                   _dtype_code(q), ctypes.cast(ms, ctypes.c_void_p),
                                   ctypes.cast(names, ctypes.c_void_p), cap)
    if n < 0:
        raise LLAError(n, "lla_forward_profile")
    return [(names[i].decode(), float(ms[i])) for i in range(min(n, cap))]


def gdn_forward(q, k, v, log_a, beta, lam, chunk: int, out=None, stream=None):
    """Log-linear Gated DeltaNet prefill, lla_gdn_forward: as ``forward`` plus ``beta`` [B,H,T] fp32."""
    torch = _torch()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (beta, "beta"), (lam, "lambda"), (out, "out")):
        _check(t_, n, q.device)
    _call(load().lla_gdn_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), beta.data_ptr(),
                                 lam.data_ptr(), out.data_ptr(), B, H, T, dk, dv, int(chunk), _stream_handle(stream),
                                 _dtype_code(q)), "lla_gdn_forward")
    return out


def gdn_forward_profile(q, k, v, log_a, beta, lam, chunk: int, out, stream=None):
    """lla_gdn_forward_profile: one synchronous call; returns [(kernel_name, ms), ...] in launch order."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    cap = 32
    ms = (ctypes.c_float * cap)()
    names = (ctypes.c_char_p * cap)()
    n = load().lla_gdn_forward_profile(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), beta.data_ptr(),
                                       lam.data_ptr(), out.data_ptr(), B, H, T, dk, dv, int(chunk),
                                       _stream_handle(stream), _dtype_code(q), ctypes.cast(ms, ctypes.c_void_p),
                                       ctypes.cast(names, ctypes.c_void_p), cap)
    if n < 0:
        raise LLAError(n, "lla_gdn_forward_profile")
    return [(names[i].decode(), float(ms[i])) for i in range(min(n, cap))]


def gdn_decode_step(q, k, v, log_a, beta, lam, states, t, out=None, stream=None):
    """One log-linear Gated DeltaNet decode step, lla_gdn_decode_step (states updated in place)."""
    torch = _torch()
    B, H, dk = q.shape
    dv = v.shape[-1]
    Lmax = states.shape[2]
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (beta, "beta"), (lam, "lambda"),
                  (states, "states"), (t, "t"), (out, "out")):
        _check(t_, n, q.device)
    _call(load().lla_gdn_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), beta.data_ptr(),
                                     lam.data_ptr(), states.data_ptr(), t.data_ptr(), out.data_ptr(),
                                     _stream_handle(stream), B, H, dk, dv, Lmax, _dtype_code(q)),
          "lla_gdn_decode_step")
    return out


def debug_set_waits(limit_cycles: int, hold: bool) -> None:
    """lla_debug_set_waits: test hook of the bounded waits (see include/lla.h)."""
    _call(load().lla_debug_set_waits(int(limit_cycles), 1 if hold else 0), "lla_debug_set_waits")


def workspace_size(B: int, H: int, T: int, dk: int, dv: int, chunk: int, dtype) -> int:
    """Bytes of caller-owned workspace lla_forward_ws needs (0 for invalid sizes)."""
    torch = _torch()
    code = LLA_BF16 if dtype == torch.bfloat16 else LLA_F32
    return int(load().lla_forward_workspace_size(B, H, T, dk, dv, int(chunk), code))


def decode_step(q, k, v, log_a, lam, states, t, out=None, stream=None):
    """One recurrent decode step, lla_decode_step. ``states`` [B,H,Lmax,dk,dv] fp32 is
    updated in place; ``t`` int64 [B] on the device. Returns out [B,H,dv]."""
    torch = _torch()
    B, H, dk = q.shape
    dv = v.shape[-1]
    Lmax = states.shape[2]
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda"), (states, "states"), (t, "t")):
        _check(t_, n, q.device)
    if states.dtype != torch.float32 or states.shape != (B, H, Lmax, dk, dv):
        raise ValueError("states must be float32 [B,H,Lmax,dk,dv]")
    if t.dtype != torch.int64 or t.shape != (B,):
        raise ValueError("t must be int64 [B]")
    if lam.shape != (B, H, Lmax) or log_a.shape != (B, H) or k.shape != q.shape or v.shape[:2] != (B, H):
        raise ValueError("shape mismatch in decode inputs")
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", q.device)
    _call(load().lla_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                 states.data_ptr(), t.data_ptr(), out.data_ptr(), _stream_handle(stream),
                                 B, H, dk, dv, Lmax, _dtype_code(q)), "lla_decode_step")
    return out


def prefill_state(k, v, log_a, states, stream=None):
    """lla_prefill_state: write into ``states`` [B,H,Lmax,dk,dv] fp32 the Fenwick state set after
    the prompt (k [B,H,T,dk], v [B,H,T,dv], log_a [B,H,T]); the next decode position is t = T."""
    torch = _torch()
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    Lmax = states.shape[2]
    for t_, n in ((k, "k"), (v, "v"), (log_a, "log_a"), (states, "states")):
        _check(t_, n, k.device)
    if states.dtype != torch.float32 or states.shape != (B, H, Lmax, dk, dv):
        raise ValueError("states must be float32 [B,H,Lmax,dk,dv]")
    _call(load().lla_prefill_state(k.data_ptr(), v.data_ptr(), log_a.data_ptr(), states.data_ptr(), B, H, T, dk, dv,
                                   Lmax, _stream_handle(stream), _dtype_code(k)), "lla_prefill_state")
    return states


def backward(q, k, v, log_a, lam, dout, chunk: int, stream=None):
    """lla_backward: gradients of sum(dout * forward(q, k, v, log_a, lam)).

    Device tensors with the shapes and dtypes of lla_forward's inputs; dout like the output.
    Returns (dq, dk, dv, dlog_a, dlambda): dq/dk/dv in q's dtype, dlog_a/dlambda fp32."""
    torch = _torch()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda"), (dout, "dout")):
        _check(t_, n, q.device)
    if k.dtype != q.dtype or v.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("q, k, v and dout must share one dtype")
    if log_a.dtype != torch.float32 or lam.dtype != torch.float32:
        raise TypeError("log_a and lambda must be float32")
    if (k.shape != q.shape or v.shape[:3] != (B, H, T) or dout.shape != v.shape or log_a.shape != (B, H, T)
            or lam.shape[:3] != (B, H, T)):
        raise ValueError("shape mismatch between q, k, v, dout, log_a and lambda")
    if lam.shape[3] != num_levels(T):
        raise ValueError(f"lambda needs {num_levels(T)} levels for T={T}, got {lam.shape[3]}")
    dq = torch.empty_like(q)
    dk_ = torch.empty_like(k)
    dv_ = torch.empty_like(v)
    dla = torch.empty_like(log_a)
    dlam = torch.empty_like(lam)
    _call(load().lla_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                              dout.data_ptr(), dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(), dla.data_ptr(),
                              dlam.data_ptr(), B, H, T, dk, dv, chunk, _stream_handle(stream), _dtype_code(q)),
          "lla_backward")
    return dq, dk_, dv_, dla, dlam


def forward_varlen(q, k, v, log_a, lam, cu_seqlens, max_T: int, chunk: int, out=None, stream=None):
    """lla_forward_varlen: packed sequences. q, k [H,total,dk]; v [H,total,dv]; log_a [H,total];
    lam [H,total,num_levels(max_T)]; cu_seqlens int32 [n+1] on the device."""
    torch = _torch()
    H, total, dk = q.shape
    dv = v.shape[-1]
    n = cu_seqlens.numel() - 1
    for t_, nm in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda"), (cu_seqlens, "cu_seqlens")):
        _check(t_, nm, q.device)
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if k.shape != q.shape or v.shape[:2] != (H, total) or log_a.shape != (H, total) or lam.shape[:2] != (H, total):
        raise ValueError("shape mismatch between packed q, k, v, log_a and lambda")
    if lam.shape[2] != num_levels(max_T):
        raise ValueError(f"lambda needs {num_levels(max_T)} levels for max_T={max_T}")
    if out is None:
        out = torch.empty((H, total, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", q.device)
    _call(load().lla_forward_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                    out.data_ptr(), cu_seqlens.data_ptr(), n, H, total, max_T, dk, dv, chunk,
                                    _stream_handle(stream), _dtype_code(q)), "lla_forward_varlen")
    return out


def prefill_state_varlen(k, v, log_a, cu_seqlens, max_T: int, states, stream=None):
    """lla_prefill_state_varlen: states [n,H,Lmax,dk,dv] fp32 after each packed sequence."""
    torch = _torch()
    H, total, dk = k.shape
    dv = v.shape[-1]
    n = cu_seqlens.numel() - 1
    Lmax = states.shape[2]
    for t_, nm in ((k, "k"), (v, "v"), (log_a, "log_a"), (cu_seqlens, "cu_seqlens"), (states, "states")):
        _check(t_, nm, k.device)
    if cu_seqlens.dtype != torch.int32 or states.dtype != torch.float32 or states.shape != (n, H, Lmax, dk, dv):
        raise ValueError("cu_seqlens must be int32 and states float32 [n,H,Lmax,dk,dv]")
    _call(load().lla_prefill_state_varlen(k.data_ptr(), v.data_ptr(), log_a.data_ptr(), cu_seqlens.data_ptr(),
                                          states.data_ptr(), n, H, total, max_T, dk, dv, Lmax,
                                          _stream_handle(stream), _dtype_code(k)), "lla_prefill_state_varlen")
    return states


def device_error(stream=None) -> int:
    """Synchronise ``stream``, then read and clear the device error word (an lla status)."""
    return int(load().lla_device_error(_stream_handle(stream)))


# The calls below are short on the GPU where they serve single tokens, so what the host does counts: each finds in
# one expression that its arguments are as they should be, and only otherwise goes through the checks that name what
# is wrong.

def _linear_inputs(names, tensors, log_a, H):
    """Checks of the linear-attention calls: CUDA tensors of one dtype and device, log_a [H] fp32."""
    torch = _torch()
    q = tensors[0]
    for n, t_ in zip(names, tensors):
        _check(t_, n, q.device)
        if t_.dtype != q.dtype:
            raise TypeError(f"{', '.join(names)} must share one dtype")
    _check(log_a, "log_a", q.device)
    if log_a.dtype != torch.float32 or log_a.shape != (H,):
        raise ValueError(f"log_a must be float32 [{H}] (one decay per head)")


def _state(t_, name, shape, device):
    """Address of an optional fp32 state tensor of the given shape (None: NULL)."""
    if t_ is None:
        return None
    torch = _torch_module
    if not (type(t_) is torch.Tensor and t_.dtype is torch.float32 and t_.shape == shape and t_.is_contiguous()
            and t_.device == device):
        _check(t_, name, device)
        if t_.dtype != torch.float32 or t_.shape != shape:
            raise ValueError(f"{name} must be float32 {list(shape)}, got {t_.dtype} {list(t_.shape)}")
    return t_.data_ptr()


def _small(t_, where, *written):
    """A per-head or per-sequence array at the library's alignment of 16 bytes: itself, or a copy where it starts between
    (a rank's part of the decays, the positions of a part of the batch). The library sees the copy, so that the call
    writes nothing over the array itself is found here."""
    at = t_.data_ptr()
    if at & 15 == 0:
        return t_
    for w in written:
        if w is not None and w.data_ptr() < at + t_.numel() * t_.element_size() and at < w.data_ptr() + w.numel() * w.element_size():
            raise LLAError(LLA_ERR_INVALID_ARG, where)
    return t_.clone()


def _elsewhere(device, stream, call, *args):
    """call(*args) with ``device`` and ``stream`` current, so that what it allocates belongs to the stream that
    writes it."""
    torch = _torch()
    with torch.cuda.device(device):
        if stream is None:
            return call(*args)
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return call(*args)


def _given(out, v):
    """The caller's output tensor, checked: like v in shape, dtype and device."""
    _check(out, "out", v.device)
    if out.dtype != v.dtype or out.shape != v.shape:
        raise ValueError(f"out must be {v.dtype} {list(v.shape)}, got {out.dtype} {list(out.shape)}")
    return out


def linear_forward(q, k, v, log_a, state0=None, state_out=None, out=None, stream=None):
    """Linear attention with one decay per head, lla_linear_forward: S_t = exp(log_a_h) S_{t-1} + k_t v_t^T,
    o_t = S_t^T q_t. Returns out [B,H,T,dv].

    q, k [B,H,T,dk]; v [B,H,T,dv] (bf16 or fp32, one dtype, any T >= 1); log_a [H] fp32. ``state0`` fp32
    [B,H,dk,dv], or [1,H,dk,dv] for one state shared by the batch, is the state the sequences go on from;
    ``state_out`` fp32 [B,H,dk,dv] is written with the state after the last token (see linear_decode_step)."""
    torch = _torch()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dtype, device, index = q.dtype, q.device, q.get_device()
    if not (type(q) is type(k) is type(v) is type(log_a) is torch.Tensor and index >= 0 and k.dtype is dtype
            and v.dtype is dtype and log_a.dtype is torch.float32 and k.shape == q.shape and v.shape == (B, H, T, dv)
            and log_a.shape == (H,) and k.get_device() == v.get_device() == log_a.get_device() == index
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and log_a.is_contiguous()):
        _linear_inputs(("q", "k", "v"), (q, k, v), log_a, H)
        if k.shape != q.shape or v.shape != (B, H, T, dv):
            raise ValueError("shape mismatch between q, k and v")
    if stream is not None or index != _current_device():
        return _elsewhere(device, stream, linear_forward, q, k, v, log_a, state0, state_out, out)
    B0 = 0 if state0 is None else int(state0.shape[0])
    s0 = _state(state0, "state0", (1 if B0 == 1 else B, H, dk, dv), device)
    s1 = _state(state_out, "state_out", (B, H, dk, dv), device)
    o = torch.empty_like(v) if out is None else _given(out, v)
    log_a = _small(log_a, "lla_linear_forward", o, state_out)
    _call(load().lla_linear_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), s0, o.data_ptr(), s1, B,
                                    B0, H, T, dk, dv, _raw_stream(index), _dtype_code(q)),
          "lla_linear_forward")
    return o


def linear_forward_varlen(q, k, v, log_a, cu_seqlens, max_T: int, state0=None, state_out=None, out=None, stream=None):
    """lla_linear_forward_varlen: packed sequences. q, k [H,total,dk]; v [H,total,dv]; log_a [H]; cu_seqlens
    int32 [n+1] on the device; state0 [n,H,dk,dv] or [1,H,dk,dv] (shared); state_out [n,H,dk,dv]. Rows of
    ``out`` that belong to no sequence are left as they were (uninitialised in a new ``out``)."""
    torch = _torch()
    H, total, dk = q.shape
    dv = v.shape[-1]
    dtype, device, index = q.dtype, q.device, q.get_device()
    if not (type(q) is type(k) is type(v) is type(log_a) is type(cu_seqlens) is torch.Tensor and index >= 0
            and k.dtype is dtype and v.dtype is dtype and log_a.dtype is torch.float32
            and cu_seqlens.dtype is torch.int32 and k.shape == q.shape and v.shape == (H, total, dv)
            and log_a.shape == (H,) and cu_seqlens.dim() == 1
            and k.get_device() == v.get_device() == log_a.get_device() == cu_seqlens.get_device() == index
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and log_a.is_contiguous()
            and cu_seqlens.is_contiguous()):
        _linear_inputs(("q", "k", "v"), (q, k, v), log_a, H)
        _check(cu_seqlens, "cu_seqlens", device)
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1:
            raise TypeError("cu_seqlens must be int32 [n+1]")
        if k.shape != q.shape or v.shape != (H, total, dv):
            raise ValueError("shape mismatch between packed q, k and v")
    if stream is not None or index != _current_device():
        return _elsewhere(device, stream, linear_forward_varlen, q, k, v, log_a, cu_seqlens, max_T, state0, state_out,
                          out)
    n = cu_seqlens.numel() - 1
    n0 = 0 if state0 is None else int(state0.shape[0])
    s0 = _state(state0, "state0", (1 if n0 == 1 else n, H, dk, dv), device)
    s1 = _state(state_out, "state_out", (n, H, dk, dv), device)
    o = torch.empty_like(v) if out is None else _given(out, v)
    log_a = _small(log_a, "lla_linear_forward_varlen", o, state_out)
    cu_seqlens = _small(cu_seqlens, "lla_linear_forward_varlen", o, state_out)
    _call(load().lla_linear_forward_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), s0, o.data_ptr(),
                                           s1, cu_seqlens.data_ptr(), n, n0, H, total, int(max_T), dk, dv,
                                           _raw_stream(index), _dtype_code(q)),
          "lla_linear_forward_varlen")
    return o


def linear_backward(q, k, v, log_a, dout, state0=None, dstate_out=None, stream=None):
    """lla_linear_backward: gradients of sum(dout * out) + sum(dstate_out * state_out) of linear_forward.

    Returns (dq, dk, dv, dstate0): dq/dk/dv in q's dtype, dstate0 fp32 like state0 (None without one; summed
    over the batch where state0 is shared). log_a is a constant and has no gradient."""
    torch = _torch()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    device, index = q.device, q.get_device()
    _linear_inputs(("q", "k", "v", "dout"), (q, k, v, dout), log_a, H)
    if k.shape != q.shape or v.shape != (B, H, T, dv) or dout.shape != v.shape:
        raise ValueError("shape mismatch between q, k, v and dout")
    if stream is not None or index != _current_device():
        return _elsewhere(device, stream, linear_backward, q, k, v, log_a, dout, state0, dstate_out)
    B0 = 0 if state0 is None else int(state0.shape[0])
    s0 = _state(state0, "state0", (1 if B0 == 1 else B, H, dk, dv), device)
    s1 = _state(dstate_out, "dstate_out", (B, H, dk, dv), device)
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds = None if state0 is None else torch.empty_like(state0)
    log_a = _small(log_a, "lla_linear_backward")
    _call(load().lla_linear_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), s0, dout.data_ptr(),
                                     s1, dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(),
                                     None if ds is None else ds.data_ptr(), B, B0, H, T, dk, dv,
                                     _raw_stream(index), _dtype_code(q)), "lla_linear_backward")
    return dq, dk_, dv_, ds


def linear_decode_step(q, k, v, log_a, state, out=None, stream=None):
    """One token of every sequence, lla_linear_decode_step. q, k [B,H,dk]; v [B,H,dv]; log_a [H] fp32;
    ``state`` [B,H,dk,dv] fp32 is updated in place. Returns out [B,H,dv]."""
    torch = _torch()
    B, H, dk = q.shape
    dv = v.shape[-1]
    dtype, index = q.dtype, q.get_device()
    if not (type(q) is type(k) is type(v) is type(log_a) is type(state) is torch.Tensor and index >= 0
            and k.dtype is dtype and v.dtype is dtype and log_a.dtype is state.dtype is torch.float32
            and k.shape == q.shape and v.shape == (B, H, dv) and log_a.shape == (H,) and state.shape == (B, H, dk, dv)
            and k.get_device() == v.get_device() == log_a.get_device() == state.get_device() == index
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and log_a.is_contiguous()
            and state.is_contiguous()):
        _linear_inputs(("q", "k", "v"), (q, k, v), log_a, H)
        if k.shape != q.shape or v.shape != (B, H, dv):
            raise ValueError("shape mismatch between q, k and v")
        if state is None:
            raise ValueError("state is needed")
        _state(state, "state", (B, H, dk, dv), q.device)
    if stream is not None or index != _current_device():
        return _elsewhere(q.device, stream, linear_decode_step, q, k, v, log_a, state, out)
    o = torch.empty_like(v) if out is None else _given(out, v)
    log_a = _small(log_a, "lla_linear_decode_step", o, state)
    _call(load().lla_linear_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), state.data_ptr(),
                                        o.data_ptr(), _raw_stream(index), B, H, dk, dv,
                                        _dtype_code(q)), "lla_linear_decode_step")
    return o


def decode_step_shared(q, k, v, log_a, lam, prefix_states, prefix_len: int, prefix_decay, states, t, out=None,
                       stream=None):
    """decode_step of a batch whose sequences share their first ``prefix_len`` tokens, lla_decode_step_shared.

    ``prefix_states`` [H,Lp,dk,dv] fp32 (read only): prefill_state of the prefix, kept once. ``prefix_decay``
    [B,H] fp32 and ``states`` [B,H,Lmax,dk,dv] fp32 (each sequence's own buckets) are updated in place and need
    no initialisation. ``t`` int64 [B] on the device, prefix_len <= t. Returns out [B,H,dv]."""
    torch = _torch()
    B, H, dk = q.shape
    dv = v.shape[-1]
    if prefix_states is None or prefix_decay is None or states is None or prefix_states.dim() != 4 or states.dim() != 5:
        raise ValueError("prefix_states [H,Lp,dk,dv], prefix_decay [B,H] and states [B,H,Lmax,dk,dv] are needed")
    Lp, Lmax = prefix_states.shape[1], states.shape[2]
    dtype, f32, index = q.dtype, torch.float32, q.get_device()
    if not (type(q) is type(k) is type(v) is type(log_a) is type(lam) is type(prefix_states) is type(prefix_decay)
            is type(states) is type(t) is torch.Tensor and index >= 0 and k.dtype is dtype and v.dtype is dtype
            and log_a.dtype is lam.dtype is prefix_states.dtype is prefix_decay.dtype is states.dtype is f32
            and t.dtype is torch.int64 and k.shape == q.shape and v.shape == (B, H, dv) and log_a.shape == (B, H)
            and lam.shape == (B, H, Lmax) and prefix_states.shape == (H, Lp, dk, dv) and prefix_decay.shape == (B, H)
            and states.shape == (B, H, Lmax, dk, dv) and t.shape == (B,)
            and k.get_device() == v.get_device() == log_a.get_device() == lam.get_device() == t.get_device()
            == prefix_states.get_device() == prefix_decay.get_device() == states.get_device() == index
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and log_a.is_contiguous()
            and lam.is_contiguous() and prefix_states.is_contiguous() and prefix_decay.is_contiguous()
            and states.is_contiguous() and t.is_contiguous()):
        for t_, n in ((q, "q"), (k, "k"), (v, "v"), (log_a, "log_a"), (lam, "lambda"), (t, "t")):
            _check(t_, n, q.device)
        if k.dtype != dtype or v.dtype != dtype:
            raise TypeError("q, k and v must share one dtype")
        if log_a.dtype != f32 or lam.dtype != f32:
            raise TypeError("log_a and lambda must be float32")
        if t.dtype != torch.int64 or t.shape != (B,):
            raise ValueError("t must be int64 [B]")
        _state(prefix_states, "prefix_states", (H, Lp, dk, dv), q.device)
        _state(prefix_decay, "prefix_decay", (B, H), q.device)
        _state(states, "states", (B, H, Lmax, dk, dv), q.device)
        if lam.shape != (B, H, Lmax) or log_a.shape != (B, H) or k.shape != q.shape or v.shape != (B, H, dv):
            raise ValueError("shape mismatch in decode inputs")
    if stream is not None or index != _current_device():
        return _elsewhere(q.device, stream, decode_step_shared, q, k, v, log_a, lam, prefix_states, prefix_len,
                          prefix_decay, states, t, out)
    o = torch.empty_like(v) if out is None else _given(out, v)
    where, written = "lla_decode_step_shared", (o, states, prefix_decay)
    decay = _small(prefix_decay, where, q, k, v, log_a, lam, prefix_states, states, t, o)
    log_a, lam, t = _small(log_a, where, *written), _small(lam, where, *written), _small(t, where, *written)
    _call(load().lla_decode_step_shared(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                        prefix_states.data_ptr(), int(prefix_len), Lp, decay.data_ptr(),
                                        states.data_ptr(), t.data_ptr(), o.data_ptr(),
                                        _raw_stream(index), B, H, dk, dv, Lmax, _dtype_code(q)),
          "lla_decode_step_shared")
    if decay is not prefix_decay:
        prefix_decay.copy_(decay)
    return o


def _fits(t_, dtype, shape, index):
    return (isinstance(t_, _torch_module.Tensor) and t_.dtype is dtype and t_.shape == shape and t_.get_device() == index
            and t_.is_contiguous())


def _want(t_, name, dtype, shape, device):
    """Says what is wrong with an argument that does not fit."""
    _check(t_, name, device)
    if t_.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t_.dtype}")
    if t_.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t_.shape)}")


def _gated_inputs(x, log_a, *like, dims, name="x"):
    """(device index, dtype code, gate's dtype code) of a gated call: x, log_a of one shape, the gate fp32 or of x's type."""
    torch = _torch()
    if type(x) is not torch.Tensor or not (x.is_cuda and x.is_contiguous()):
        _check(x, name)
    code = _dtype_code(x)
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(x.shape)}")
    gate = torch.float32 if isinstance(log_a, torch.Tensor) and log_a.dtype is torch.float32 else x.dtype
    index = x.get_device()
    if not _fits(log_a, gate, x.shape, index):
        _want(log_a, "log_a", gate, x.shape, x.device)
    for n, t_ in like:
        if not _fits(t_, x.dtype, x.shape, index):
            _want(t_, n, x.dtype, x.shape, x.device)
    return index, code, LLA_F32 if gate is torch.float32 else code


def _gated_state(t_, name, n, D, device):
    """(rows, address) of an entering state [n,D] or [1,D], or (0, NULL)."""
    if t_ is None:
        return 0, None
    one = isinstance(t_, _torch_module.Tensor) and t_.dim() == 2 and t_.shape[0] == 1
    return (1 if one else n), _state(t_, name, (1 if one else n, D), device)


def _cu(cu_seqlens, device):
    torch = _torch()
    _check(cu_seqlens, "cu_seqlens", device)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise TypeError("cu_seqlens must be int32 [n+1]")
    return cu_seqlens.numel() - 1


def gated_forward(x, log_a, state0=None, state_out=None, out=None, stream=None):
    """The gated linear recurrence, lla_gated_forward: h_t = exp(log_a_t) h_{t-1} + x_t, every channel by itself.
    Returns out [B,T,D], the states in x's type.

    x [B,T,D] (bf16 or fp32, any T and D >= 1); log_a [B,T,D], fp32 or x's type. ``state0`` fp32 [B,D], or [1,D] for
    one state shared by the batch; ``state_out`` fp32 [B,D] is written with the last state (see gated_decode_step)."""
    index, code, gate = _gated_inputs(x, log_a, dims=3)
    if stream is not None or index != _current_device():
        return _elsewhere(x.device, stream, gated_forward, x, log_a, state0, state_out, out)
    B, T, D = x.shape
    n0, s0 = _gated_state(state0, "state0", B, D, x.device)
    s1 = _state(state_out, "state_out", (B, D), x.device)
    o = _torch_module.empty_like(x) if out is None else _given(out, x)
    _call(load().lla_gated_forward(x.data_ptr(), log_a.data_ptr(), s0, o.data_ptr(), s1, B, n0, T, D, _raw_stream(index),
                                   code, gate), "lla_gated_forward")
    return o


def gated_forward_varlen(x, log_a, cu_seqlens, state0=None, state_out=None, out=None, stream=None):
    """lla_gated_forward_varlen: packed sequences. x, log_a [total,D]; cu_seqlens int32 [n+1] on the device; state0
    [n,D] or [1,D] (shared); state_out [n,D]. Rows of ``out`` that belong to no sequence are left as they were
    (uninitialised in a new ``out``)."""
    index, code, gate = _gated_inputs(x, log_a, dims=2)
    n = _cu(cu_seqlens, x.device)
    if stream is not None or index != _current_device():
        return _elsewhere(x.device, stream, gated_forward_varlen, x, log_a, cu_seqlens, state0, state_out, out)
    T, D = x.shape
    n0, s0 = _gated_state(state0, "state0", n, D, x.device)
    s1 = _state(state_out, "state_out", (n, D), x.device)
    o = _torch_module.empty_like(x) if out is None else _given(out, x)
    cu_seqlens = _small(cu_seqlens, "lla_gated_forward_varlen", o, state_out)
    _call(load().lla_gated_forward_varlen(x.data_ptr(), log_a.data_ptr(), s0, o.data_ptr(), s1, cu_seqlens.data_ptr(), n,
                                          n0, T, D, _raw_stream(index), code, gate), "lla_gated_forward_varlen")
    return o


def gated_backward(log_a, out, dout, state0=None, dstate_out=None, stream=None):
    """lla_gated_backward: gradients of sum(dout * out) + sum(dstate_out * state_out) of gated_forward, whose output
    is given as it was kept.

    Returns (dx, dlog_a, dstate0): dx in out's type, dlog_a in log_a's, dstate0 fp32 like state0 (None without one;
    summed over the batch where state0 is shared)."""
    index, code, gate = _gated_inputs(out, log_a, ("dout", dout), dims=3, name="out")
    if stream is not None or index != _current_device():
        return _elsewhere(out.device, stream, gated_backward, log_a, out, dout, state0, dstate_out)
    B, T, D = out.shape
    n0, s0 = _gated_state(state0, "state0", B, D, out.device)
    s1 = _state(dstate_out, "dstate_out", (B, D), out.device)
    dx, da = _torch_module.empty_like(out), _torch_module.empty_like(log_a)
    ds = None if state0 is None else _torch_module.empty_like(state0)
    _call(load().lla_gated_backward(log_a.data_ptr(), out.data_ptr(), s0, dout.data_ptr(), s1, dx.data_ptr(),
                                    da.data_ptr(), None if ds is None else ds.data_ptr(), B, n0, T, D,
                                    _raw_stream(index), code, gate), "lla_gated_backward")
    return dx, da, ds


def gated_backward_varlen(log_a, out, dout, cu_seqlens, state0=None, dstate_out=None, stream=None):
    """lla_gated_backward_varlen: gradients of packed sequences (see gated_forward_varlen); dstate_out [n,D]. Gradients
    of rows that belong to no sequence are 0."""
    index, code, gate = _gated_inputs(out, log_a, ("dout", dout), dims=2, name="out")
    n = _cu(cu_seqlens, out.device)
    if stream is not None or index != _current_device():
        return _elsewhere(out.device, stream, gated_backward_varlen, log_a, out, dout, cu_seqlens, state0, dstate_out)
    T, D = out.shape
    n0, s0 = _gated_state(state0, "state0", n, D, out.device)
    s1 = _state(dstate_out, "dstate_out", (n, D), out.device)
    dx, da = _torch_module.empty_like(out), _torch_module.empty_like(log_a)
    ds = None if state0 is None else _torch_module.empty_like(state0)
    cu_seqlens = _small(cu_seqlens, "lla_gated_backward_varlen")
    _call(load().lla_gated_backward_varlen(log_a.data_ptr(), out.data_ptr(), s0, dout.data_ptr(), s1, dx.data_ptr(),
                                           da.data_ptr(), None if ds is None else ds.data_ptr(), cu_seqlens.data_ptr(),
                                           n, n0, T, D, _raw_stream(index), code, gate), "lla_gated_backward_varlen")
    return dx, da, ds


def gated_decode_step(x, log_a, state, out=None, stream=None):
    """One token of every sequence, lla_gated_decode_step. x, log_a [B,D]; ``state`` [B,D] fp32 is updated in place.
    Returns out [B,D]."""
    index, code, gate = _gated_inputs(x, log_a, dims=2)
    if stream is not None or index != _current_device():
        return _elsewhere(x.device, stream, gated_decode_step, x, log_a, state, out)
    B, D = x.shape
    if not _fits(state, _torch_module.float32, x.shape, index):
        _want(state, "state", _torch_module.float32, x.shape, x.device)
    o = _torch_module.empty_like(x) if out is None else _given(out, x)
    _call(load().lla_gated_decode_step(x.data_ptr(), log_a.data_ptr(), state.data_ptr(), o.data_ptr(),
                                       _raw_stream(index), B, D, code, gate), "lla_gated_decode_step")
    return o


def _parent(parent, B, N, index, device):
    """Rows of a parent array: int32 [N] or [1,N] (one tree for the batch), or [B,N]."""
    torch = _torch()
    if _fits(parent, torch.int32, (B, N), index):
        return B
    if not (_fits(parent, torch.int32, (N,), index) or _fits(parent, torch.int32, (1, N), index)):
        _check(parent, "parent", device)
        raise ValueError(f"parent must be int32 [{N}] or [{B},{N}], got {parent.dtype} {list(parent.shape)}")
    return 1


def _accepted(count, path, B, index, device):
    """M of a commit: count int32 [B], path int32 [B,M] or None (M = 0)."""
    torch = _torch()
    if not _fits(count, torch.int32, (B,), index):
        _want(count, "count", torch.int32, (B,), device)
    if path is None:
        return 0
    if not isinstance(path, torch.Tensor):
        _check(path, "path")
    if path.dim() != 2 or path.shape[0] != B or path.shape[1] < 1:
        raise ValueError(f"path must be int32 [{B},M], got {list(path.shape)}")
    if not _fits(path, torch.int32, path.shape, index):
        _want(path, "path", torch.int32, path.shape, device)
    return path.shape[1]


def gated_decode_tree(x, log_a, state, parent, out=None, stream=None):
    """Outputs of a tree of drafted tokens, lla_gated_decode_tree: h_i = exp(log_a_i) h_parent(i) + x_i. x, log_a
    [B,N,D]; ``state`` [B,D] fp32 is read; ``parent`` int32 [N] or [B,N] (see decode_tree). Returns out [B,N,D]."""
    index, code, gate = _gated_inputs(x, log_a, dims=3)
    if stream is not None or index != _current_device():
        return _elsewhere(x.device, stream, gated_decode_tree, x, log_a, state, parent, out)
    B, N, D = x.shape
    if not _fits(state, _torch_module.float32, (B, D), index):
        _want(state, "state", _torch_module.float32, (B, D), x.device)
    trees = _parent(parent, B, N, index, x.device)
    o = _torch_module.empty_like(x) if out is None else _given(out, x)
    parent = _small(parent, "lla_gated_decode_tree", o)
    _call(load().lla_gated_decode_tree(x.data_ptr(), log_a.data_ptr(), state.data_ptr(), parent.data_ptr(), o.data_ptr(),
                                       _raw_stream(index), B, trees, N, D, code, gate), "lla_gated_decode_tree")
    return o


def gated_decode_commit(x, log_a, state, count, path=None, stream=None):
    """Accepted tokens into the states, lla_gated_decode_commit (see decode_commit). x, log_a [B,N,D]; ``state`` [B,D]
    fp32 is updated in place and returned."""
    index, code, gate = _gated_inputs(x, log_a, dims=3)
    if stream is not None or index != _current_device():
        return _elsewhere(x.device, stream, gated_decode_commit, x, log_a, state, count, path)
    B, N, D = x.shape
    if not _fits(state, _torch_module.float32, (B, D), index):
        _want(state, "state", _torch_module.float32, (B, D), x.device)
    M = _accepted(count, path, B, index, x.device)
    count = _small(count, "lla_gated_decode_commit", state)
    path = None if path is None else _small(path, "lla_gated_decode_commit", state)
    _call(load().lla_gated_decode_commit(x.data_ptr(), log_a.data_ptr(), state.data_ptr(), count.data_ptr(),
                                         None if path is None else path.data_ptr(), _raw_stream(index), B, N, M, D, code,
                                         gate), "lla_gated_decode_commit")
    return state


def _nodes(names, tokens, log_a, gates):
    """Says what is wrong with a tree's or a commit's tokens: q, k [B,H,N,dk], v [B,H,N,dv] of one dtype, log_a fp32."""
    v = tokens[-1]
    for n, t_ in zip(names, tokens):
        _check(t_, n, v.device if isinstance(v, _torch().Tensor) and v.is_cuda else None)
        if t_.dim() != 4:
            raise ValueError(f"{n} must have 4 dimensions, got {list(t_.shape)}")
    k = tokens[-2]
    for n, t_ in zip(names, tokens):
        _want(t_, n, k.dtype, tuple(k.shape[:3]) + (v.shape[3],) if n == "v" else k.shape, k.device)
    shape = gates(*k.shape[:3])
    _want(log_a, "log_a", _torch_module.float32, shape, k.device)


def _one_gate(B, H, N):
    return (H,)


def _node_gates(B, H, N):
    return (B, H, N)


def _places(where, written, *arrays):
    """Small arrays at the library's alignment (see _small)."""
    return [None if a is None else _small(a, where, written) for a in arrays]


def decode_tree(q, k, v, log_a, lam, states, t, parent, out=None, stream=None):
    """Outputs of a tree of drafted tokens over the states of decode_step, lla_decode_tree. Nothing but ``out`` is
    written: the accepted tokens go into the states with decode_commit.

    q, k [B,H,N,dk]; v [B,H,N,dv] (bf16 or fp32, N up to 128); log_a [B,H,N], lam [B,H,N,Lmax] fp32; ``states``
    [B,H,Lmax,dk,dv] fp32 with tokens 0..t-1, ``t`` int64 [B] on the device. ``parent`` int32 [N] (one tree for the
    batch) or [B,N] on the device: the node that a node goes on from, before it in the list, -1 for the last token of
    the states, -2 for no node (its row of ``out`` is left as it was; uninitialised in a new ``out``). Returns out
    [B,H,N,dv]."""
    torch = _torch()
    if not (type(q) is type(k) is type(v) is type(log_a) is torch.Tensor and q.dim() == v.dim() == 4):
        _nodes(("q", "k", "v"), (q, k, v), log_a, _node_gates)
    B, H, N, dk = q.shape
    dv, dtype, index = v.shape[3], q.dtype, q.get_device()
    if not isinstance(states, torch.Tensor) or states.dim() != 5:
        raise ValueError("states must be float32 [B,H,Lmax,dk,dv]")
    L = states.shape[2]
    if not (index >= 0 and k.dtype is dtype and v.dtype is dtype and k.shape == q.shape and v.shape == (B, H, N, dv)
            and log_a.dtype is torch.float32 and log_a.shape == (B, H, N) and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and log_a.is_contiguous()
            and k.get_device() == v.get_device() == log_a.get_device() == index
            and _fits(states, torch.float32, (B, H, L, dk, dv), index) and _fits(lam, torch.float32, (B, H, N, L), index)
            and _fits(t, torch.int64, (B,), index)):
        _nodes(("q", "k", "v"), (q, k, v), log_a, _node_gates)
        _want(states, "states", torch.float32, (B, H, L, dk, dv), q.device)
        _want(lam, "lambda", torch.float32, (B, H, N, L), q.device)
        _want(t, "t", torch.int64, (B,), q.device)
    if stream is not None or index != _current_device():
        return _elsewhere(q.device, stream, decode_tree, q, k, v, log_a, lam, states, t, parent, out)
    trees = _parent(parent, B, N, index, q.device)
    o = torch.empty_like(v) if out is None else _given(out, v)
    if (log_a.data_ptr() | lam.data_ptr() | t.data_ptr() | parent.data_ptr()) & 15:
        log_a, lam, t, parent = _places("lla_decode_tree", o, log_a, lam, t, parent)
    _call(load().lla_decode_tree(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), lam.data_ptr(),
                                 states.data_ptr(), t.data_ptr(), parent.data_ptr(), o.data_ptr(), _raw_stream(index), B,
                                 trees, H, N, dk, dv, L, _dtype_code(q)), "lla_decode_tree")
    return o


def decode_commit(k, v, log_a, states, t, count, path=None, stream=None):
    """Accepted tokens into the states of decode_step, lla_decode_commit: what a decode step for each would leave, in
    one pass. k [B,H,N,dk]; v [B,H,N,dv]; log_a [B,H,N] fp32, as decode_tree takes them; ``states`` [B,H,Lmax,dk,dv]
    fp32 is updated in place and returned; ``t`` int64 [B], not advanced (the caller adds ``count``).

    ``count`` int32 [B]: accepted tokens of each sequence (0: left as it is); ``path`` int32 [B,M]: their nodes in order
    (entries past count are not read); without it tokens 0..count-1."""
    torch = _torch()
    if not (type(k) is type(v) is type(log_a) is torch.Tensor and k.dim() == v.dim() == 4):
        _nodes(("k", "v"), (k, v), log_a, _node_gates)
    B, H, N, dk = k.shape
    dv, dtype, index = v.shape[3], k.dtype, k.get_device()
    if not isinstance(states, torch.Tensor) or states.dim() != 5:
        raise ValueError("states must be float32 [B,H,Lmax,dk,dv]")
    L = states.shape[2]
    if not (index >= 0 and v.dtype is dtype and v.shape == (B, H, N, dv) and log_a.dtype is torch.float32
            and log_a.shape == (B, H, N) and k.is_contiguous() and v.is_contiguous() and log_a.is_contiguous()
            and v.get_device() == log_a.get_device() == index and _fits(states, torch.float32, (B, H, L, dk, dv), index)
            and _fits(t, torch.int64, (B,), index)):
        _nodes(("k", "v"), (k, v), log_a, _node_gates)
        _want(states, "states", torch.float32, (B, H, L, dk, dv), k.device)
        _want(t, "t", torch.int64, (B,), k.device)
    if stream is not None or index != _current_device():
        return _elsewhere(k.device, stream, decode_commit, k, v, log_a, states, t, count, path)
    M = _accepted(count, path, B, index, k.device)
    at = 0 if path is None else path.data_ptr()
    if (log_a.data_ptr() | t.data_ptr() | count.data_ptr() | at) & 15:
        log_a, t, count, path = _places("lla_decode_commit", states, log_a, t, count, path)
    _call(load().lla_decode_commit(k.data_ptr(), v.data_ptr(), log_a.data_ptr(), states.data_ptr(), t.data_ptr(),
                                   count.data_ptr(), None if path is None else path.data_ptr(), _raw_stream(index), B, H,
                                   N, M, dk, dv, L, _dtype_code(k)), "lla_decode_commit")
    return states


def linear_decode_tree(q, k, v, log_a, state, parent, out=None, stream=None):
    """Outputs of a tree of drafted tokens over the state of linear_decode_step, lla_linear_decode_tree (see
    decode_tree). log_a [H] fp32; ``state`` [B,H,dk,dv] fp32 is read. Returns out [B,H,N,dv]."""
    torch = _torch()
    if not (type(q) is type(k) is type(v) is type(log_a) is torch.Tensor and q.dim() == v.dim() == 4):
        _nodes(("q", "k", "v"), (q, k, v), log_a, _one_gate)
    B, H, N, dk = q.shape
    dv, dtype, index = v.shape[3], q.dtype, q.get_device()
    if not (index >= 0 and k.dtype is dtype and v.dtype is dtype and k.shape == q.shape and v.shape == (B, H, N, dv)
            and log_a.dtype is torch.float32 and log_a.shape == (H,) and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and log_a.is_contiguous()
            and k.get_device() == v.get_device() == log_a.get_device() == index
            and _fits(state, torch.float32, (B, H, dk, dv), index)):
        _nodes(("q", "k", "v"), (q, k, v), log_a, _one_gate)
        _want(state, "state", torch.float32, (B, H, dk, dv), q.device)
    if stream is not None or index != _current_device():
        return _elsewhere(q.device, stream, linear_decode_tree, q, k, v, log_a, state, parent, out)
    trees = _parent(parent, B, N, index, q.device)
    o = torch.empty_like(v) if out is None else _given(out, v)
    if (log_a.data_ptr() | parent.data_ptr()) & 15:
        log_a, parent = _places("lla_linear_decode_tree", o, log_a, parent)
    _call(load().lla_linear_decode_tree(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_a.data_ptr(), state.data_ptr(),
                                        parent.data_ptr(), o.data_ptr(), _raw_stream(index), B, trees, H, N, dk, dv,
                                        _dtype_code(q)), "lla_linear_decode_tree")
    return o


def linear_decode_commit(k, v, log_a, state, count, path=None, stream=None):
    """Accepted tokens into the state of linear_decode_step, lla_linear_decode_commit (see decode_commit). log_a [H]
    fp32; ``state`` [B,H,dk,dv] fp32 is updated in place and returned."""
    torch = _torch()
    if not (type(k) is type(v) is type(log_a) is torch.Tensor and k.dim() == v.dim() == 4):
        _nodes(("k", "v"), (k, v), log_a, _one_gate)
    B, H, N, dk = k.shape
    dv, dtype, index = v.shape[3], k.dtype, k.get_device()
    if not (index >= 0 and v.dtype is dtype and v.shape == (B, H, N, dv) and log_a.dtype is torch.float32
            and log_a.shape == (H,) and k.is_contiguous() and v.is_contiguous() and log_a.is_contiguous()
            and v.get_device() == log_a.get_device() == index and _fits(state, torch.float32, (B, H, dk, dv), index)):
        _nodes(("k", "v"), (k, v), log_a, _one_gate)
        _want(state, "state", torch.float32, (B, H, dk, dv), k.device)
    if stream is not None or index != _current_device():
        return _elsewhere(k.device, stream, linear_decode_commit, k, v, log_a, state, count, path)
    M = _accepted(count, path, B, index, k.device)
    at = 0 if path is None else path.data_ptr()
    if (log_a.data_ptr() | count.data_ptr() | at) & 15:
        log_a, count, path = _places("lla_linear_decode_commit", state, log_a, count, path)
    _call(load().lla_linear_decode_commit(k.data_ptr(), v.data_ptr(), log_a.data_ptr(), state.data_ptr(),
                                          count.data_ptr(), None if path is None else path.data_ptr(),
                                          _raw_stream(index), B, H, N, M, dk, dv, _dtype_code(k)),
          "lla_linear_decode_commit")
    return state
