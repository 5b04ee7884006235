"""Python binding of the retention C ABI (``include/retention.h``).

Argument marshalling only: every step of retention runs in the CUDA kernels
of ``libretention.so``.  PyTorch supplies device memory and the stream.  If
the library has not been built this module raises at import; there is no
fallback implementation.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import functools
import operator
import os

import torch

from . import build as _build

F32, BF16 = 0, 1
NORM_SCALE, NORM_DROW, NORM_RSUM = 1, 2, 4
NORM_ALL = NORM_SCALE | NORM_DROW | NORM_RSUM
STATUS = {0: "RET_OK", 1: "RET_EINVAL", 2: "RET_EUNSUPPORTED", 3: "RET_EWORKSPACE",
          4: "RET_ECUDA", 5: "RET_ETIMEOUT"}
MAX_HEADS = 256

MAX_TOP = 128
MAX_STATES = 64

_I64x2 = ctypes.c_int64 * 2
_I64x3 = ctypes.c_int64 * 3


class RetDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int),
                ("d_k", ctypes.c_int), ("d_v", ctypes.c_int), ("chunk", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("gamma", ctypes.POINTER(ctypes.c_double)),
                ("theta_base", ctypes.c_double), ("norm_flags", ctypes.c_int),
                ("gn_eps", ctypes.c_float), ("pos0", ctypes.c_int64),
                ("rotate", ctypes.c_int),
                ("sq", _I64x3), ("sk", _I64x3), ("sv", _I64x3), ("so", _I64x3)]


class MsrDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("d_model", ctypes.c_int),
                ("H", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
                ("chunk", ctypes.c_int), ("gamma", ctypes.POINTER(ctypes.c_double)),
                ("theta_base", ctypes.c_double), ("norm_flags", ctypes.c_int),
                ("gn_eps", ctypes.c_float), ("pos0", ctypes.c_int64)]


class BlockDesc(ctypes.Structure):
    _fields_ = [("msr", MsrDesc), ("d_ffn", ctypes.c_int), ("ln_eps", ctypes.c_float)]


class StackDesc(ctypes.Structure):
    _fields_ = [("block", BlockDesc), ("n_layers", ctypes.c_int)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("n0", ctypes.c_int64), ("n1", ctypes.c_int64), ("d", ctypes.c_int),
                ("dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("sx", _I64x2), ("sg", _I64x2), ("so", _I64x2)]


class LogitsDesc(ctypes.Structure):
    _fields_ = [("n0", ctypes.c_int64), ("n1", ctypes.c_int64), ("V", ctypes.c_int),
                ("dtype", ctypes.c_int), ("temperature", ctypes.c_double), ("top", ctypes.c_int),
                ("id_bytes", ctypes.c_int), ("tail", ctypes.c_int),
                ("sx", _I64x2), ("sd", _I64x2)]


class ScanDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("E", ctypes.c_int),
                ("S", ctypes.c_int), ("G", ctypes.c_int), ("dtype", ctypes.c_int),
                ("softplus", ctypes.c_int), ("len_bytes", ctypes.c_int),
                ("sx", _I64x2), ("sdt", _I64x2), ("sz", _I64x2), ("sy", _I64x2),
                ("sdy", _I64x2), ("sdx", _I64x2), ("sddt", _I64x2), ("sdz", _I64x2),
                ("sB", _I64x3), ("sC", _I64x3)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("E", ctypes.c_int),
                ("W", ctypes.c_int), ("dtype", ctypes.c_int), ("silu", ctypes.c_int),
                ("len_bytes", ctypes.c_int), ("sx", _I64x2), ("sg", _I64x2), ("so", _I64x2)]


class RmsNormDesc(ctypes.Structure):
    _fields_ = [("n0", ctypes.c_int64), ("n1", ctypes.c_int64), ("d", ctypes.c_int),
                ("dtype", ctypes.c_int), ("eps", ctypes.c_float), ("group", ctypes.c_int),
                ("sx", _I64x2), ("sr", _I64x2), ("sh", _I64x2), ("sg", _I64x2), ("so", _I64x2)]


LAYER_KEYS = ("ln1_w", "ln1_b", "WQ", "WK", "WV", "WG", "WO", "ln2_w", "ln2_b", "W1", "W2")


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LAYER_KEYS]


# Every symbol include/retention.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_SIGS = {
    "retention_desc_init": (None, [ctypes.POINTER(RetDesc), ctypes.c_int, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                   ctypes.POINTER(ctypes.c_double)]),
    "retention_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(RetDesc)]),
    "retention_rotate": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P,
                                        ctypes.POINTER(ctypes.c_int64), ctypes.c_int, _P,
                                        ctypes.c_int, _P, _P]),
    "retention_parallel_fwd": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P, _P, _P, _P, _P,
                                              ctypes.c_size_t, _P]),
    "retention_chunkwise_fwd": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P, _P, _P, _P, _P,
                                               _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "retention_recurrent_step": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P, _P, _P, _P, _P,
                                                _P, _P, ctypes.c_size_t, _P]),
    "retention_chunkwise_fwd_noalloc": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P, _P, _P, _P,
                                                       _P, _P, _P, _P, _P]),
    "retention_state_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(RetDesc)]),
    "retention_chunkwise_state": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P, _P, _P, _P, _P,
                                                 _P, _P, ctypes.c_size_t, _P]),
    "retention_state_combine": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                               ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                               ctypes.c_int, ctypes.POINTER(ctypes.c_void_p),
                                               ctypes.POINTER(ctypes.c_void_p),
                                               ctypes.POINTER(ctypes.c_int64), _P, _P, _P]),
    "retention_backward_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(RetDesc)]),
    "retention_chunkwise_bwd": (ctypes.c_int, [ctypes.POINTER(RetDesc), _P, _P, _P, _P, _P,
                                               _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "msr_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(MsrDesc)]),
    "retention_gemm_workspace_size": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int,
                                                        ctypes.c_int]),
    "retention_gemm_bf16": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           _P, ctypes.c_size_t, _P]),
    "msr_layer_fwd": (ctypes.c_int, [ctypes.POINTER(MsrDesc), _P, _P, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]),
    "retnet_block_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(BlockDesc)]),
    "retnet_block_fwd": (ctypes.c_int, [ctypes.POINTER(BlockDesc)] + [_P] * 14 +
                         [ctypes.c_size_t, _P]),
    "retnet_decode_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(StackDesc)]),
    "retnet_decode_step": (ctypes.c_int, [ctypes.POINTER(StackDesc), ctypes.POINTER(LayerWeights),
                                          ctypes.POINTER(ctypes.c_void_p),
                                          ctypes.POINTER(ctypes.c_void_p), _P, _P,
                                          ctypes.c_size_t, _P]),
    "retnet_layernorm_fwd": (ctypes.c_int, [ctypes.POINTER(LayerNormDesc)] + [_P] * 7),
    "retnet_layernorm_bwd_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LayerNormDesc)]),
    "retnet_layernorm_bwd": (ctypes.c_int, [ctypes.POINTER(LayerNormDesc)] + [_P] * 9 +
                             [ctypes.c_size_t, _P]),
    "retnet_token_logprobs": (ctypes.c_int, [ctypes.POINTER(LogitsDesc)] + [_P] * 7),
    "retnet_distill_fwd": (ctypes.c_int, [ctypes.POINTER(LogitsDesc)] + [_P] * 6),
    "retnet_distill_bwd": (ctypes.c_int, [ctypes.POINTER(LogitsDesc)] + [_P] * 7),
    "retnet_distill_step": (ctypes.c_int, [ctypes.POINTER(LogitsDesc)] + [_P] * 8),
    "retnet_selective_scan_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(ScanDesc)]),
    "retnet_selective_scan_fwd": (ctypes.c_int, [ctypes.POINTER(ScanDesc)] + [_P] * 13 +
                                  [ctypes.c_size_t, _P]),
    "retnet_selective_scan_step": (ctypes.c_int, [ctypes.POINTER(ScanDesc)] + [_P] * 12),
    "retnet_selective_scan_bwd_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(ScanDesc)]),
    "retnet_selective_scan_bwd": (ctypes.c_int, [ctypes.POINTER(ScanDesc)] + [_P] * 22 +
                                  [ctypes.c_size_t, _P]),
    "retnet_causal_conv_fwd": (ctypes.c_int, [ctypes.POINTER(ConvDesc)] + [_P] * 8),
    "retnet_causal_conv_bwd_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(ConvDesc)]),
    "retnet_causal_conv_bwd": (ctypes.c_int, [ctypes.POINTER(ConvDesc)] + [_P] * 12 +
                               [ctypes.c_size_t, _P]),
    "retnet_rmsnorm_fwd": (ctypes.c_int, [ctypes.POINTER(RmsNormDesc)] + [_P] * 7),
    "retnet_rmsnorm_quant": (ctypes.c_int, [ctypes.POINTER(RmsNormDesc)] + [_P] * 7),
    "retnet_rmsnorm_bwd_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(RmsNormDesc)]),
    "retnet_rmsnorm_bwd": (ctypes.c_int, [ctypes.POINTER(RmsNormDesc)] + [_P] * 8 +
                           [ctypes.c_size_t, _P]),
    "retention_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "retention_last_cuda_error": (ctypes.c_int, []),
    "retention_poll_status": (ctypes.c_int, [_P, _P]),
    "retention_kernel_timer_enable": (None, [ctypes.c_int]),
    "retention_set_report_wait_budget": (None, [ctypes.c_uint]),
    "retention_kernel_timer_reset": (None, []),
    "retention_kernel_count": (ctypes.c_int, []),
    "retention_kernel_name": (ctypes.c_char_p, [ctypes.c_int]),
    "retention_launch_count": (ctypes.c_longlong, []),
    "retention_tc_probe": (ctypes.c_int, [ctypes.c_int] * 9 + [_P, _P, _P, _P, _P]),
    "retention_tc_probe_scale_d": (ctypes.c_int, [ctypes.c_int, _P, _P, _P, _P, _P]),
    "retention_tc_probe_pair": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + [_P] * 6),
    "retention_kernel_timer_read": (ctypes.c_int, [ctypes.c_int,
                                                   ctypes.POINTER(ctypes.c_double),
                                                   ctypes.POINTER(ctypes.c_longlong),
                                                   ctypes.POINTER(ctypes.c_int)]),
}


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"CUDA library not built: {path} is missing "
                          "(run __graft_entry__.build() or linear_recurrent_sequence_gb300/build.py)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


lib = _load()


class RetentionError(RuntimeError):
    def __init__(self, status, where):
        msg = lib.retention_status_string(status).decode()
        if status == 4:
            msg += f" (cudaError {lib.retention_last_cuda_error()})"
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")
        self.status = status


def _check(status, where):
    if status != 0:
        raise RetentionError(status, where)


def _ptr(t):
    """Device address of a tensor for the C ABI.  Only CUDA tensors on the
    current device are accepted: any other address would reach a kernel."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device)")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object around it, where this
# torch has that (3 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {dt}")


def _bhnd_strides(t, name):
    """Element strides (b, h, n) of a [B, H, N, d] tensor with unit feature stride."""
    if t.dim() != 4:
        raise ValueError(f"{name} must be 4-D [B,H,N,d], got {tuple(t.shape)}")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}: the feature dimension must be contiguous")
    return (t.stride(0), t.stride(1), t.stride(2))


class _Gamma:
    """Keeps a float64 host copy of the decays alive for the call."""

    def __init__(self, gamma, H):
        import numpy as np
        g = np.ascontiguousarray(np.broadcast_to(np.asarray(gamma, dtype=np.float64), (H,)))
        self.arr = g
        self.ptr = g.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def make_desc(q, k, v, o, gamma, *, chunk=64, norm_flags=0, gn_eps=1e-6, pos0=0,
              rotate=True, theta_base=10000.0):
    B, H, N, dk = q.shape
    dv = v.shape[3]
    g = _Gamma(gamma, H)
    d = RetDesc()
    d.B, d.H, d.N, d.d_k, d.d_v, d.chunk = B, H, N, dk, dv, int(chunk)
    d.in_dtype = _dtype_code(q.dtype)
    d.out_dtype = _dtype_code(o.dtype)
    d.gamma = g.ptr
    d.theta_base = float(theta_base)
    d.norm_flags = int(norm_flags)
    d.gn_eps = float(-1.0 if gn_eps is None else gn_eps)
    d.pos0 = int(pos0)
    d.rotate = int(bool(rotate))
    d.sq = _I64x3(*_bhnd_strides(q, "q"))
    d.sk = _I64x3(*_bhnd_strides(k, "k"))
    d.sv = _I64x3(*_bhnd_strides(v, "v"))
    d.so = _I64x3(*_bhnd_strides(o, "o"))
    return d, g


def workspace_size(desc):
    return int(lib.retention_workspace_size(ctypes.byref(desc)))


def _on(stream):
    """Context in which memory for one call is allocated: in the order of the
    stream that the call runs on.  A block of the current stream's would be given
    to its next allocation as soon as the call returns, and would be zeroed at
    any time, while a call on another stream still uses it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _empty(stream, shape, dtype, device, strides=None):
    """Memory of an output that the caller gave none for.  Like a workspace it
    belongs to the stream that the call runs on: the caller may drop an output at
    once, and its block then goes to what follows on that stream.  The current
    stream, where the caller goes on with the output, is noted as a user, so that a
    block freed after its last use there waits for that."""
    if stream is None and strides is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        t = (torch.empty(shape, dtype=dtype, device=device) if strides is None else
             torch.empty_strided(shape, strides, dtype=dtype, device=device))
    if stream is not None and t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def new_workspace(nbytes, device, stream=None):
    """A workspace for calls on the given stream (None: the current one)."""
    # zeroed once: its first bytes hold the device status word
    with _on(stream):
        return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _prep(q, k, v, out, out_dtype, stream):
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        B, H, N, _ = q.shape
        out = _empty(stream, (B, H, N, v.shape[3]), out_dtype or q.dtype, q.device)
    return out


def chunkwise_fwd(q, k, v, gamma, *, chunk=64, norm_flags=0, gn_eps=1e-6, pos0=0,
                  rotate=True, theta_base=10000.0, S_in=None, z_in=None, S_out=None,
                  z_out=None, out=None, out_dtype=None, workspace=None, stream=None):
    """Chunkwise retention forward; q,k [B,H,N,d_k], v [B,H,N,d_v] (any strides
    with a contiguous feature dimension).  Returns the output tensor."""
    out = _prep(q, k, v, out, out_dtype, stream)
    d, g = make_desc(q, k, v, out, gamma, chunk=chunk, norm_flags=norm_flags, gn_eps=gn_eps,
                     pos0=pos0, rotate=rotate, theta_base=theta_base)
    if workspace is None:
        workspace = new_workspace(workspace_size(d), q.device, stream)
    st = lib.retention_chunkwise_fwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(S_in),
                                     _ptr(z_in), _ptr(S_out), _ptr(z_out), _ptr(out),
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "retention_chunkwise_fwd")
    return out


def state_workspace_size(desc):
    return int(lib.retention_state_workspace_size(ctypes.byref(desc)))


def chunkwise_state(k, v, gamma, *, pos0=0, rotate=True, theta_base=10000.0, S_in=None,
                    z_in=None, S_out=None, z_out=None, with_z=True, workspace=None,
                    stream=None):
    """The recurrent state after the tokens of k [B,H,N,d_k], v [B,H,N,d_v]
    (no outputs): S = gamma^N S_in + sum_m gamma^(N-1-m) K'_m^T V_m and z
    likewise.  Returns (S_out, z_out); z_out is None when with_z is False."""
    B, H, N, dk = k.shape
    dv = v.shape[3]
    if S_out is None:
        S_out = _empty(stream, (B, H, dk, dv), torch.float32, k.device)
    if with_z and z_out is None:
        z_out = _empty(stream, (B, H, dk), torch.float32, k.device)
    d, g = make_desc(k, k, v, v, gamma, pos0=pos0, rotate=rotate, theta_base=theta_base)
    if workspace is None:
        workspace = new_workspace(state_workspace_size(d), k.device, stream)
    st = lib.retention_chunkwise_state(ctypes.byref(d), _ptr(k), _ptr(v), _ptr(S_in),
                                       _ptr(z_in), _ptr(S_out), _ptr(z_out), _ptr(workspace),
                                       workspace.numel(), _stream(stream))
    _check(st, "retention_chunkwise_state")
    return S_out, (z_out if with_z else None)


def state_combine(parts, tokens, gamma, *, S_out, z_out=None, stream=None):
    """S_out = sum_i gamma_h^(tokens[i]) S_i (z likewise) over parts, a list of
    (S_i, z_i) pairs of fp32 device tensors (None for a zero state)."""
    B, H, dk, dv = S_out.shape
    n = len(parts)
    Sp = (ctypes.c_void_p * max(n, 1))(*[_ptr(S) for S, _ in parts])
    zp = (ctypes.c_void_p * max(n, 1))(*[_ptr(z) for _, z in parts])
    tk = (ctypes.c_int64 * max(n, 1))(*[int(t) for t in tokens])
    g = (ctypes.c_double * H)(*[float(x) for x in gamma])
    st = lib.retention_state_combine(B, H, dk, dv, g, n, Sp, zp, tk, _ptr(S_out), _ptr(z_out),
                                     _stream(stream))
    _check(st, "retention_state_combine")
    return S_out, z_out


def backward_workspace_size(desc):
    return int(lib.retention_backward_workspace_size(ctypes.byref(desc)))


def chunkwise_bwd(q, k, v, dO, gamma, *, norm_flags=0, pos0=0, rotate=True,
                  theta_base=10000.0, S_in=None, dS_out=None, dS_in=None, dq=None, dk=None,
                  dv=None, workspace=None, stream=None):
    """Gradients of retention without GroupNorm (gn_eps < 0) and without the
    third normalisation: returns (dq, dk, dv, dS_in).  dq, dk, dv take the
    layouts and dtype of q, k, v; dS_in (fp32 [B,H,d_k,d_v]) is returned only
    when passed in (it may be dS_out itself)."""
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")

    def like(x, given, name):
        if given is None:
            return _empty(stream, x.shape, x.dtype, x.device, x.stride())
        if given.shape != x.shape or given.stride() != x.stride() or given.dtype != x.dtype:
            raise ValueError(f"{name} must have the shape, strides and dtype of its input")
        return given

    dq, dk, dv = like(q, dq, "dq"), like(k, dk, "dk"), like(v, dv, "dv")
    d, g = make_desc(q, k, v, dO, gamma, norm_flags=norm_flags, gn_eps=None, pos0=pos0,
                     rotate=rotate, theta_base=theta_base)
    if workspace is None:
        workspace = new_workspace(backward_workspace_size(d), q.device, stream)
    st = lib.retention_chunkwise_bwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(S_in),
                                     _ptr(dO), _ptr(dS_out), _ptr(dq), _ptr(dk), _ptr(dv),
                                     _ptr(dS_in), _ptr(workspace), workspace.numel(),
                                     _stream(stream))
    _check(st, "retention_chunkwise_bwd")
    return dq, dk, dv, dS_in


def chunkwise_fwd_noalloc(q, k, v, gamma, *, chunk=64, norm_flags=0, gn_eps=1e-6, pos0=0,
                          rotate=True, theta_base=10000.0, S_in=None, z_in=None, S_out=None,
                          z_out=None, out=None, out_dtype=None, stream=None):
    """Chunkwise forward whose workspace is the library's own fixed device
    array (for callers that cannot allocate); see retention.h."""
    out = _prep(q, k, v, out, out_dtype, stream)
    d, g = make_desc(q, k, v, out, gamma, chunk=chunk, norm_flags=norm_flags, gn_eps=gn_eps,
                     pos0=pos0, rotate=rotate, theta_base=theta_base)
    st = lib.retention_chunkwise_fwd_noalloc(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v),
                                             _ptr(S_in), _ptr(z_in), _ptr(S_out), _ptr(z_out),
                                             _ptr(out), _stream(stream))
    _check(st, "retention_chunkwise_fwd_noalloc")
    return out


def parallel_fwd(q, k, v, gamma, *, norm_flags=0, gn_eps=1e-6, pos0=0, rotate=True,
                 theta_base=10000.0, out=None, out_dtype=None, workspace=None, stream=None):
    out = _prep(q, k, v, out, out_dtype, stream)
    d, g = make_desc(q, k, v, out, gamma, norm_flags=norm_flags, gn_eps=gn_eps, pos0=pos0,
                     rotate=rotate, theta_base=theta_base)
    if workspace is None:
        workspace = new_workspace(workspace_size(d), q.device, stream)
    st = lib.retention_parallel_fwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                    _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "retention_parallel_fwd")
    return out


def recurrent_step(q, k, v, S, gamma, *, z=None, pos, norm_flags=0, gn_eps=1e-6,
                   rotate=True, theta_base=10000.0, out=None, out_dtype=None,
                   workspace=None, stream=None):
    """One decode step at absolute position ``pos``.  q,k [B,H,d_k], v [B,H,d_v]
    (or with a length-1 token axis); S fp32 [B,H,d_k,d_v] updated in place."""
    q4 = q if q.dim() == 4 else q.unsqueeze(2)
    k4 = k if k.dim() == 4 else k.unsqueeze(2)
    v4 = v if v.dim() == 4 else v.unsqueeze(2)
    out = _prep(q4, k4, v4, out if out is None or out.dim() == 4 else out.unsqueeze(2), out_dtype,
                stream)
    d, g = make_desc(q4, k4, v4, out, gamma, norm_flags=norm_flags, gn_eps=gn_eps, pos0=pos,
                     rotate=rotate, theta_base=theta_base)
    if workspace is None:
        workspace = new_workspace(256, q.device, stream)
    st = lib.retention_recurrent_step(ctypes.byref(d), _ptr(q4), _ptr(k4), _ptr(v4), _ptr(S),
                                      _ptr(z), _ptr(out), _ptr(workspace), workspace.numel(),
                                      _stream(stream))
    _check(st, "retention_recurrent_step")
    return out


def rotate(x, *, pos0=0, theta_base=10000.0, scale=None, out_dtype=None, stream=None):
    """Theta applied to x [B,H,N,d]; returns a contiguous tensor."""
    B, H, N, dd = x.shape
    out = _empty(stream, (B, H, N, dd), out_dtype or x.dtype, x.device)
    d, g = make_desc(x, x, x[..., :2], out[..., :2], [1.0] * H, pos0=pos0,
                     theta_base=theta_base)
    sx = _I64x3(*_bhnd_strides(x, "x"))
    st = lib.retention_rotate(ctypes.byref(d), _ptr(x), sx, dd, _ptr(out),
                              _dtype_code(out.dtype), _ptr(scale), _stream(stream))
    _check(st, "retention_rotate")
    return out


def msr_desc(B, N, d_model, H, d_k, d_v, gamma, *, chunk=128, norm_flags=0, gn_eps=1e-6,
             pos0=0, theta_base=10000.0):
    g = _Gamma(gamma, H)
    m = MsrDesc()
    m.B, m.N, m.d_model, m.H, m.d_k, m.d_v, m.chunk = B, N, d_model, H, d_k, d_v, chunk
    m.gamma = g.ptr
    m.theta_base = float(theta_base)
    m.norm_flags = int(norm_flags)
    m.gn_eps = float(-1.0 if gn_eps is None else gn_eps)
    m.pos0 = int(pos0)
    return m, g


def msr_layer_fwd(X, WQ, WK, WV, WG, WO, *, H, d_k, d_v, gamma, chunk=128, norm_flags=0,
                  gn_eps=1e-6, pos0=0, theta_base=10000.0, out=None, workspace=None,
                  stream=None):
    B, N, dm = X.shape
    m, g = msr_desc(B, N, dm, H, d_k, d_v, gamma, chunk=chunk, norm_flags=norm_flags,
                    gn_eps=gn_eps, pos0=pos0, theta_base=theta_base)
    if out is None:
        out = _empty(stream, (B, N, dm), torch.bfloat16, X.device)
    if workspace is None:
        workspace = new_workspace(int(lib.msr_workspace_size(ctypes.byref(m))), X.device, stream)
    for name, t in (("X", X), ("WQ", WQ), ("WK", WK), ("WV", WV), ("WG", WG), ("WO", WO)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor")
    st = lib.msr_layer_fwd(ctypes.byref(m), _ptr(X), _ptr(WQ), _ptr(WK), _ptr(WV), _ptr(WG),
                           _ptr(WO), _ptr(out), _ptr(workspace), workspace.numel(),
                           _stream(stream))
    _check(st, "msr_layer_fwd")
    return out


def block_desc(B, N, d_model, H, d_k, d_v, d_ffn, gamma, *, chunk=128, norm_flags=0,
               gn_eps=1e-6, ln_eps=1e-5, pos0=0, theta_base=10000.0):
    m, g = msr_desc(B, N, d_model, H, d_k, d_v, gamma, chunk=chunk, norm_flags=norm_flags,
                    gn_eps=gn_eps, pos0=pos0, theta_base=theta_base)
    d = BlockDesc()
    d.msr = m
    d.d_ffn = int(d_ffn)
    d.ln_eps = float(ln_eps)
    return d, g


def retnet_block_fwd(X, ln1_w, ln1_b, WQ, WK, WV, WG, WO, ln2_w, ln2_b, W1, W2, *, H, d_k, d_v,
                     gamma, chunk=128, norm_flags=0, gn_eps=1e-6, ln_eps=1e-5, pos0=0,
                     theta_base=10000.0, out=None, workspace=None, stream=None):
    """One RetNet block: Y = MSR(LN1(X)) + X, X' = gelu(LN2(Y) W1) W2 + Y.
    bf16 activations and weights, fp32 LayerNorm gains and biases."""
    B, N, dm = X.shape
    d, g = block_desc(B, N, dm, H, d_k, d_v, W1.shape[1], gamma, chunk=chunk,
                      norm_flags=norm_flags, gn_eps=gn_eps, ln_eps=ln_eps, pos0=pos0,
                      theta_base=theta_base)
    if out is None:
        out = _empty(stream, (B, N, dm), torch.bfloat16, X.device)
    if workspace is None:
        workspace = new_workspace(int(lib.retnet_block_workspace_size(ctypes.byref(d))),
                                  X.device, stream)
    for name, t in (("X", X), ("WQ", WQ), ("WK", WK), ("WV", WV), ("WG", WG), ("WO", WO),
                    ("W1", W1), ("W2", W2)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor")
    for name, t in (("ln1_w", ln1_w), ("ln1_b", ln1_b), ("ln2_w", ln2_w), ("ln2_b", ln2_b)):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != dm:
            raise ValueError(f"{name} must be a contiguous fp32 tensor of d_model values")
    st = lib.retnet_block_fwd(ctypes.byref(d), _ptr(X), _ptr(ln1_w), _ptr(ln1_b), _ptr(WQ),
                              _ptr(WK), _ptr(WV), _ptr(WG), _ptr(WO), _ptr(ln2_w), _ptr(ln2_b),
                              _ptr(W1), _ptr(W2), _ptr(out), _ptr(workspace), workspace.numel(),
                              _stream(stream))
    _check(st, "retnet_block_fwd")
    return out


def stack_desc(B, d_model, H, d_k, d_v, d_ffn, n_layers, gamma, *, pos, norm_flags=0,
               gn_eps=1e-6, ln_eps=1e-5, theta_base=10000.0):
    b, g = block_desc(B, 1, d_model, H, d_k, d_v, d_ffn, gamma, norm_flags=norm_flags,
                      gn_eps=gn_eps, ln_eps=ln_eps, pos0=pos, theta_base=theta_base)
    d = StackDesc()
    d.block = b
    d.n_layers = int(n_layers)
    return d, g


def retnet_decode_step(X, layers, S, z=None, *, H, d_k, d_v, gamma, pos, norm_flags=0,
                       gn_eps=1e-6, ln_eps=1e-5, theta_base=10000.0, workspace=None,
                       stream=None):
    """One decode step of a stack of RetNet blocks: X [B, d_model] bf16 is the
    token's input and is overwritten with the stack's output; `layers` is a
    list of dicts with the keys LAYER_KEYS (bf16 weights, fp32 LayerNorm
    gains and biases); S (and z, with the third normalisation) lists of the
    layers' fp32 states, updated in place."""
    if X.dim() != 2 or X.dtype != torch.bfloat16 or not X.is_contiguous():
        raise ValueError("X must be a contiguous bf16 [B, d_model] tensor")
    B, dm = X.shape
    n = len(layers)
    if len(S) != n or (z is not None and len(z) != n):
        raise ValueError("one state per layer")
    d_ffn = layers[0]["W1"].shape[1] if n else 1
    d, g = stack_desc(B, dm, H, d_k, d_v, d_ffn, n, gamma, pos=pos, norm_flags=norm_flags,
                      gn_eps=gn_eps, ln_eps=ln_eps, theta_base=theta_base)
    if workspace is None:
        workspace = new_workspace(int(lib.retnet_decode_workspace_size(ctypes.byref(d))),
                                  X.device, stream)
    recs = (LayerWeights * max(n, 1))()
    for i, L in enumerate(layers):
        for k in LAYER_KEYS:
            t = L[k]
            want = torch.float32 if k.startswith("ln") else torch.bfloat16
            if t.dtype != want or not t.is_contiguous():
                raise ValueError(f"layer {i} {k}: contiguous {want} expected")
        for k, p in zip(LAYER_KEYS, _ptrs(*(L[k] for k in LAYER_KEYS))):
            setattr(recs[i], k, p)
    Sp = (ctypes.c_void_p * max(n, 1))(*_ptrs(*S))
    zp = None if z is None else (ctypes.c_void_p * max(n, 1))(*_ptrs(*z))
    st = lib.retnet_decode_step(ctypes.byref(d), recs, Sp, zp, _ptr(X), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check(st, "retnet_decode_step")
    return X


def gemm_bf16(A, B, out=None, workspace=None, stream=None):
    """C = A @ B for bf16 row-major matrices (the MSR projections' GEMM)."""
    M, K = A.shape
    N = B.shape[1]
    if out is None:
        out = _empty(stream, (M, N), torch.bfloat16, A.device)
    if workspace is None:
        workspace = new_workspace(int(lib.retention_gemm_workspace_size(M, N, K)), A.device,
                                  stream)
    _check(lib.retention_gemm_bf16(_ptr(A), _ptr(B), _ptr(out), M, N, K, _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "retention_gemm_bf16")
    return out


def _row_strides(name, shape, *strides):
    """(n0, n1) and the two element strides of each tensor for rows along the
    last dimension, from their common shape and their strides.  More than two
    leading dimensions are folded where every tensor's strides allow it."""
    lead = shape[:-1]
    for s in strides:
        if s[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
    if 0 in lead:
        return 0, 0, [(0, 0)] * len(strides)
    dims = [(n, [s[i] for s in strides]) for i, n in enumerate(lead) if n != 1]
    i = 0
    while len(dims) > 2 and i + 1 < len(dims):
        (n0, s0), (n1, s1) = dims[i], dims[i + 1]
        if all(a == n1 * b for a, b in zip(s0, s1)):
            dims[i:i + 2] = [(n0 * n1, s1)]
        else:
            i += 1
    if len(dims) > 2:
        raise ValueError(f"{name}: rows of shape {tuple(lead)} do not fold into two strides")
    dims = [(1, [0] * len(strides))] * (2 - len(dims)) + dims
    return dims[0][0], dims[1][0], list(zip(dims[0][1], dims[1][1]))


def _f32(name, t, shape):
    """Checks for a contiguous fp32 tensor of the given shape (None passes)."""
    if t is not None and (t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {tuple(shape)}")


def _like(name, t, x):
    """Checks a tensor given by the caller for x's shape and dtype."""
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError(f"{name} must have the shape {tuple(x.shape)} and dtype {x.dtype}")


def _ptrs(*tensors):
    """Device addresses as _ptr gives them (the current device asked for once)."""
    dev = torch.cuda.current_device() if tensors and tensors[0].is_cuda else -1
    return [None if t is None else t.data_ptr() if t.get_device() == dev >= 0 else _ptr(t)
            for t in tensors]


# The descriptors below depend on shapes, strides and options alone, and a
# program calls with the same ones over and over: building one costs 5 us,
# finding it here less than one.  Options are plain numbers by then: a tensor
# would be found by its identity, whatever it holds now.
@functools.lru_cache(maxsize=256)
def _ln_desc(shape, dtype, eps, sx, sg, so, device):
    """(descriptor, workspace bytes of the backward on that device)."""
    n0, n1, st = _row_strides("layernorm", shape, sx, sg, so)
    d = LayerNormDesc(n0, n1, shape[-1], _dtype_code(dtype), eps, *st)
    return d, int(lib.retnet_layernorm_bwd_workspace_size(ctypes.byref(d)))


def layernorm_fwd(x, w=None, b=None, *, eps=1e-5, out=None, mean=None, rstd=None, stream=None):
    """LayerNorm over the last dimension of x (bf16 or fp32, any two row
    strides): y = (x - mean) rstd w + b with fp32 gains w and biases b (None: 1
    and 0).  Returns (y, mean, rstd); mean and rstd, fp32 of x.shape[:-1], are
    what layernorm_bwd takes.  out may be x itself."""
    shape = x.shape
    lead, d = shape[:-1], shape[-1:]
    if out is None:
        out = _empty(stream, shape, x.dtype, x.device)
    else:
        _like("out", out, x)
    if mean is None:
        mean = _empty(stream, lead, torch.float32, x.device)
    if rstd is None:
        rstd = _empty(stream, lead, torch.float32, x.device)
    _f32("w", w, d)
    _f32("b", b, d)
    _f32("mean", mean, lead)
    _f32("rstd", rstd, lead)
    so = out.stride()
    desc, _ = _ln_desc(shape, x.dtype, float(eps), x.stride(), so, so, x.device)
    st = lib.retnet_layernorm_fwd(ctypes.byref(desc), *_ptrs(x, w, b, out, mean, rstd),
                                  _stream(stream))
    _check(st, "retnet_layernorm_fwd")
    return out, mean, rstd


def layernorm_bwd(x, dy, w, mean, rstd, *, dx=None, dw=None, db=None, workspace=None, stream=None):
    """Gradients of layernorm_fwd: returns (dx, dw, db), dx in x's dtype, dw
    and db fp32 (w may be None; dw and db are the sums all the same).  The sums
    over the rows are added in a fixed order.  dx may be x or dy itself."""
    shape = x.shape
    lead, d = shape[:-1], shape[-1:]
    if dx is None:
        dx = _empty(stream, shape, x.dtype, x.device)
    else:
        _like("dx", dx, x)
    if dw is None:
        dw = _empty(stream, d, torch.float32, x.device)
    if db is None:
        db = _empty(stream, d, torch.float32, x.device)
    _like("dy", dy, x)
    _f32("w", w, d)
    _f32("mean", mean, lead)
    _f32("rstd", rstd, lead)
    _f32("dw", dw, d)
    _f32("db", db, d)
    desc, nbytes = _ln_desc(shape, x.dtype, 0.0, x.stride(), dy.stride(), dx.stride(), x.device)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    st = lib.retnet_layernorm_bwd(ctypes.byref(desc),
                                  *_ptrs(x, dy, w, mean, rstd, dx, dw, db, workspace),
                                  workspace.numel(), _stream(stream))
    _check(st, "retnet_layernorm_bwd")
    return dx, dw, db


def _ids(name, t, shape):
    """Bytes of an id of a contiguous int32 or int64 tensor of the given shape."""
    if t.dtype is not torch.int64 and t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")
    return 8 if t.dtype is torch.int64 else 4


@functools.lru_cache(maxsize=256)
def _logits_desc(shape, dtype, temperature, top, id_bytes, tail, sx, sd):
    n0, n1, s = _row_strides("logits", shape, sx, sd)
    return LogitsDesc(n0, n1, shape[-1], _dtype_code(dtype), temperature, top, id_bytes, tail, *s)


def token_logprobs(logits, tokens=None, *, top=0, temperature=1.0, logprob=None, entropy=None,
                   top_logprobs=None, top_ids=None, stream=None):
    """Log probabilities under softmax(logits / temperature) over the last
    dimension (bf16 or fp32, any two row strides): of the given tokens (int32 or
    int64 of logits.shape[:-1]; negative = none, 0), the entropy, and the `top`
    (<= MAX_TOP) largest with their ids, equal logits by the lower id.  Returns
    (logprob, entropy, top_logprobs, top_ids); logprob is None without tokens
    and the last two are None for top=0.  A logit of -inf is a masked token; the
    missing alternatives of a row have id -1."""
    shape, dev = logits.shape, logits.device
    lead = shape[:-1]
    top, id_bytes = operator.index(top), 8
    if tokens is not None:
        id_bytes = _ids("tokens", tokens, lead)
        if logprob is None:
            logprob = _empty(stream, lead, torch.float32, dev)
    elif logprob is not None:
        raise ValueError("logprob needs tokens")
    if entropy is None:
        entropy = _empty(stream, lead, torch.float32, dev)
    if top:
        tops = (*lead, top)
        if top_logprobs is None:
            top_logprobs = _empty(stream, tops, torch.float32, dev)
        if top_ids is None:
            top_ids = _empty(stream, tops, torch.int64, dev)
        if _ids("top_ids", top_ids, tops) != 8:
            raise TypeError("top_ids must be int64")
        _f32("top_logprobs", top_logprobs, tops)
    else:
        top_logprobs = top_ids = None
    _f32("logprob", logprob, lead)
    _f32("entropy", entropy, lead)
    s = logits.stride()
    d = _logits_desc(shape, logits.dtype, float(temperature), top, id_bytes, False, s, s)
    st = lib.retnet_token_logprobs(
        ctypes.byref(d), *_ptrs(logits, tokens, logprob, entropy, top_logprobs, top_ids),
        _stream(stream))
    _check(st, "retnet_token_logprobs")
    return logprob, entropy, top_logprobs, top_ids


def _distill_desc(student, ids, values, temperature, tail, dstudent):
    shape, top = student.shape, ids.shape[-1]
    lists = (*shape[:-1], top)
    id_bytes = _ids("ids", ids, lists)
    _f32("values", values, lists)
    s = student.stride()
    return _logits_desc(shape, student.dtype, float(temperature), top, id_bytes, bool(tail), s,
                        s if dstudent is None else dstudent.stride())


def distill_fwd(student, ids, values, *, temperature=1.0, tail=False, loss=None, stats=None,
                stream=None):
    """Distillation loss of each row of the student's logits (bf16 or fp32,
    any two row strides) against a teacher's list: ids (int32 or int64, negative
    = absent) and values (fp32), both [.., k] with k <= MAX_TOP.  With tail
    False the teacher is softmax(values / temperature) over the list; with tail
    True the values are log probabilities over the whole vocabulary and the
    tokens that are not listed form one more bucket.  A list of one token with
    tail False is the cross entropy of that token.  Returns (loss, stats): the
    loss times temperature^2, fp32 of student.shape[:-1], and what distill_bwd
    needs, [.., 2]."""
    lead = student.shape[:-1]
    pairs = (*lead, 2)
    if loss is None:
        loss = _empty(stream, lead, torch.float32, student.device)
    if stats is None:
        stats = _empty(stream, pairs, torch.float32, student.device)
    _f32("loss", loss, lead)
    _f32("stats", stats, pairs)
    d = _distill_desc(student, ids, values, temperature, tail, None)
    st = lib.retnet_distill_fwd(ctypes.byref(d), *_ptrs(student, ids, values, loss, stats),
                                _stream(stream))
    _check(st, "retnet_distill_fwd")
    return loss, stats


def distill_bwd(student, ids, values, weight, stats, *, temperature=1.0, tail=False, dstudent=None,
                stream=None):
    """Gradient with respect to the student's logits, in their dtype: weight
    (fp32, or None for 1) is the gradient of the caller's loss with respect to
    each row's; rows of weight 0 get zeros.  Rows whose stats are beyond 256 in
    size are read a second time.  dstudent may be student itself."""
    lead = student.shape[:-1]
    if dstudent is None:
        dstudent = _empty(stream, student.shape, student.dtype, student.device)
    else:
        _like("dstudent", dstudent, student)
    _f32("weight", weight, lead)
    _f32("stats", stats, (*lead, 2))
    d = _distill_desc(student, ids, values, temperature, tail, dstudent)
    st = lib.retnet_distill_bwd(ctypes.byref(d),
                                *_ptrs(student, ids, values, weight, stats, dstudent),
                                _stream(stream))
    _check(st, "retnet_distill_bwd")
    return dstudent


def distill_step(student, ids, values, weight=None, *, temperature=1.0, tail=False, loss=None,
                 dstudent=None, stream=None):
    """distill_fwd and distill_bwd in one call that reads the logits from
    memory once: returns (loss, dstudent).  dstudent may be student itself."""
    lead = student.shape[:-1]
    if loss is None:
        loss = _empty(stream, lead, torch.float32, student.device)
    if dstudent is None:
        dstudent = _empty(stream, student.shape, student.dtype, student.device)
    else:
        _like("dstudent", dstudent, student)
    _f32("weight", weight, lead)
    _f32("loss", loss, lead)
    d = _distill_desc(student, ids, values, temperature, tail, dstudent)
    st = lib.retnet_distill_step(ctypes.byref(d),
                                 *_ptrs(student, ids, values, weight, loss, None, dstudent),
                                 _stream(stream))
    _check(st, "retnet_distill_step")
    return loss, dstudent


# The calls below check their tensors once for each set of shapes, strides and
# types that they meet (a step's checks cost 12 us, finding them here 4), and
# keep the descriptor with them.
def _meta(t):
    """What the checks look at."""
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _meta_contiguous(m):
    shape, stride, _ = m
    want = 1
    for n, s in zip(reversed(shape), reversed(stride)):
        if n != 1 and s != want and 0 not in shape:
            return False
        want *= n
    return True


def _meta_f32(name, m, shape):
    """Checks for a contiguous fp32 tensor of the given shape (None passes)."""
    if m is not None and (m[2] != torch.float32 or tuple(m[0]) != tuple(shape) or not _meta_contiguous(m)):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {tuple(shape)}")


def _meta_like(name, m, x):
    """Checks a tensor for x's shape and dtype (None passes) and gives its batch
    and token strides."""
    if m is None:
        return (0, 0)
    if m[0] != x[0] or m[2] != x[2]:
        raise ValueError(f"{name} must have the shape {tuple(x[0])} and dtype {x[2]}")
    if m[1][-1] != 1 and m[0][-1] > 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    return (m[1][0], m[1][1] if len(m[0]) == 3 else 0)


def _meta_lengths(m, B):
    """Bytes of a length (8 without lengths)."""
    if m is None:
        return 8
    if m[2] is not torch.int64 and m[2] is not torch.int32:
        raise TypeError(f"lengths must be int32 or int64, got {m[2]}")
    if tuple(m[0]) != (B,) or not _meta_contiguous(m):
        raise ValueError(f"lengths must be a contiguous tensor of shape {(B,)}")
    return 8 if m[2] is torch.int64 else 4


def _meta_sequences(x, step):
    """(B, N, E) of x [B, N, E], or of a step's [B, E]."""
    shape = x[0]
    if len(shape) != (2 if step else 3):
        raise ValueError(f"x must be {'[B, E]' if step else '[B, N, E]'}, got {tuple(shape)}")
    _dtype_code(x[2])
    return (shape[0], 1, shape[1]) if step else tuple(shape)


@functools.lru_cache(maxsize=256)
def _scan_plan(step, softplus, device, x, dt, A, B, C, D, z, dt_bias, lengths, h_in, h_out, y=None, dy=None,
               dx=None, ddt=None, dz=None, dA=None, dB=None, dC=None, dD=None, ddt_bias=None):
    """(descriptor, workspace bytes of the forward and of the backward on that
    device), after checks of the tensors' shapes, strides and types."""
    Bn, N, E = _meta_sequences(x, step)
    lead = 1 if step else 2
    if len(A[0]) != 2:
        raise ValueError(f"A must be [E, S], got {tuple(A[0])}")
    S = A[0][1]
    h_name = "h_out" if dy is None else "dh_out"
    for name, m, shape in (("A", A, (E, S)), ("D", D, (E,)), ("dt_bias", dt_bias, (E,)), ("h_in", h_in, (Bn, E, S)),
                           (h_name, h_out, (Bn, E, S)), ("dA", dA, (E, S)), ("dD", dD, (E,)),
                           ("ddt_bias", ddt_bias, (E,))):
        _meta_f32(name, m, shape)
    strides = [_meta_like(name, m, x) for name, m in (("x", x), ("dt", dt), ("z", z), ("out", y), ("dy", dy),
                                                       ("dx", dx), ("ddt", ddt), ("dz", dz))]
    rows, groups = tuple(x[0][:-1]), []
    for name, (shape, s, dtype) in (("B", B), ("C", C)):
        shape, s = tuple(shape), tuple(s)
        if len(shape) == lead + 1:
            shape, s = (*shape[:lead], 1, shape[lead]), (*s[:lead], 0, s[lead])
        if len(shape) != lead + 2 or shape[:lead] != rows or shape[-1] != S or dtype != x[2]:
            raise ValueError(f"{name} must have the shape {rows + ('groups', S)} and dtype {x[2]}")
        if s[-1] != 1 and S > 1:
            raise ValueError(f"{name}: the states must be contiguous")
        groups.append((shape[lead], (s[0], s[1] if lead == 2 else 0, s[lead])))
    (G, sB), (GC, sC) = groups
    if GC != G or G < 1 or E % G:
        raise ValueError(f"B and C must have equal groups that divide the {E} channels")
    for name, m, like in (("dB", dB, B), ("dC", dC, C)):
        if m is not None and (m[0] != like[0] or m[2] != like[2] or not _meta_contiguous(m)):
            raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(like[0])} and dtype {like[2]}")
    d = ScanDesc(Bn, N, E, S, G, _dtype_code(x[2]), softplus, _meta_lengths(lengths, Bn), *strides, sB, sC)
    return (d, int(lib.retnet_selective_scan_workspace_size(ctypes.byref(d))),
            int(lib.retnet_selective_scan_bwd_workspace_size(ctypes.byref(d))))


def selective_scan_fwd(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, h_in=None,
                       lengths=None, out=None, h_out=None, workspace=None, stream=None):
    """Selective state space scan of x, dt [B, N, E] (bf16 or fp32, any batch and
    token strides) with A [E, S] fp32 (S <= MAX_STATES) and B, C [B, N, G, S] (or
    [B, N, S]): with delta = softplus(dt + dt_bias),
        h_t = exp(delta_t A) h_(t-1) + delta_t x_t B_t,
        y_t = (C_t . h_t + D x_t) silu(z_t).
    A decay exp(delta_t A) below 2^-126 counts as 0.
    D, dt_bias fp32 [E]; z like x; h_in fp32 [B, E, S] (None: 0); lengths int32
    or int64 [B] on the device: tokens of each sequence of a padded batch, rows
    of y behind them are zeros.  Returns (y, the states after the last tokens)."""
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    if h_out is None:
        h_out = _empty(stream, (x.shape[0], x.shape[-1], A.shape[-1]), torch.float32, x.device)
    desc, nbytes, _ = _scan_plan(False, bool(softplus), x.device, _meta(x), _meta(dt), _meta(A), _meta(B), _meta(C),
                                 _meta(D), _meta(z), _meta(dt_bias), _meta(lengths), _meta(h_in), _meta(h_out),
                                 _meta(out))
    if workspace is None and nbytes:
        with _on(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    st = lib.retnet_selective_scan_fwd(
        ctypes.byref(desc), *_ptrs(x, dt, A, B, C, D, z, dt_bias, h_in, lengths, out, h_out, workspace),
        0 if workspace is None else workspace.numel(), _stream(stream))
    _check(st, "retnet_selective_scan_fwd")
    return out, h_out


def selective_scan_step(x, dt, A, B, C, h, *, D=None, z=None, dt_bias=None, softplus=True, h_out=None,
                        out=None, stream=None):
    """One token of selective_scan_fwd: x, dt, z [B, E], B, C [B, G, S] (or [B, S]);
    the states h fp32 [B, E, S] are updated in place, or written to h_out.
    Returns y [B, E]."""
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    if h_out is None:
        h_out = h
    desc, _, _ = _scan_plan(True, bool(softplus), x.device, _meta(x), _meta(dt), _meta(A), _meta(B), _meta(C),
                            _meta(D), _meta(z), _meta(dt_bias), None, _meta(h), _meta(h_out), _meta(out))
    st = lib.retnet_selective_scan_step(
        ctypes.byref(desc), *_ptrs(x, dt, A, B, C, D, z, dt_bias, h, out, h_out), _stream(stream))
    _check(st, "retnet_selective_scan_step")
    return out


ScanGrads = collections.namedtuple("ScanGrads", "dx ddt dA dB dC dD dz ddt_bias dh_in")


def selective_scan_bwd(x, dt, A, B, C, dy, *, D=None, z=None, dt_bias=None, softplus=True, h_in=None,
                       dh_out=None, lengths=None, dx=None, ddt=None, dA=None, dB=None, dC=None, dD=None,
                       dz=None, ddt_bias=None, dh_in=None, workspace=None, stream=None):
    """Gradients of selective_scan_fwd from its inputs, dy (like x) and dh_out
    (fp32, of the states after the last tokens, None: 0).  Returns a ScanGrads:
    dx, ddt, dz like x, dB, dC like B (contiguous), dA, dD, ddt_bias, dh_in fp32;
    None where the input was None.  All sums are added in a fixed order."""
    dev = x.device

    def new(given, like):
        if given is None and like is not None:
            given = _empty(stream, like.shape, like.dtype, dev)
        return given if like is not None else None

    dx, ddt, dz = new(dx, x), new(ddt, dt), new(dz, z)
    dA, dB, dC = new(dA, A), new(dB, B), new(dC, C)
    dD, ddt_bias, dh_in = new(dD, D), new(ddt_bias, dt_bias), new(dh_in, h_in)
    desc, _, nbytes = _scan_plan(False, bool(softplus), dev, *map(_meta, (
        x, dt, A, B, C, D, z, dt_bias, lengths, h_in, dh_out, None, dy, dx, ddt, dz, dA, dB, dC, dD, ddt_bias)))
    if dh_in is not None:
        _f32("dh_in", dh_in, h_in.shape)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = lib.retnet_selective_scan_bwd(
        ctypes.byref(desc),
        *_ptrs(x, dt, A, B, C, D, z, dt_bias, h_in, lengths, dy, dh_out, dx, ddt, dA, dB, dC, dD, dz,
               ddt_bias, dh_in, workspace), workspace.numel(), _stream(stream))
    _check(st, "retnet_selective_scan_bwd")
    return ScanGrads(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh_in)


@functools.lru_cache(maxsize=256)
def _conv_plan(step, silu, device, x, w, b, lengths, out, states, dy=None, dw=None, db=None):
    """(descriptor, workspace bytes of the backward on that device), after checks
    of the tensors; states: (name, kept inputs or their gradient)."""
    Bn, N, E = _meta_sequences(x, step)
    if len(w[0]) != 2:
        raise ValueError(f"w must be [E, taps], got {tuple(w[0])}")
    W = w[0][1]
    for name, m, shape in (("w", w, (E, W)), ("b", b, (E,)), ("dw", dw, (E, W)), ("db", db, (E,))):
        _meta_f32(name, m, shape)
    for name, m in states:
        if m is not None and (tuple(m[0]) != (Bn, W - 1, E) or m[2] != x[2] or not _meta_contiguous(m)):
            raise ValueError(f"{name} must be a contiguous tensor of shape {(Bn, W - 1, E)} and dtype {x[2]}")
    d = ConvDesc(Bn, N, E, W, _dtype_code(x[2]), silu, _meta_lengths(lengths, Bn), _meta_like("x", x, x),
                 _meta_like("dy", dy, x), _meta_like("out", out, x))
    return d, int(lib.retnet_causal_conv_bwd_workspace_size(ctypes.byref(d)))


def causal_conv_fwd(x, w, b=None, *, silu=True, state_in=None, lengths=None, out=None, state_out=None,
                    stream=None):
    """Causal convolution of each channel of x [B, N, E] (bf16 or fp32, any batch
    and token strides) with w [E, taps] fp32 (2 to 4 taps, the last one the
    token's own) and b fp32 [E], then silu.  state_in [B, taps - 1, E] in x's
    dtype: the inputs before the first token, the oldest first (None: 0).
    lengths as for selective_scan_fwd.  Returns (y, the last taps - 1 inputs of
    each sequence); state_out may be state_in."""
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    if state_out is None:
        state_out = _empty(stream, (x.shape[0], w.shape[-1] - 1, x.shape[-1]), x.dtype, x.device)
    desc, _ = _conv_plan(False, bool(silu), x.device, _meta(x), _meta(w), _meta(b), _meta(lengths), _meta(out),
                         (("state_in", _meta(state_in)), ("state_out", _meta(state_out))))
    st = lib.retnet_causal_conv_fwd(ctypes.byref(desc),
                                    *_ptrs(x, w, b, state_in, lengths, out, state_out), _stream(stream))
    _check(st, "retnet_causal_conv_fwd")
    return out, state_out


def causal_conv_step(x, w, b, state, *, silu=True, state_out=None, out=None, stream=None):
    """One token of causal_conv_fwd: x [B, E]; the state [B, taps - 1, E] is
    updated in place, or written to state_out.  Returns y [B, E]."""
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    if state_out is None:
        state_out = state
    desc, _ = _conv_plan(True, bool(silu), x.device, _meta(x), _meta(w), _meta(b), None, _meta(out),
                         (("state", _meta(state)), ("state_out", _meta(state_out))))
    st = lib.retnet_causal_conv_fwd(ctypes.byref(desc), *_ptrs(x, w, b, state, None, out, state_out),
                                    _stream(stream))
    _check(st, "retnet_causal_conv_fwd")
    return out


def causal_conv_bwd(x, w, b, dy, *, silu=True, state_in=None, dstate_out=None, lengths=None, dx=None,
                    dw=None, db=None, dstate_in=None, workspace=None, stream=None):
    """Gradients of causal_conv_fwd from its inputs, dy (like x) and dstate_out
    (of the state after the last token, None: 0).  Returns (dx, dw, db,
    dstate_in); db is None without b, dstate_in without state_in.  The sums over
    the tokens are added in a fixed order."""
    dev = x.device
    if dx is None:
        dx = _empty(stream, x.shape, x.dtype, dev)
    if dw is None:
        dw = _empty(stream, w.shape, torch.float32, dev)
    if b is None:
        db = None
    elif db is None:
        db = _empty(stream, b.shape, torch.float32, dev)
    if state_in is None:
        dstate_in = None
    elif dstate_in is None:
        dstate_in = _empty(stream, state_in.shape, x.dtype, dev)
    states = (("state_in", _meta(state_in)), ("dstate_out", _meta(dstate_out)), ("dstate_in", _meta(dstate_in)))
    desc, nbytes = _conv_plan(False, bool(silu), dev, _meta(x), _meta(w), _meta(b), _meta(lengths), _meta(dx), states,
                              _meta(dy), _meta(dw), _meta(db))
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = lib.retnet_causal_conv_bwd(
        ctypes.byref(desc), *_ptrs(x, w, b, state_in, lengths, dy, dstate_out, dx, dw, db, dstate_in, workspace),
        workspace.numel(), _stream(stream))
    _check(st, "retnet_causal_conv_bwd")
    return dx, dw, db, dstate_in


@functools.lru_cache(maxsize=256)
def _rms_plan(device, eps, group, x, r, w, h, out, vectors, dy=None):
    """(descriptor, workspace bytes of the backward on that device), after checks
    of the tensors: r, h (None: x), out and dy like x (out with a group: e4m3);
    vectors: (name, fp32 tensor, its shape)."""
    shape = x[0]
    for name, m in (("residual", r), ("residual_out", h), ("dy", dy), ("out", out if group is None else None)):
        if m is not None and (m[0] != shape or m[2] != x[2]):
            name = {"residual": "dh", "out": "dx"}.get(name, name) if dy is not None else name
            raise ValueError(f"{name} must have the shape {tuple(shape)} and dtype {x[2]}")
    if group is not None and (out[0] != shape or out[2] != torch.float8_e4m3fn):
        raise ValueError(f"out must have the shape {tuple(shape)} and dtype torch.float8_e4m3fn")
    _meta_f32("w", w, shape[-1:])
    for name, m, want in vectors:
        _meta_f32(name, m, want)
    sx = x[1]
    n0, n1, st = _row_strides("rmsnorm", shape, sx, sx if r is None else r[1], sx if h is None else h[1],
                              sx if dy is None else dy[1], out[1])
    d = RmsNormDesc(n0, n1, shape[-1], _dtype_code(x[2]), eps, group or 0, *st)
    return d, int(lib.retnet_rmsnorm_bwd_workspace_size(ctypes.byref(d)))


def _rms_sum(x, residual, residual_out, stream):
    """Where the sum is kept (None without a residual: x is the sum)."""
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return None
    return _empty(stream, x.shape, x.dtype, x.device) if residual_out is None else residual_out


def rmsnorm_fwd(x, w=None, *, residual=None, eps=1e-5, out=None, residual_out=None, rstd=None, stream=None):
    """Root-mean-square norm over the last dimension (bf16 or fp32, any two row
    strides) of h = x + residual, rounded to x's dtype: y = h rstd w with rstd =
    1 / sqrt(mean(h^2) + eps) and fp32 gains w (None: 1).  Returns (y, h, rstd): h
    (x itself without a residual) and rstd, fp32 of x.shape[:-1], are what
    rmsnorm_bwd takes.  residual_out, where h is kept, and out may be x or
    residual, but not the same one."""
    h = _rms_sum(x, residual, residual_out, stream)
    shape = x.shape
    if out is None:
        out = _empty(stream, shape, x.dtype, x.device)
    if rstd is None:
        rstd = _empty(stream, shape[:-1], torch.float32, x.device)
    desc, _ = _rms_plan(x.device, float(eps), None, _meta(x), _meta(residual), _meta(w), _meta(h), _meta(out),
                        (("rstd", _meta(rstd), shape[:-1]),))
    st = lib.retnet_rmsnorm_fwd(ctypes.byref(desc), *_ptrs(x, residual, w, h, out, rstd), _stream(stream))
    _check(st, "retnet_rmsnorm_fwd")
    return out, x if h is None else h, rstd


def rmsnorm_quant(x, w=None, *, residual=None, eps=1e-5, group=0, out=None, scales=None, residual_out=None,
                  stream=None):
    """rmsnorm_fwd with y as e4m3 values q (torch.float8_e4m3fn) and an fp32
    scale for each `group` columns (a multiple of 8; 0: the whole row): y = q
    scale, scale = max |y| / 448 (NaN, like all of q, where the group has a NaN).
    Returns (q, scales, h), scales of x.shape[:-1] + (groups,)."""
    h = _rms_sum(x, residual, residual_out, stream)
    group, d = operator.index(group), x.shape[-1]
    if group < 0 or group % 8:
        raise ValueError(f"group must be 0 or a multiple of 8, got {group}")
    if out is None:
        out = _empty(stream, x.shape, torch.float8_e4m3fn, x.device)
    shape = (*x.shape[:-1], -(-d // group) if group else 1)
    if scales is None:
        scales = _empty(stream, shape, torch.float32, x.device)
    desc, _ = _rms_plan(x.device, float(eps), group, _meta(x), _meta(residual), _meta(w), _meta(h), _meta(out),
                        (("scales", _meta(scales), shape),))
    st = lib.retnet_rmsnorm_quant(ctypes.byref(desc), *_ptrs(x, residual, w, h, out, scales), _stream(stream))
    _check(st, "retnet_rmsnorm_quant")
    return out, scales, x if h is None else h


def rmsnorm_bwd(h, dy, w, rstd, *, dh=None, dx=None, dw=None, workspace=None, stream=None):
    """Gradients of rmsnorm_fwd: returns (dx, dw); dx, in h's dtype, is the
    gradient of x and of the residual: that of the norm and dh, which reaches h
    itself (None: 0).  dw fp32 (w may be None; dw is the sum all the same), added
    in a fixed order.  dx may be h, dy or dh."""
    shape, d = h.shape, h.shape[-1:]
    if dx is None:
        dx = _empty(stream, shape, h.dtype, h.device)
    if dw is None:
        dw = _empty(stream, d, torch.float32, h.device)
    desc, nbytes = _rms_plan(h.device, 0.0, None, _meta(h), _meta(dh), _meta(w), None, _meta(dx),
                             (("rstd", _meta(rstd), shape[:-1]), ("dw", _meta(dw), d)), _meta(dy))
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=h.device)
    st = lib.retnet_rmsnorm_bwd(ctypes.byref(desc), *_ptrs(h, dy, dh, w, rstd, dx, dw, workspace),
                                workspace.numel(), _stream(stream))
    _check(st, "retnet_rmsnorm_bwd")
    return dx, dw


def poll_status(workspace, stream=None):
    """Reads and clears the device status word (synchronises the stream)."""
    return int(lib.retention_poll_status(_ptr(workspace), _stream(stream)))


def kernel_times():
    """{kernel name: (total ms of timed launches, launches, timed launches)}
    since the last reset; call after synchronising the streams."""
    out = {}
    for i in range(lib.retention_kernel_count()):
        ms, n, t = ctypes.c_double(), ctypes.c_longlong(), ctypes.c_int()
        _check(lib.retention_kernel_timer_read(i, ctypes.byref(ms), ctypes.byref(n),
                                               ctypes.byref(t)), "kernel_timer_read")
        if n.value:
            out[lib.retention_kernel_name(i).decode()] = (ms.value, n.value, t.value)
    return out
