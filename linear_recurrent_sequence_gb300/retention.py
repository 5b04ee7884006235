"""Python binding of the retention C ABI (``include/retention.h``).

Argument marshalling only: every step of retention runs in the CUDA kernels
of ``libretention.so``.  PyTorch supplies device memory and the stream.  If
the library has not been built this module raises at import; there is no
fallback implementation.
"""
from __future__ import annotations

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


def new_workspace(nbytes, device, stream=None):
    """A workspace for calls on the given stream (None: the current one)."""
    # zeroed once: its first bytes hold the device status word
    with _on(stream):
        return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _prep(q, k, v, out, out_dtype):
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        B, H, N, _ = q.shape
        out = torch.empty((B, H, N, v.shape[3]), dtype=out_dtype or q.dtype, device=q.device)
    return out


def chunkwise_fwd(q, k, v, gamma, *, chunk=64, norm_flags=0, gn_eps=1e-6, pos0=0,
                  rotate=True, theta_base=10000.0, S_in=None, z_in=None, S_out=None,
                  z_out=None, out=None, out_dtype=None, workspace=None, stream=None):
    """Chunkwise retention forward; q,k [B,H,N,d_k], v [B,H,N,d_v] (any strides
    with a contiguous feature dimension).  Returns the output tensor."""
    out = _prep(q, k, v, out, out_dtype)
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
        S_out = torch.empty(B, H, dk, dv, dtype=torch.float32, device=k.device)
    if with_z and z_out is None:
        z_out = torch.empty(B, H, dk, dtype=torch.float32, device=k.device)
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
            return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
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
    out = _prep(q, k, v, out, out_dtype)
    d, g = make_desc(q, k, v, out, gamma, chunk=chunk, norm_flags=norm_flags, gn_eps=gn_eps,
                     pos0=pos0, rotate=rotate, theta_base=theta_base)
    st = lib.retention_chunkwise_fwd_noalloc(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v),
                                             _ptr(S_in), _ptr(z_in), _ptr(S_out), _ptr(z_out),
                                             _ptr(out), _stream(stream))
    _check(st, "retention_chunkwise_fwd_noalloc")
    return out


def parallel_fwd(q, k, v, gamma, *, norm_flags=0, gn_eps=1e-6, pos0=0, rotate=True,
                 theta_base=10000.0, out=None, out_dtype=None, workspace=None, stream=None):
    out = _prep(q, k, v, out, out_dtype)
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
    out = _prep(q4, k4, v4, out if out is None or out.dim() == 4 else out.unsqueeze(2), out_dtype)
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
    out = torch.empty((B, H, N, dd), dtype=out_dtype or x.dtype, device=x.device)
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
        out = torch.empty((B, N, dm), dtype=torch.bfloat16, device=X.device)
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
        out = torch.empty((B, N, dm), dtype=torch.bfloat16, device=X.device)
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
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
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
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _like("out", out, x)
    if mean is None:
        mean = torch.empty(lead, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
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
        dx = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _like("dx", dx, x)
    if dw is None:
        dw = torch.empty(d, dtype=torch.float32, device=x.device)
    if db is None:
        db = torch.empty(d, dtype=torch.float32, device=x.device)
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
            logprob = torch.empty(lead, dtype=torch.float32, device=dev)
    elif logprob is not None:
        raise ValueError("logprob needs tokens")
    if entropy is None:
        entropy = torch.empty(lead, dtype=torch.float32, device=dev)
    if top:
        tops = (*lead, top)
        if top_logprobs is None:
            top_logprobs = torch.empty(tops, dtype=torch.float32, device=dev)
        if top_ids is None:
            top_ids = torch.empty(tops, dtype=torch.int64, device=dev)
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
        loss = torch.empty(lead, dtype=torch.float32, device=student.device)
    if stats is None:
        stats = torch.empty(pairs, dtype=torch.float32, device=student.device)
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
        dstudent = torch.empty(student.shape, dtype=student.dtype, device=student.device)
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
        loss = torch.empty(lead, dtype=torch.float32, device=student.device)
    if dstudent is None:
        dstudent = torch.empty(student.shape, dtype=student.dtype, device=student.device)
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
