"""Kimi Delta Attention (KDA) for NVIDIA B200 -- Python binding of ``libkda.so``.

The functions here only marshal arguments into the C ABI declared in
``include/kda.h`` (same names); every step of the computation runs in the
library's CUDA kernels. PyTorch supplies device memory and the current CUDA
stream. If the library is missing the calls raise -- there is no fallback.

Build the library with ``python -m gated_delta_rule_125_b200.build``.
"""
from __future__ import annotations

import collections
import ctypes
import math
import os

import torch

__all__ = ["kda_prefill", "kda_decode_step", "kda_prefill_workspace_size", "kda_prefill_launches",
           "kda_device_error", "kda_prefill_noalloc", "kda_short_conv_swish", "kda_backward",
           "kda_prefill_workspace_min", "kda_set_wait_limit_ns", "kda_status_string", "kda_version", "KDAError",
           "library_path", "load_library", "KDA_OK", "KDA_ERR_INVALID_ARG",
           "KDA_ERR_UNSUPPORTED", "KDA_ERR_MISALIGNED", "KDA_ERR_WORKSPACE", "KDA_ERR_CUDA",
           "KDA_ERR_TIMEOUT", "KDA_FLAG_NO_L2NORM", "KDA_FLAG_EXACT", "KDA_FLAG_SCALAR_GATE", "KDA_FLAG_SOFTPLUS",
           "kda_ssm_prefill", "kda_ssm_step", "kda_ssm_backward",
           "kda_short_conv_step", "kda_short_conv_backward", "kda_residual_norm", "kda_residual_norm_backward"]

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_MISALIGNED = 0, 1, 2, 3
KDA_ERR_WORKSPACE, KDA_ERR_CUDA, KDA_ERR_TIMEOUT = 4, 5, 6
KDA_DTYPE_F32, KDA_DTYPE_BF16 = 0, 1
KDA_FLAG_NO_L2NORM, KDA_FLAG_EXACT, KDA_FLAG_SCALAR_GATE = 0x1, 0x2, 0x4
KDA_FLAG_SOFTPLUS = 0x8
KDA_SSM_TILE = 128

EXPORTED_SYMBOLS = ("kda_status_string", "kda_version", "kda_prefill_workspace_size",
                    "kda_prefill_workspace_min", "kda_prefill_launches", "kda_prefill",
                    "kda_prefill_ex", "kda_decode_step", "kda_decode_step_ex", "kda_device_error",
                    "kda_prefill_noalloc", "kda_short_conv_swish", "kda_short_conv_launches",
                    "kda_decode_step_conv", "kda_backward_workspace_size", "kda_backward",
                    "kda_set_wait_limit_ns", "kda_prefill_conv", "kda_ssm_tile_states_size", "kda_ssm_prefill",
                    "kda_ssm_prefill_workspace_size", "kda_ssm_prefill_launches",
                    "kda_ssm_step", "kda_ssm_backward_workspace_size", "kda_ssm_backward",
                    "kda_short_conv_swish_ex", "kda_short_conv_step", "kda_short_conv_backward_workspace_size",
                    "kda_short_conv_backward", "kda_residual_norm", "kda_residual_norm_backward_workspace_size",
                    "kda_residual_norm_backward")


class OutputGate(ctypes.Structure):
    """``kda_output_gate``: the fused output step (RMSNorm over d_v, sigmoid gate)."""
    _fields_ = [("gate", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


class ShortConv(ctypes.Structure):
    """``kda_short_conv``: causal short convolution + Swish (width, weight, states)."""
    _fields_ = [("width", ctypes.c_int32), ("weight", ctypes.c_void_p), ("state_in", ctypes.c_void_p),
                ("state_out", ctypes.c_void_p)]


class Ssm(ctypes.Structure):
    """``kda_ssm``: sizes and parameters of a selective scan."""
    _fields_ = [("channels", ctypes.c_int32), ("states", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class SsmGrads(ctypes.Structure):
    """``kda_ssm_grads``: where the gradients of a selective scan go."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias", "dS0")]


class ResidualNorm(ctypes.Structure):
    """``kda_residual_norm_args``: inputs of the norms around a block."""
    _fields_ = [("y", ctypes.c_void_p), ("r", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("w_post", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("w_pre", ctypes.c_void_p), ("res_scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("rows", ctypes.c_int64), ("D", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("res_dtype", ctypes.c_int)]


_lib = None


def library_path() -> str:
    return os.environ.get("KDA_LIBRARY",
                          os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so"))


class KDAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s" % (what, kda_status_string(status)))
        self.status = status


def load_library():
    """Load ``libkda.so`` (raises ``OSError`` if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise OSError("libkda.so not found at %s; build it with "
                      "`python -m gated_delta_rule_125_b200.build`" % path)
    lib = ctypes.CDLL(path)
    vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    i32, i64, u32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_version.restype = i32
    for f in (lib.kda_prefill_workspace_size, lib.kda_prefill_workspace_min):
        f.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_int, i32, u32]
        f.restype = sz
    lib.kda_prefill_launches.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_int, i32, u32, sz]
    lib.kda_prefill_launches.restype = i64
    lib.kda_prefill.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i64, i32, i32, i32, i32,
                                ctypes.c_int, i32, u32, vp, fp, vp, sz, vp]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, i32, i32, i32, i32, ctypes.c_int,
                                    u32, vp, vp]
    lib.kda_decode_step.restype = ctypes.c_int
    og = ctypes.POINTER(OutputGate)
    lib.kda_prefill_ex.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i64, i32, i32, i32, i32,
                                   ctypes.c_int, i32, u32, og, vp, fp, vp, sz, vp]
    lib.kda_prefill_ex.restype = ctypes.c_int
    lib.kda_decode_step_ex.argtypes = [vp, vp, vp, fp, fp, fp, i32, i32, i32, i32, ctypes.c_int,
                                       u32, og, vp, vp]
    lib.kda_decode_step_ex.restype = ctypes.c_int
    lib.kda_prefill_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i64, i32, i32, i32,
                                        i32, ctypes.c_int, i32, u32, vp, fp, vp]
    lib.kda_prefill_noalloc.restype = ctypes.c_int
    lib.kda_device_error.argtypes = [ctypes.POINTER(i32), i32]
    lib.kda_device_error.restype = ctypes.c_int
    sc = ctypes.POINTER(ShortConv)
    lib.kda_short_conv_swish.argtypes = [vp, vp, sc, ip, i32, i64, i32, ctypes.c_int, vp]
    lib.kda_short_conv_swish.restype = ctypes.c_int
    lib.kda_short_conv_launches.argtypes = [i32, i32, i64]
    lib.kda_short_conv_launches.restype = i64
    lib.kda_decode_step_conv.argtypes = [vp, vp, vp, fp, fp, fp, i32, i32, i32, i32, ctypes.c_int,
                                         u32, sc, sc, sc, og, vp, vp]
    lib.kda_decode_step_conv.restype = ctypes.c_int
    lib.kda_prefill_conv.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i64, i32, i32, i32, i32,
                                     ctypes.c_int, i32, u32, sc, sc, sc, og, vp, fp, vp, sz, vp]
    lib.kda_prefill_conv.restype = ctypes.c_int
    lib.kda_backward_workspace_size.argtypes = [i32, i64, i32, i32, i32, i32, ctypes.c_int, i32, u32]
    lib.kda_backward_workspace_size.restype = sz
    lib.kda_backward.argtypes = [vp, vp, vp, fp, fp, fp, ip, i32, i64, i32, i32, i32, i32, ctypes.c_int, i32, u32,
                                 vp, fp, fp, fp, fp, fp, fp, fp, vp, sz, vp]
    lib.kda_backward.restype = ctypes.c_int
    lib.kda_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.kda_set_wait_limit_ns.restype = ctypes.c_uint64
    sp = ctypes.POINTER(Ssm)
    lib.kda_ssm_tile_states_size.argtypes = [i32, i64, i32, i32]
    lib.kda_ssm_tile_states_size.restype = sz
    lib.kda_ssm_prefill_workspace_size.argtypes = lib.kda_ssm_prefill_launches.argtypes = [i32, i64, i32, i32, i32]
    lib.kda_ssm_prefill_workspace_size.restype, lib.kda_ssm_prefill_launches.restype = sz, i64
    lib.kda_ssm_prefill.argtypes = [vp, vp, vp, vp, vp, sp, fp, ip, i32, i64, ctypes.c_int, u32, vp, fp, fp, vp, sz, vp]
    lib.kda_ssm_prefill.restype = ctypes.c_int
    lib.kda_ssm_step.argtypes = [vp, vp, vp, vp, vp, sp, fp, i32, ctypes.c_int, u32, vp, vp]
    lib.kda_ssm_step.restype = ctypes.c_int
    lib.kda_ssm_backward_workspace_size.argtypes = [i32, i64, i32, i32, i32]
    lib.kda_ssm_backward_workspace_size.restype = sz
    lib.kda_ssm_backward.argtypes = [vp, vp, vp, vp, vp, sp, fp, ip, i32, i64, ctypes.c_int, u32, fp, vp, fp,
                                     ctypes.POINTER(SsmGrads), vp, sz, vp]
    lib.kda_ssm_backward.restype = ctypes.c_int
    lib.kda_short_conv_swish_ex.argtypes = [vp, vp, sc, fp, ip, i32, i64, i32, ctypes.c_int, vp]
    lib.kda_short_conv_swish_ex.restype = ctypes.c_int
    lib.kda_short_conv_step.argtypes = [vp, vp, sc, fp, i32, i32, ctypes.c_int, vp]
    lib.kda_short_conv_step.restype = ctypes.c_int
    lib.kda_short_conv_backward_workspace_size.argtypes = [i64, i32, i32]
    lib.kda_short_conv_backward_workspace_size.restype = sz
    lib.kda_short_conv_backward.argtypes = [vp, sc, fp, ip, i32, i64, i32, ctypes.c_int, vp, ctypes.c_int, fp, fp, fp,
                                            fp, vp, sz, vp]
    lib.kda_short_conv_backward.restype = ctypes.c_int
    rn = ctypes.POINTER(ResidualNorm)
    lib.kda_residual_norm.argtypes = [rn, vp, vp, vp]
    lib.kda_residual_norm.restype = ctypes.c_int
    lib.kda_residual_norm_backward_workspace_size.argtypes = [i64, i32]
    lib.kda_residual_norm_backward_workspace_size.restype = sz
    lib.kda_residual_norm_backward.argtypes = [rn, vp, fp, fp, fp, fp, fp, fp, fp, vp, sz, vp]
    lib.kda_residual_norm_backward.restype = ctypes.c_int
    _lib = lib
    return lib


def kda_status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def kda_version() -> int:
    return int(load_library().kda_version())


def kda_device_error(reset: bool = True) -> int:
    """Device error word of the current device (0: no bounded wait ran out). Synchronous."""
    code = ctypes.c_int32(0)
    load_library().kda_device_error(ctypes.byref(code), int(bool(reset)))
    return int(code.value)


def kda_set_wait_limit_ns(ns: int) -> int:
    """Bound (ns) of the prefill's waits between CTAs for later calls; 0 = default (2 s).
    Returns the previous bound (``kda_set_wait_limit_ns`` in ``include/kda.h``)."""
    return int(load_library().kda_set_wait_limit_ns(int(ns)))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError("q/k/v must be bfloat16 or float32, got %s" % t.dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr() or None


def _out_gate(out_gate):
    """(gate, weight, eps) -> a ``kda_output_gate`` (None -> NULL)."""
    if out_gate is None:
        return None
    g, w, eps = out_gate
    return ctypes.byref(OutputGate(_ptr(g), _ptr(w), float(eps)))


def _conv(conv):
    """(weight [C, W] fp32, state_in or None, state_out or None) -> a ``kda_short_conv`` (None -> NULL)."""
    if conv is None:
        return None
    w, sin, sout = conv
    return ctypes.byref(ShortConv(int(w.shape[-1]), _ptr(w), _ptr(sin), _ptr(sout)))


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _flags(l2norm, exact, scalar_gate=False):
    return ((0 if l2norm else KDA_FLAG_NO_L2NORM) | (KDA_FLAG_EXACT if exact else 0) |
            (KDA_FLAG_SCALAR_GATE if scalar_gate else 0))


def kda_prefill_workspace_size(num_seqs, total_tokens, max_seqlen, H, dk, dv, dtype,
                               chunk=64, l2norm=True, exact=False) -> int:
    code = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return int(load_library().kda_prefill_workspace_size(num_seqs, total_tokens, max_seqlen, H,
                                                        dk, dv, code, chunk,
                                                        _flags(l2norm, exact)))


def kda_prefill_workspace_min(num_seqs, total_tokens, max_seqlen, H, dk, dv, dtype,
                              chunk=64, l2norm=True, exact=False) -> int:
    code = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return int(load_library().kda_prefill_workspace_min(num_seqs, total_tokens, max_seqlen, H,
                                                       dk, dv, code, chunk,
                                                       _flags(l2norm, exact)))


def kda_prefill_launches(num_seqs, total_tokens, max_seqlen, H, dk, dv, dtype, workspace_bytes,
                         chunk=64, l2norm=True, exact=False) -> int:
    code = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return int(load_library().kda_prefill_launches(num_seqs, total_tokens, max_seqlen, H, dk, dv,
                                                  code, chunk, _flags(l2norm, exact),
                                                  workspace_bytes))


def kda_prefill(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, *, max_seqlen=None,
                chunk=64, l2norm=True, exact=False, o=None, S_T=None, workspace=None,
                out_gate=None, conv=None, stream=None):
    """Chunkwise KDA prefill (``kda_prefill`` in ``include/kda.h``).

    q, k ``[T,H,dk]``, v ``[T,H,dv]`` (bf16 or fp32), log_alpha ``[T,H,dk]`` fp32
    (or ``[T,H]``: one gate per token and head, the Gated DeltaNet form), beta ``[T,H]`` fp32, S0 ``[N,H,dk,dv]`` fp32 or None, cu_seqlens ``[N+1]`` int32
    on the device or None. Returns ``(o [T,H,dv], S_T [N,H,dk,dv])``. Outputs and
    the workspace are allocated with torch when not given. ``max_seqlen`` (host
    int) avoids a device-to-host read of ``cu_seqlens``. ``out_gate = (gate
    [T,H,dv] (dtype of q), weight [dv] fp32, eps)`` fuses the layer's output step
    (``kda_prefill_ex``): o <- RMSNorm(o) * weight * sigmoid(gate). ``conv=(cq, ck, cv)``,
    each None or ``(weight [H*d, W] fp32, state_in, state_out)`` with states
    ``[N, W-1, H*d]`` (None: zeros / not written): q, k, v are the raw projections and the
    short convolution + Swish runs inside the prefill's loads (``kda_prefill_conv``).
    """
    lib = load_library()
    T, H, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if max_seqlen is None:
        if cu_seqlens is None:
            max_seqlen = T
        else:
            c = cu_seqlens.to("cpu", torch.int64)
            max_seqlen = int((c[1:] - c[:-1]).max()) if N > 0 else 0
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    if S_T is None:
        S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    code = _dtype_code(q)
    flags = _flags(l2norm, exact, log_alpha.dim() == 2)
    if workspace is None:
        nbytes = lib.kda_prefill_workspace_size(N, T, max_seqlen, H, dk, dv, code, chunk, flags)
        if nbytes == 0:
            nbytes = 256
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if conv is None:
        rc = lib.kda_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                _ptr(cu_seqlens), N, T, int(max_seqlen), H, dk, dv, code, chunk, flags,
                                _out_gate(out_gate), _ptr(o), _ptr(S_T), _ptr(workspace),
                                workspace.numel(), _stream(stream, dev))
    else:
        cq, ck, cv = conv
        rc = lib.kda_prefill_conv(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                  _ptr(cu_seqlens), N, T, int(max_seqlen), H, dk, dv, code, chunk, flags,
                                  _conv(cq), _conv(ck), _conv(cv), _out_gate(out_gate), _ptr(o), _ptr(S_T),
                                  _ptr(workspace), workspace.numel(), _stream(stream, dev))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_prefill")
    return o, S_T


def kda_prefill_noalloc(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, *, max_seqlen,
                        chunk=64, l2norm=True, exact=False, o, S_T, stream=None):
    """``kda_prefill_noalloc`` in ``include/kda.h``: the prefill with the library's fixed
    scratch array instead of a workspace, for callers that cannot allocate device
    memory. Outputs ``o`` and ``S_T`` are the caller's; nothing is allocated here.
    Calls sharing the array must not overlap on the GPU."""
    lib = load_library()
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    rc = lib.kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                 _ptr(cu_seqlens), N, T, int(max_seqlen), H, dk, dv, _dtype_code(q),
                                 chunk, _flags(l2norm, exact, log_alpha.dim() == 2), _ptr(o), _ptr(S_T),
                                 _stream(stream, q.device))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_prefill_noalloc")
    return o, S_T


def kda_decode_step(q, k, v, log_alpha, beta, S, *, l2norm=True, o=None, out_gate=None,
                    conv=None, stream=None):
    """One KDA decode step (``kda_decode_step`` in ``include/kda.h``), S updated in place.

    q, k ``[N,H,dk]``, v ``[N,H,dv]``, log_alpha ``[N,H,dk]`` (or ``[N,H]``, one gate per
    head) fp32, beta ``[N,H]`` fp32,
    S ``[N,H,dk,dv]`` fp32. Returns o ``[N,H,dv]``. ``conv=(cq, ck, cv)``, each None or
    ``(weight [H*d, W] fp32, state_in, state_out)`` with states ``[N, W-1, H*d]``: the
    short convolution + Swish fused into the loads (``kda_decode_step_conv``).
    """
    lib = load_library()
    N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    if conv is None:
        rc = lib.kda_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S),
                                    N, H, dk, dv, _dtype_code(q), _flags(l2norm, False, log_alpha.dim() == 2),
                                    _out_gate(out_gate), _ptr(o), _stream(stream, q.device))
    else:
        cq, ck, cv = conv
        rc = lib.kda_decode_step_conv(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S),
                                      N, H, dk, dv, _dtype_code(q), _flags(l2norm, False, log_alpha.dim() == 2),
                                      _conv(cq), _conv(ck), _conv(cv), _out_gate(out_gate), _ptr(o),
                                      _stream(stream, q.device))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_decode_step")
    return o


def kda_short_conv_swish(x, weight, cu_seqlens=None, *, state_in=None, state_out=None, bias=None, y=None,
                         stream=None):
    """Causal short convolution + Swish (``kda_short_conv_swish`` in ``include/kda.h``).

    x ``[T, C]`` (or ``[T, H, d]``, C = H * d) in bf16 or fp32, weight ``[C, W]`` fp32,
    states ``[N, W-1, C]`` in x's dtype (state_out may be state_in). Returns y like x.
    With ``bias`` ``[C]`` fp32 (``kda_short_conv_swish_ex``) it is added before the Swish.
    """
    if bias is not None:
        return _conv_bias(x, weight, cu_seqlens, state_in, state_out, bias, y, stream)
    lib = load_library()
    T = x.shape[0]
    C = int(math.prod(x.shape[1:]))
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if y is None:
        y = torch.empty_like(x)
    c = ShortConv(int(weight.shape[-1]), _ptr(weight), _ptr(state_in), _ptr(state_out))
    rc = lib.kda_short_conv_swish(_ptr(x), _ptr(y), ctypes.byref(c), _ptr(cu_seqlens), N, T, C,
                                  _dtype_code(x), _stream(stream, x.device))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_short_conv_swish")
    return y


def kda_backward(q, k, v, log_alpha, beta, do, dS_T=None, S0=None, cu_seqlens=None, *, max_seqlen=None,
                 l2norm=True, workspace=None, want_dS0=True, stream=None):
    """Backward of the prefill (``kda_backward`` in ``include/kda.h``): the gradients of a
    loss through ``o`` and ``S_T`` given ``do = dL/do`` ``[T,H,dv]`` (io dtype) and
    ``dS_T = dL/dS_T`` ``[N,H,dk,dv]`` fp32 (None: zero). Returns fp32
    ``(dq, dk, dv, dlog_alpha, dbeta, dS0)`` (dS0 None unless ``want_dS0``)."""
    lib = load_library()
    T, H, dk = q.shape
    dv = v.shape[-1]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if max_seqlen is None:
        max_seqlen = T if cu_seqlens is None else int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item())
    f32 = dict(dtype=torch.float32, device=q.device)
    dq, dkk = torch.empty((T, H, dk), **f32), torch.empty((T, H, dk), **f32)
    dvv = torch.empty((T, H, dv), **f32)
    dla = torch.empty(tuple(log_alpha.shape), **f32)  # [T,H,dk], or [T,H] with one gate per head
    db = torch.empty((T, H), **f32)
    dS0 = torch.empty((N, H, dk, dv), **f32) if want_dS0 else None
    flags = _flags(l2norm, False, log_alpha.dim() == 2)
    code = _dtype_code(q)
    if workspace is None:
        nbytes = lib.kda_backward_workspace_size(N, T, max_seqlen, H, dk, dv, code, 64, flags)
        if nbytes == 0:
            raise KDAError(KDA_ERR_INVALID_ARG, "kda_backward_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    rc = lib.kda_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(cu_seqlens),
                          N, T, max_seqlen, H, dk, dv, code, 64, flags, _ptr(do), _ptr(dS_T),
                          _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dla), _ptr(db), _ptr(dS0),
                          _ptr(workspace), workspace.numel(), _stream(stream, q.device))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_backward")
    return dq, dkk, dvv, dla, db, dS0


# ------------------------------------------------- the layer around the recurrences ----
# These calls check shapes, dtypes and devices here (the C ABI sees only pointers), may be made on
# tensors of a device other than the current one, and take what they allocate from the pool of the
# stream they run on.

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(device, stream, body):
    """``body(handle of the stream)`` with the tensors' device current, and ``stream`` if one is given."""
    index = device.index
    if stream is None:
        if _current_device() == index:
            return body(_raw_stream(index))
        with torch.cuda.device(index):
            return body(_raw_stream(index))
    if stream.device != device:
        raise ValueError("stream must be on %s, got %s" % (device, stream.device))
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _arg(name, t, dtype, shape, device):
    """The address of a contiguous ``t`` of this dtype and shape on this device (None: NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr() or None
    if t.device != device:
        raise ValueError("%s must live on %s, got %s" % (name, device, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _out(name, t, like, device):
    """(``t``, its address): a caller's output checked against ``like``, or a new one."""
    if t is None:
        t = torch.empty_like(like)
        return t, t.data_ptr() or None
    return t, _arg(name, t, like.dtype, like.shape, device)


def _scratch(workspace, device):
    """(address, bytes) of a workspace tensor (None: none)."""
    if workspace is None:
        return None, 0
    return _arg("workspace", workspace, workspace.dtype, workspace.shape, device), workspace.numel() * workspace.element_size()


def _cuda(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    return t.device


def _seqs(cu_seqlens, device):
    """(number of sequences, address) of an int32 ``cu_seqlens`` [N + 1] (None: one sequence)."""
    if cu_seqlens is None:
        return 1, None
    return cu_seqlens.numel() - 1, _arg("cu_seqlens", cu_seqlens, torch.int32, (max(cu_seqlens.numel(), 2),), device)


def _ssm(x, dt, B, C, A, z, D, dt_bias):
    """Checks a scan's inputs; (device, rows, kda_ssm, addresses of x, dt, B, C, z)."""
    dev = _cuda(x)
    if x.dim() < 2 or B.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [T, channels], B and C [T, groups, states], A [channels, states]")
    T, (ch, n), f32 = x.shape[0], A.shape, torch.float32
    if math.prod(x.shape[1:]) != ch:
        raise ValueError("x must have the %d channels of A, got %s" % (ch, tuple(x.shape)))
    bc = (T, B.shape[1], n)
    p = Ssm(ch, n, B.shape[1], _arg("A", A, f32, (ch, n), dev), _arg("D", D, f32, (ch,), dev),
            _arg("dt_bias", dt_bias, f32, (ch,), dev))
    io = x.dtype
    return dev, T, p, (_arg("x", x, io, x.shape, dev), _arg("dt", dt, io, x.shape, dev), _arg("B", B, io, bc, dev),
                       _arg("C", C, io, bc, dev), _arg("z", z, io, x.shape, dev))


def kda_ssm_prefill(x, dt, B, C, A, S0=None, cu_seqlens=None, *, D=None, dt_bias=None, z=None, softplus=True,
                    save_states=False, y=None, S_T=None, workspace=None, stream=None):
    """Selective state space scan over packed prompts (``kda_ssm_prefill`` in ``include/kda.h``).

    x, dt, z ``[T, channels]`` (trailing axes may be split, as ``[T, H, d]``) and B, C
    ``[T, groups, states]`` in bf16 or fp32; A ``[channels, states]``, D, dt_bias ``[channels]`` and
    S0 ``[N, channels, states]`` fp32; cu_seqlens ``[N + 1]`` int32 on the device or None. Returns
    ``(y, S_T)``, and with ``save_states`` the tile states that ``kda_ssm_backward`` reads as a third.
    Outputs and the workspace are allocated with torch when not given.
    """
    lib = load_library()
    dev, T, p, (px, pdt, pB, pC, pz) = _ssm(x, dt, B, C, A, z, D, dt_bias)
    code = _dtype_code(x)
    N, pcu = _seqs(cu_seqlens, dev)
    f32, st = torch.float32, (N, p.channels, p.states)
    def body(on):
        out, py = _out("y", y, x, dev)
        last = S_T
        if last is None:
            last = A.new_empty(st) if S0 is None else torch.empty_like(S0)
        nbytes = 0 if workspace is not None else lib.kda_ssm_prefill_workspace_size(N, T, p.channels, p.states, p.groups)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else workspace
        tiles = A.new_empty((T // KDA_SSM_TILE + N, p.channels, p.states)) if save_states else None
        rc = lib.kda_ssm_prefill(px, pdt, pB, pC, pz, ctypes.byref(p), _arg("S0", S0, f32, st, dev), pcu, N, T, code,
                                 KDA_FLAG_SOFTPLUS if softplus else 0, py, _arg("S_T", last, f32, st, dev),
                                 tiles.data_ptr() or None if save_states else None, *_scratch(ws, dev), on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_ssm_prefill")
        return (out, last, tiles) if save_states else (out, last)

    return _run(dev, stream, body)


def kda_ssm_step(x, dt, B, C, A, S, *, D=None, dt_bias=None, z=None, softplus=True, y=None, stream=None):
    """One token of each sequence through the selective scan (``kda_ssm_step`` in ``include/kda.h``):
    x, dt, z ``[N, channels]``, B, C ``[N, groups, states]``, S ``[N, channels, states]`` fp32 updated in
    place. Returns y like x."""
    lib = load_library()
    dev, N, p, (px, pdt, pB, pC, pz) = _ssm(x, dt, B, C, A, z, D, dt_bias)
    code = _dtype_code(x)
    pS = _arg("S", S, torch.float32, (N, p.channels, p.states), dev)
    def body(on):
        out, py = _out("y", y, x, dev)
        rc = lib.kda_ssm_step(px, pdt, pB, pC, pz, ctypes.byref(p), pS, N, code, KDA_FLAG_SOFTPLUS if softplus else 0,
                              py, on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_ssm_step")
        return out

    return _run(dev, stream, body)


SsmGradients = collections.namedtuple("SsmGradients", "dx ddt dB dC dz dA dD ddt_bias dS0")


def kda_ssm_backward(x, dt, B, C, A, dy, tile_states, dS_T=None, S0=None, cu_seqlens=None, *, D=None, dt_bias=None,
                     z=None, softplus=True, workspace=None, stream=None):
    """Backward of ``kda_ssm_prefill`` (``kda_ssm_backward`` in ``include/kda.h``): the gradients of a loss
    through y and S_T given ``dy = dL/dy`` (like x) and ``dS_T = dL/dS_T`` (fp32, None: zero), with the
    ``tile_states`` that the forward call returned. Returns fp32 ``SsmGradients(dx, ddt, dB, dC, dz, dA, dD,
    ddt_bias, dS0)``, each shaped like its input (None where that is None)."""
    lib = load_library()
    dev, T, p, (px, pdt, pB, pC, pz) = _ssm(x, dt, B, C, A, z, D, dt_bias)
    code = _dtype_code(x)
    N, pcu = _seqs(cu_seqlens, dev)
    f32, st = torch.float32, (N, p.channels, p.states)
    pt = _arg("tile_states", tile_states, f32, (T // KDA_SSM_TILE + N, p.channels, p.states), dev)
    pdy, pdS, pS0 = _arg("dy", dy, x.dtype, x.shape, dev), _arg("dS_T", dS_T, f32, st, dev), _arg("S0", S0, f32, st, dev)
    def body(on):
        nonlocal workspace
        g = SsmGradients(*(None if t is None else torch.empty_like(t, dtype=f32)
                           for t in (x, dt, B, C, z, A, D, dt_bias, S0)))
        if workspace is None:
            nbytes = lib.kda_ssm_backward_workspace_size(N, T, p.channels, p.states, p.groups)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        rc = lib.kda_ssm_backward(px, pdt, pB, pC, pz, ctypes.byref(p), pS0, pcu, N, T, code,
                                  KDA_FLAG_SOFTPLUS if softplus else 0, pt, pdy, pdS,
                                  ctypes.byref(SsmGrads(*(None if t is None else t.data_ptr() or None for t in g))),
                                  *_scratch(workspace, dev), on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_ssm_backward")
        return g

    return _run(dev, stream, body)


def _conv_args(x, weight, bias, num_seqs, state_in, state_out):
    """Checks a convolution's inputs; (device, rows, C, dtype code, kda_short_conv, addresses of x and bias)."""
    dev = _cuda(x)
    if x.dim() < 2 or weight.dim() != 2:
        raise ValueError("x must be [T, C], weight [C, W]")
    T, C, W = x.shape[0], math.prod(x.shape[1:]), weight.shape[1]
    st = (num_seqs, W - 1, C)
    c = ShortConv(W, _arg("weight", weight, torch.float32, (C, W), dev), _arg("state_in", state_in, x.dtype, st, dev),
                  _arg("state_out", state_out, x.dtype, st, dev))
    return dev, T, C, _dtype_code(x), c, _arg("x", x, x.dtype, x.shape, dev), _arg("bias", bias, torch.float32, (C,), dev)


def _conv_bias(x, weight, cu_seqlens, state_in, state_out, bias, y, stream):
    lib = load_library()
    N, pcu = _seqs(cu_seqlens, _cuda(x))
    dev, T, C, code, c, px, pb = _conv_args(x, weight, bias, N, state_in, state_out)
    def body(on):
        out, py = _out("y", y, x, dev)
        rc = lib.kda_short_conv_swish_ex(px, py, ctypes.byref(c), pb, pcu, N, T, C, code, on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_short_conv_swish")
        return out

    return _run(dev, stream, body)


def kda_short_conv_step(x, weight, state, *, bias=None, y=None, stream=None):
    """The short convolution + Swish of one token of each sequence (``kda_short_conv_step`` in
    ``include/kda.h``): x ``[N, C]``, weight ``[C, W]`` and bias ``[C]`` fp32, state ``[N, W-1, C]`` in x's
    dtype, shifted in place (None for W = 1). Returns y like x."""
    lib = load_library()
    dev, N, C, code, c, px, pb = _conv_args(x, weight, bias, x.shape[0], None, state)
    def body(on):
        out, py = _out("y", y, x, dev)
        rc = lib.kda_short_conv_step(px, py, ctypes.byref(c), pb, N, C, code, on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_short_conv_step")
        return out

    return _run(dev, stream, body)


def kda_short_conv_backward(x, weight, dy, cu_seqlens=None, *, bias=None, state_in=None, want_dstate=False,
                            workspace=None, stream=None):
    """Backward of ``kda_short_conv_swish`` (``kda_short_conv_backward`` in ``include/kda.h``) given
    ``dy = dL/dy`` like x, in fp32 or x's dtype. Returns fp32 ``(dx like x, dweight [C, W], dbias [C] (None
    without bias), dstate [N, W-1, C] (None unless want_dstate))``."""
    lib = load_library()
    N, pcu = _seqs(cu_seqlens, _cuda(x))
    dev, T, C, code, c, px, pb = _conv_args(x, weight, bias, N, state_in, None)
    f32 = dict(dtype=torch.float32, device=dev)
    pdy = _arg("dy", dy, dy.dtype, x.shape, dev)
    def body(on):
        nonlocal workspace
        dx, dw = torch.empty_like(x, dtype=torch.float32), torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        ds = torch.empty((N, weight.shape[1] - 1, C), **f32) if want_dstate else None
        if workspace is None:
            nbytes = lib.kda_short_conv_backward_workspace_size(T, C, weight.shape[1])
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        rc = lib.kda_short_conv_backward(px, ctypes.byref(c), pb, pcu, N, T, C, code, pdy, _dtype_code(dy),
                                         dx.data_ptr() or None, dw.data_ptr(), None if db is None else db.data_ptr(),
                                         None if ds is None else ds.data_ptr() or None, *_scratch(workspace, dev), on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_short_conv_backward")
        return dx, dw, db, ds

    return _run(dev, stream, body)


def _norm_args(y, r, w_pre, w_post, gate, scale, res_scale, eps):
    """Checks the norms' inputs; (device, kda_residual_norm_args)."""
    dev = _cuda(y)
    D, rows = y.shape[-1], math.prod(y.shape[:-1])
    res = y.dtype if r is None else r.dtype
    code = _dtype_code(y)
    w = lambda n, t: _arg(n, t, torch.float32, (D,), dev)
    return dev, ResidualNorm(_arg("y", y, y.dtype, y.shape, dev), _arg("r", r, res, y.shape, dev),
                             _arg("gate", gate, y.dtype, y.shape, dev), w("w_post", w_post), w("scale", scale),
                             w("w_pre", w_pre), float(res_scale), float(eps), rows, D, code,
                             code if r is None else _dtype_code(r))


def kda_residual_norm(y, r=None, w_pre=None, *, w_post=None, gate=None, scale=None, res_scale=1.0, eps=1e-6, x=None,
                      r_out=None, stream=None):
    """The norm after a block, its gate and residual scale, the residual stream and the norm before the
    next block, in one pass (``kda_residual_norm`` in ``include/kda.h``):

        r_out = res_scale * r + scale * sigmoid(gate) * RMSNorm(y) * w_post,   x = RMSNorm(r_out) * w_pre.

    y, gate ``[..., D]`` in bf16 or fp32; r, r_out in y's dtype or fp32; w_post, scale, w_pre ``[D]`` fp32.
    Each of r, w_pre, w_post, gate, scale may be None (no stream yet, no norm before, no norm after, no
    gate, scale 1). Returns ``(x, r_out)`` (x None without w_pre); ``r_out`` may be ``r``."""
    lib = load_library()
    dev, a = _norm_args(y, r, w_pre, w_post, gate, scale, res_scale, eps)
    def body(on):
        new_x, px = (None, None) if x is None and w_pre is None else _out("x", x, y, dev)
        new_r, pr = _out("r_out", r_out, y if r is None else r, dev)
        rc = lib.kda_residual_norm(ctypes.byref(a), px, pr, on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_residual_norm")
        return new_x, new_r

    return _run(dev, stream, body)


ResidualNormGradients = collections.namedtuple("ResidualNormGradients", "dy dr dgate dw_post dscale dw_pre")


def kda_residual_norm_backward(y, r, w_pre, dx, dr_out=None, *, w_post=None, gate=None, scale=None, res_scale=1.0,
                               eps=1e-6, workspace=None, stream=None):
    """Backward of ``kda_residual_norm`` (``kda_residual_norm_backward`` in ``include/kda.h``) given
    ``dx = dL/dx`` (like y; None without w_pre) and ``dr_out = dL/dr_out`` (fp32, None: zero). Returns fp32
    ``ResidualNormGradients(dy, dr, dgate, dw_post, dscale, dw_pre)``, each None where its input is."""
    lib = load_library()
    dev, a = _norm_args(y, r, w_pre, w_post, gate, scale, res_scale, eps)
    pdx, pdr = _arg("dx", dx, y.dtype, y.shape, dev), _arg("dr_out", dr_out, torch.float32, y.shape, dev)
    def body(on):
        nonlocal workspace
        g = ResidualNormGradients(*(None if t is None else torch.empty_like(t, dtype=torch.float32)
                                    for t in (y, r, gate, w_post, scale, w_pre)))
        if workspace is None:
            nbytes = lib.kda_residual_norm_backward_workspace_size(a.rows, a.D)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        rc = lib.kda_residual_norm_backward(ctypes.byref(a), pdx, pdr, *(None if t is None else t.data_ptr() or None for t in g),
                                            *_scratch(workspace, dev), on)
        if rc != KDA_OK:
            raise KDAError(rc, "kda_residual_norm_backward")
        return g

    return _run(dev, stream, body)
