"""Thin Python binding of libkdn.so (the C ABI declared in include/kdn.h).

The raw functions keep the C names (``kdn_forward_chunkwise``, ``kdn_decode_step``,
``kdn_gain_scan``, ``kdn_backward``, ``kdn_workspace_size``, ``kdn_last_device_error``,
``kdn_status_string``, ``kdn_version``) and take plain integers for pointers.
``forward``, ``backward``, ``decode_step`` and ``gain_scan`` marshal torch CUDA tensors into those
calls: they allocate outputs and workspace with torch and pass the current stream.  So do
``linear_forward``, ``linear_backward``, ``linear_decode_step`` and ``linear_decode_tokens`` (linear
attention with a decay for each head) and ``layer_norm`` and ``layer_norm_backward``, whose common call
goes through the extension module ``_kdn_marshal.so`` instead of ctypes (where it is built: it saves microseconds).
Every step of the computation runs in the library's kernels; there is no CPU or
PyTorch fallback -- a missing library or device raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkdn.so")
MARSHAL_PATH = os.path.join(PKG, "_kdn_marshal.so")

KDN_OK, KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED, KDN_ERR_CUDA, KDN_ERR_TIMEOUT, KDN_ERR_RANGE, KDN_ERR_WORKSPACE = range(7)
KDN_DTYPE_F32, KDN_DTYPE_BF16 = 0, 1


class KdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {kdn_status_string(code)} (status {code})")


class kdn_problem_t(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("d_k", ctypes.c_int),
                ("d_v", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("mu", ctypes.c_float), ("chunk", ctypes.c_int),
                ("max_seqlen", ctypes.c_int), ("variant", ctypes.c_int)]


class kdn_linear_problem_t(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("d_k", ctypes.c_int),
                ("d_v", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("scale", ctypes.c_float), ("decay", ctypes.c_int)]


KDN_DECAY_NONE, KDN_DECAY_TOKEN, KDN_DECAY_HEAD = 0, 1, 2

_lib = None
_lock = threading.Lock()
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_PP = ctypes.POINTER(kdn_problem_t)
_PL = ctypes.POINTER(kdn_linear_problem_t)
_ll, _psz = ctypes.c_longlong, ctypes.POINTER(_sz)

_SIGS = {
    "kdn_workspace_size": (_i, [_PP, ctypes.POINTER(_sz)]),
    "kdn_forward_chunkwise": (_i, [_PP] + [_vp] * 6 + [_vp] * 2 + [_vp] * 3 + [_vp, _sz, _vp]),
    "kdn_decode_step": (_i, [_i, _i, _i, _i, _i, _f] + [_vp] * 6 + [_vp] * 3 + [_vp]),
    "kdn_decode_tokens": (_i, [_i, _i, _i, _i, _i, _i, _f] + [_vp] * 6 + [_vp] * 3 + [_vp]),
    "kdn_decode_tokens_iso": (_i, [_i, _i, _i, _i, _i, _i, _f] + [_vp] * 6 + [_vp] * 3 + [_vp]),
    "kdn_gain_scan": (_i, [_PP] + [_vp] * 4 + [_vp] + [_vp] * 3 + [_vp, _sz, _vp]),
    "kdn_last_device_error": (_i, [_vp]),
    "kdn_selftest_bounded_wait": (_i, [ctypes.c_longlong, _vp]),
    "kdn_status_string": (ctypes.c_char_p, [_i]),
    "kdn_version": (ctypes.c_char_p, []),
    "kdn_execution_path": (_i, [_PP]),
    "kdn_gain_scan_noalloc": (_i, [_PP] + [_vp] * 4 + [_vp] + [_vp] * 3 + [_vp]),
    "kdn_backward_workspace_size": (_i, [_PP, ctypes.POINTER(_sz)]),
    "kdn_linear_workspace_size": (_i, [_PL, _psz]),
    "kdn_linear_forward": (_i, [_PL] + [_vp] * 7 + [_vp, _sz, _vp]),
    "kdn_linear_decode_tokens": (_i, [_i] * 6 + [_f, _i] + [_vp] * 6 + [_vp]),
    "kdn_linear_backward_workspace_size": (_i, [_PL, _psz]),
    "kdn_linear_backward": (_i, [_PL] + [_vp] * 12 + [_vp, _sz, _vp]),
    "kdn_layer_norm": (_i, [_ll, _i, _i, _i, _f] + [_vp] * 6 + [_vp]),
    "kdn_layer_norm_backward_workspace_size": (_i, [_ll, _i, _i, _psz]),
    "kdn_layer_norm_backward": (_i, [_ll, _i, _i, _i] + [_vp] * 8 + [_vp, _sz, _vp]),
    "kdn_backward": (_i, [_PP] + [_vp] * 6 + [_vp] * 2 + [_vp] * 3 + [_vp] * 6 + [_vp] * 2 + [_vp, _sz, _vp]),
}


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkdn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libkdn.so not found at {path}; build it with "
                                   "`python -m kalman_delta_rule_b200.build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            _lib = lib
    return _lib


# ------------------------------------------------------------------ raw C names
def kdn_workspace_size(problem: kdn_problem_t) -> int:
    n = ctypes.c_size_t(0)
    st = load().kdn_workspace_size(ctypes.byref(problem), ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, "kdn_workspace_size")
    return n.value


def kdn_forward_chunkwise(problem, q, k, v, alpha, sigma, r, S0, P0, o, S_out, P_out, workspace, workspace_bytes, stream):
    return load().kdn_forward_chunkwise(ctypes.byref(problem), q, k, v, alpha, sigma, r, S0, P0, o, S_out, P_out,
                                        workspace, workspace_bytes, stream)


def kdn_decode_step(N, H, d_k, d_v, in_dtype, mu, q, k, v, alpha, sigma, r, S, P, o, stream):
    return load().kdn_decode_step(N, H, d_k, d_v, in_dtype, mu, q, k, v, alpha, sigma, r, S, P, o, stream)


def kdn_decode_tokens(N, n_tokens, H, d_k, d_v, in_dtype, mu, q, k, v, alpha, sigma, r, S, P, o, stream):
    return load().kdn_decode_tokens(N, n_tokens, H, d_k, d_v, in_dtype, mu, q, k, v, alpha, sigma, r, S, P, o, stream)


def kdn_decode_tokens_iso(N, n_tokens, H, d_k, d_v, in_dtype, mu, q, k, v, alpha, sigma, r, S, P, o, stream):
    return load().kdn_decode_tokens_iso(N, n_tokens, H, d_k, d_v, in_dtype, mu, q, k, v, alpha, sigma, r, S, P, o,
                                        stream)


def kdn_gain_scan(problem, k, alpha, sigma, r, P0, g, beta_eff, P_out, workspace, workspace_bytes, stream):
    return load().kdn_gain_scan(ctypes.byref(problem), k, alpha, sigma, r, P0, g, beta_eff, P_out,
                                workspace, workspace_bytes, stream)


def kdn_gain_scan_noalloc(problem, k, alpha, sigma, r, P0, g, beta_eff, P_out, stream):
    """The gain scan on the library's fixed scratch array: for callers that cannot
    allocate device memory when they call (no workspace argument)."""
    return load().kdn_gain_scan_noalloc(ctypes.byref(problem), k, alpha, sigma, r, P0, g, beta_eff, P_out, stream)


def kdn_backward_workspace_size(problem: kdn_problem_t) -> int:
    n = ctypes.c_size_t(0)
    st = load().kdn_backward_workspace_size(ctypes.byref(problem), ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, "kdn_backward_workspace_size")
    return n.value


def kdn_backward(problem, q, k, v, alpha, sigma, r, S0, P0, d_o, dS_T, dP_T, dq, dk, dv, dalpha, dsigma, dr,
                 dS0, dP0, workspace, workspace_bytes, stream):
    return load().kdn_backward(ctypes.byref(problem), q, k, v, alpha, sigma, r, S0, P0, d_o, dS_T, dP_T,
                               dq, dk, dv, dalpha, dsigma, dr, dS0, dP0, workspace, workspace_bytes, stream)


def kdn_linear_workspace_size(problem: kdn_linear_problem_t) -> int:
    n = ctypes.c_size_t(0)
    _check(load().kdn_linear_workspace_size(ctypes.byref(problem), ctypes.byref(n)), "kdn_linear_workspace_size")
    return n.value


def kdn_linear_forward(problem, q, k, v, g, S0, o, S_out, workspace, workspace_bytes, stream):
    return load().kdn_linear_forward(ctypes.byref(problem), q, k, v, g, S0, o, S_out, workspace, workspace_bytes, stream)


def kdn_linear_decode_tokens(N, n_tokens, H, d_k, d_v, in_dtype, scale, decay, q, k, v, g, S, o, stream):
    return load().kdn_linear_decode_tokens(N, n_tokens, H, d_k, d_v, in_dtype, scale, decay, q, k, v, g, S, o, stream)


def kdn_linear_backward_workspace_size(problem: kdn_linear_problem_t) -> int:
    n = ctypes.c_size_t(0)
    _check(load().kdn_linear_backward_workspace_size(ctypes.byref(problem), ctypes.byref(n)),
           "kdn_linear_backward_workspace_size")
    return n.value


def kdn_linear_backward(problem, q, k, v, g, S0, d_o, dS_T, dq, dk, dv, dg, dS0, workspace, workspace_bytes, stream):
    return load().kdn_linear_backward(ctypes.byref(problem), q, k, v, g, S0, d_o, dS_T, dq, dk, dv, dg, dS0,
                                      workspace, workspace_bytes, stream)


def kdn_layer_norm(n, G, d, dtype, eps, x, weight, bias, y, mean, rstd, stream):
    return load().kdn_layer_norm(n, G, d, dtype, eps, x, weight, bias, y, mean, rstd, stream)


def kdn_layer_norm_backward_workspace_size(n: int, G: int, d: int) -> int:
    b = ctypes.c_size_t(0)
    _check(load().kdn_layer_norm_backward_workspace_size(n, G, d, ctypes.byref(b)), "kdn_layer_norm_backward_workspace_size")
    return b.value


def kdn_layer_norm_backward(n, G, d, dtype, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, workspace_bytes,
                            stream):
    return load().kdn_layer_norm_backward(n, G, d, dtype, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace,
                                          workspace_bytes, stream)


def kdn_last_device_error(stream=None) -> int:
    return load().kdn_last_device_error(stream)


def kdn_execution_path(problem) -> int:
    return load().kdn_execution_path(ctypes.byref(problem))


def kdn_status_string(code: int) -> str:
    return load().kdn_status_string(code).decode()


def kdn_version() -> str:
    return load().kdn_version().decode()


# ------------------------------------------------------------------ torch marshalling
def _torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("kalman_delta_rule_b200 needs a CUDA device (B200, sm_100a)")
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return KDN_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDN_DTYPE_F32
    raise TypeError(f"unsupported input dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream or None


def _check(st: int, where: str):
    if st != KDN_OK:
        raise KdnError(st, where)


VARIANTS = {"diagonal": 0, "isotropic": 1}


def make_problem(q, v, H=None, cu_seqlens=None, mu: float = 1.0, chunk: int = 64, max_seqlen: int = 0,
                 variant: str = "diagonal") -> kdn_problem_t:
    B, T, H_, dk = q.shape
    p = kdn_problem_t()
    p.B, p.T, p.H, p.d_k, p.d_v = B, T, H_, dk, v.shape[-1]
    p.cu_seqlens = _ptr(cu_seqlens)
    p.num_seqs = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    p.in_dtype = _dtype_code(q)
    p.mu = float(mu)
    p.chunk = int(chunk)
    p.max_seqlen = int(max_seqlen)
    p.variant = VARIANTS[variant]
    return p


def forward(q, k, v, alpha, sigma, r, cu_seqlens=None, S0=None, P0=None, mu: float = 1.0, chunk: int = 64,
            o=None, S_out=None, P_out=None, workspace=None, want_state: bool = True, stream=None,
            variant: str = "diagonal", max_seqlen: int = 0):
    """Run kdn_forward_chunkwise on torch tensors ([B,T,H,d]; varlen: B = 1 with int32 cu_seqlens).

    Returns (o, S_out, P_out); P is [N,H,dk] (diagonal) or [N,H] (isotropic).  Outputs are
    allocated when not given; so is the workspace when ``workspace`` is None (``False``
    passes none: the tensor-core path needs one, so such a call runs the fp32 chunk kernel)."""
    torch = _torch()
    p = make_problem(q, v, cu_seqlens=cu_seqlens, mu=mu, chunk=chunk, variant=variant, max_seqlen=max_seqlen)
    N = p.num_seqs
    dev = q.device
    if o is None:
        o = torch.empty(q.shape[:3] + (p.d_v,), dtype=q.dtype, device=dev)
    if want_state and S_out is None:
        S_out = torch.empty((N, p.H, p.d_k, p.d_v), dtype=torch.float32, device=dev)
    if want_state and P_out is None:
        P_out = torch.empty((N, p.H) + ((p.d_k,) if p.variant == 0 else ()), dtype=torch.float32, device=dev)
    if workspace is False:
        workspace = None
    elif workspace is None:
        need = kdn_workspace_size(p)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = kdn_forward_chunkwise(p, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(sigma), _ptr(r), _ptr(S0), _ptr(P0),
                               _ptr(o), _ptr(S_out), _ptr(P_out), _ptr(workspace), wbytes, _stream_handle(stream))
    _check(st, "kdn_forward_chunkwise")
    return o, S_out, P_out


def backward(q, k, v, alpha, sigma, r, d_o, cu_seqlens=None, S0=None, P0=None, dS=None, dP=None, mu: float = 1.0,
             workspace=None, want_initial: bool = True, stream=None, variant: str = "diagonal", max_seqlen: int = 0):
    """Run kdn_backward on torch tensors laid out as for ``forward``.

    Returns a dict of fp32 gradients of <o, d_o> + <S_T, dS> + <P_T, dP>: dq, dk, dv,
    dalpha, dsigma ([B,T,H,d]), dr ([B,T,H]) and, with ``want_initial``, dS0 [N,H,dk,dv]
    and dP0 ([N,H,dk] diagonal, [N,H] isotropic).  The workspace is allocated when not given.
    ``max_seqlen`` (packed sequences; 0 = unknown) bounds the chunk-parallel work lists."""
    torch = _torch()
    if d_o.dtype != q.dtype:
        raise ValueError("d_o must have the dtype of the inputs")
    p = make_problem(q, v, cu_seqlens=cu_seqlens, mu=mu, chunk=0, variant=variant, max_seqlen=max_seqlen)
    N = p.num_seqs
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty(q.shape, **f32), dk=torch.empty(k.shape, **f32), dv=torch.empty(v.shape, **f32),
               dalpha=torch.empty(alpha.shape, **f32), dsigma=torch.empty(sigma.shape, **f32),
               dr=torch.empty(r.shape, **f32))
    if want_initial:
        out["dS0"] = torch.empty((N, p.H, p.d_k, p.d_v), **f32)
        out["dP0"] = torch.empty((N, p.H) + ((p.d_k,) if p.variant == 0 else ()), **f32)
    if workspace is None:
        workspace = torch.empty(kdn_backward_workspace_size(p), dtype=torch.uint8, device=dev)
    wbytes = workspace.numel() * workspace.element_size()
    st = kdn_backward(p, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(sigma), _ptr(r), _ptr(S0), _ptr(P0),
                      _ptr(d_o), _ptr(dS), _ptr(dP), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                      _ptr(out["dalpha"]), _ptr(out["dsigma"]), _ptr(out["dr"]), _ptr(out.get("dS0")),
                      _ptr(out.get("dP0")), _ptr(workspace), wbytes, _stream_handle(stream))
    _check(st, "kdn_backward")
    return out


def decode_step(q, k, v, alpha, sigma, r, S, P, mu: float = 1.0, o=None, stream=None, variant: str = "diagonal"):
    """One decode step on [N,H,d] token tensors; S [N,H,dk,dv] and P [N,H,dk] ([N,H] isotropic)
    updated in place."""
    torch = _torch()
    if VARIANTS[variant] == 1:
        o4 = None if o is None else o.unsqueeze(1)
        return decode_tokens(*(x.unsqueeze(1) for x in (q, k, v, alpha, sigma, r)), S, P, mu=mu, o=o4,
                             stream=stream, variant=variant).squeeze(1)
    N, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    st = kdn_decode_step(N, H, dk, dv, _dtype_code(q), float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                         _ptr(sigma), _ptr(r), _ptr(S), _ptr(P), _ptr(o), _stream_handle(stream))
    _check(st, "kdn_decode_step")
    return o


def decode_tokens(q, k, v, alpha, sigma, r, S, P, mu: float = 1.0, o=None, stream=None,
                  variant: str = "diagonal"):
    """n tokens per sequence in one launch on [N, n, H, d] token tensors; S, P updated in place
    (P [N,H,dk] diagonal, [N,H] isotropic)."""
    torch = _torch()
    N, n, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((N, n, H, dv), dtype=q.dtype, device=q.device)
    fn = kdn_decode_tokens_iso if VARIANTS[variant] == 1 else kdn_decode_tokens
    st = fn(N, n, H, dk, dv, _dtype_code(q), float(mu), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                           _ptr(sigma), _ptr(r), _ptr(S), _ptr(P), _ptr(o), _stream_handle(stream))
    _check(st, "kdn_decode_tokens")
    return o


def gain_scan(k, alpha, sigma, r, cu_seqlens=None, P0=None, mu: float = 1.0, chunk: int = 64,
              want_g: bool = True, want_beta: bool = True, workspace=None, stream=None, max_seqlen: int = 0):
    """Run kdn_gain_scan; returns (g [B,T,H,dk] fp32 or None, beta_eff [B,T,H] or None, P_out [N,H,dk])."""
    torch = _torch()
    p = make_problem(k, k, cu_seqlens=cu_seqlens, mu=mu, chunk=chunk, max_seqlen=max_seqlen)
    dev = k.device
    g = torch.empty(k.shape, dtype=torch.float32, device=dev) if want_g else None
    be = torch.empty(k.shape[:3], dtype=torch.float32, device=dev) if want_beta else None
    P_out = torch.empty((p.num_seqs, p.H, p.d_k), dtype=torch.float32, device=dev)
    need = kdn_workspace_size(p)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = kdn_gain_scan(p, _ptr(k), _ptr(alpha), _ptr(sigma), _ptr(r), _ptr(P0), _ptr(g), _ptr(be), _ptr(P_out),
                       _ptr(workspace), wbytes, _stream_handle(stream))
    _check(st, "kdn_gain_scan")
    return g, be, P_out


# ------------------------------------------------------------------ linear attention, layer norm
# These wrappers serve single-token decoding too, where the kernel takes a few microseconds.  The common call --
# contiguous tensors of the expected types and shapes on the current device, its current stream, no caller's workspace --
# goes from the tensors to the C ABI in one native step (csrc/kdn_marshal.cpp).  For any other that returns None, and
# the code here checks, dispatches and raises.  (A call that the library began and failed in raises there.)
_native_mod = None
_mod = None
_raw_stream = None   # device index -> handle of its current stream


def _cuda():
    """torch, once a CUDA device has been seen."""
    global _mod, _raw_stream
    if _mod is None:
        torch = _torch()
        # (a Stream object costs several microseconds; torch's own code generators read the handle this way)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _mod = torch
    return _mod


class _NoNative:
    """In the place of an extension module that is not there: every call is left to the code here."""
    linear_forward = linear_decode = linear_backward = layer_norm = layer_norm_backward = staticmethod(lambda *a: None)


def _native_module(torch):
    """The built extension module, or None (with a warning) if it is missing or was built for another torch."""
    import importlib.util
    import sys
    import warnings
    abi, why = f"{torch.__version__} {sys.implementation.cache_tag}", "is not built"
    if os.path.exists(MARSHAL_PATH):
        try:
            spec = importlib.util.spec_from_file_location("_kdn_marshal", MARSHAL_PATH)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            if mod.abi == abi:
                return mod
            why = f"was built for {mod.abi}, this is {abi}"
        except ImportError as e:
            why = f"cannot be loaded ({e})"
    warnings.warn(f"{MARSHAL_PATH} {why}; calls go through ctypes, several microseconds slower each "
                  "(`python -m kalman_delta_rule_b200.build` builds it)")
    return None


def _native():
    """The extension module, bound to the loaded library's functions."""
    global _native_mod
    lib, torch = load(), _cuda()
    with _lock:
        if _native_mod is None:
            mod = _native_module(torch)
            if mod is None:
                _native_mod = _NoNative
                return _native_mod
            names = ("linear_workspace_size", "linear_forward", "linear_decode_tokens", "linear_backward_workspace_size",
                     "linear_backward", "layer_norm", "layer_norm_backward_workspace_size", "layer_norm_backward")
            mod.bind(*(ctypes.cast(getattr(lib, "kdn_" + n), _vp).value for n in names))
            mod.raise_with(KdnError)
            _native_mod = mod
    return _native_mod


def _type_of(torch, name, t):
    if t.dtype is torch.bfloat16:
        return KDN_DTYPE_BF16
    if t.dtype is torch.float32:
        return KDN_DTYPE_F32
    raise TypeError(f"{name} is {t.dtype} (float32 or bfloat16 expected)")


def _expect(name, t, shape, dtype, device):
    """Raise unless ``t`` is a contiguous tensor of this shape, type and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _device_of(name, t):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} is on {dev}, expected a CUDA device")
    return dev


def _launch(torch, dev, stream, fn):
    """fn(stream handle) with the tensors' device and the caller's stream current: outputs and workspace come from
    that stream's allocator, and the kernels are launched on it.  ``stream`` None is that device's current one."""
    if stream is None:
        if torch.cuda.current_device() == dev.index:
            return fn(_raw_stream(dev.index) or None)
        with torch.cuda.device(dev):
            return fn(_raw_stream(dev.index) or None)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        return fn(stream.cuda_stream or None)


def _work(torch, name, workspace, need, dev):
    """(the caller's workspace, or a new one of ``need`` bytes; its pointer; its bytes)"""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"{name}: the workspace must be contiguous and on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


_sizes = {}   # workspace bytes by problem: a function of the sizes alone


def _need(fn, p, packed):
    key = (fn, p.B, p.T, p.H, p.d_k, p.d_v, p.num_seqs, packed, p.in_dtype)
    n = _sizes.get(key)
    if n is None:
        if len(_sizes) > 4096:
            _sizes.clear()
        n = _sizes[key] = fn(p)
    return n


def _linear_problem(q, k, v, g, cu_seqlens, scale):
    torch = _mod or _cuda()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B, T, H, d]")
    shape, dtype, dev = q.shape, q.dtype, _device_of("q", q)
    B, T, H, dk = shape
    dv = v.shape[3]
    code = _type_of(torch, "q", q)
    _expect("q", q, shape, dtype, dev)
    _expect("k", k, shape, dtype, dev)
    _expect("v", v, (B, T, H, dv), dtype, dev)
    n, cu = B, None
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be one-dimensional, with at least one entry")
        _expect("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, dev)
        if B != 1:
            raise ValueError("packed sequences need B = 1")
        n, cu = cu_seqlens.shape[0] - 1, cu_seqlens.data_ptr()
    decay, gp = KDN_DECAY_NONE, None
    if g is not None:
        if g.dim() == 1:
            decay = KDN_DECAY_HEAD
            _expect("g", g, (H,), torch.float32, dev)
        else:
            decay = KDN_DECAY_TOKEN
            _expect("g", g, (B, T, H), torch.float32, dev)
        gp = g.data_ptr()
    return torch, dev, kdn_linear_problem_t(B, T, H, dk, dv, cu, n, code, scale, decay), (n, H, dk, dv), gp


def _state_ptr(torch, name, t, shape, dev):
    if t is None:
        return None
    _expect(name, t, shape, torch.float32, dev)
    return t.data_ptr()


def linear_forward(q, k, v, g=None, cu_seqlens=None, S0=None, scale: float = 1.0, o=None, S_out=None,
                   want_state: bool = True, workspace=None, stream=None):
    """Linear attention with a decay for each head over whole sequences (kdn_linear_forward):
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k [B,T,H,dk] and v [B,T,H,dv] in bf16 or fp32; g the fp32 log decay, [B,T,H], [H] or None (no
    decay); varlen: B = 1 with int32 cu_seqlens; S0 [N,H,dk,dv] fp32.  Returns (o, S_out); outputs
    and workspace are allocated when not given (S_out stays None without ``want_state``)."""
    if stream is None and workspace is None:
        done = (_native_mod or _native()).linear_forward(q, k, v, g, cu_seqlens, S0, scale, o, S_out, want_state)
        if done is not None:
            return done
    torch, dev, p, states, gp = _linear_problem(q, k, v, g, cu_seqlens, scale)
    s0 = _state_ptr(torch, "S0", S0, states, dev)
    if o is not None:
        _expect("o", o, v.shape, q.dtype, dev)
    so = _state_ptr(torch, "S_out", S_out, states, dev)

    def run(handle):
        out = torch.empty_like(v) if o is None else o
        last, lp = S_out, so
        if last is None and want_state:
            last = torch.empty(states, dtype=torch.float32, device=dev)
            lp = last.data_ptr()
        ws, wp, wb = _work(torch, "linear_forward", workspace, _need(kdn_linear_workspace_size, p, cu_seqlens is not None), dev)
        st = _lib.kdn_linear_forward(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), gp, s0, out.data_ptr(), lp, wp,
                                     wb, handle)
        if st != KDN_OK:
            raise KdnError(st, "kdn_linear_forward")
        return out, last

    load()
    return _launch(torch, dev, stream, run)


def linear_decode_tokens(q, k, v, g, S, scale: float = 1.0, o=None, stream=None):
    """n tokens per sequence of the recurrent form in one launch on [N, n, H, d] token tensors
    (kdn_linear_decode_tokens); g [N, n, H], [H] or None; S [N,H,dk,dv] fp32, updated in place."""
    if stream is None:
        done = (_native_mod or _native()).linear_decode(q, k, v, g, S, scale, o, 4)
        if done is not None:
            return done
    torch, dev, p, states, gp = _linear_problem(q, k, v, g, None, scale)
    _expect("S", S, states, torch.float32, dev)
    if o is not None:
        _expect("o", o, v.shape, q.dtype, dev)

    def run(handle):
        out = torch.empty_like(v) if o is None else o
        st = _lib.kdn_linear_decode_tokens(p.B, p.T, p.H, p.d_k, p.d_v, p.in_dtype, p.scale, p.decay, q.data_ptr(), k.data_ptr(),
                                           v.data_ptr(), gp, S.data_ptr(), out.data_ptr(), handle)
        if st != KDN_OK:
            raise KdnError(st, "kdn_linear_decode_tokens")
        return out

    load()
    return _launch(torch, dev, stream, run)


def linear_decode_step(q, k, v, g, S, scale: float = 1.0, o=None, stream=None):
    """One token of the recurrent form on [N, H, d] token tensors; g [N, H], [H] or None.  A one-dimensional
    g is the per-head decay."""
    if stream is None:
        done = (_native_mod or _native()).linear_decode(q, k, v, g, S, scale, o, 3)
        if done is not None:
            return done
    g4 = g if g is None or g.dim() == 1 else g.unsqueeze(1)
    o4 = None if o is None else o.unsqueeze(1)
    return linear_decode_tokens(q.unsqueeze(1), k.unsqueeze(1), v.unsqueeze(1), g4, S, scale=scale, o=o4,
                                stream=stream).squeeze(1)


def linear_backward(q, k, v, g, d_o, cu_seqlens=None, S0=None, dS=None, scale: float = 1.0, want_initial: bool = True,
                    workspace=None, stream=None):
    """Gradients of <o, d_o> + <S_T, dS> for ``linear_forward``'s inputs (kdn_linear_backward).

    Returns a dict: dq, dk, dv (shapes and type of q, k, v), with a decay dg (fp32, shape of g), and with
    ``want_initial`` dS0 [N,H,dk,dv] fp32.  The workspace is allocated when not given."""
    if stream is None and workspace is None:
        done = (_native_mod or _native()).linear_backward(q, k, v, g, d_o, cu_seqlens, S0, dS, scale, want_initial)
        if done is not None:
            return done
    torch, dev, p, states, gp = _linear_problem(q, k, v, g, cu_seqlens, scale)
    _expect("d_o", d_o, v.shape, q.dtype, dev)
    s0, ds = _state_ptr(torch, "S0", S0, states, dev), _state_ptr(torch, "dS", dS, states, dev)

    def run(handle):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        out = {"dq": dq, "dk": dk, "dv": dv}
        dgp = dsp = None
        if g is not None:
            out["dg"] = torch.empty_like(g)
            dgp = out["dg"].data_ptr()
        if want_initial:
            out["dS0"] = torch.empty(states, dtype=torch.float32, device=dev)
            dsp = out["dS0"].data_ptr()
        ws, wp, wb = _work(torch, "linear_backward", workspace,
                           _need(kdn_linear_backward_workspace_size, p, cu_seqlens is not None), dev)
        st = _lib.kdn_linear_backward(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), gp, s0, d_o.data_ptr(), ds,
                                      dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dgp, dsp, wp, wb, handle)
        if st != KDN_OK:
            raise KdnError(st, "kdn_linear_backward")
        return out

    load()
    return _launch(torch, dev, stream, run)


def _norm_rows(x, weight):
    """(rows n, groups G, width d): with a [G, d] weight the rows are [..., G, d], else one group."""
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    d = x.shape[-1]
    G = 1
    if weight is not None and weight.dim() == 2:
        G = weight.shape[0]
        if x.dim() < 2 or x.shape[-2] != G:
            raise ValueError(f"a weight of {G} groups needs x [..., {G}, {d}], got {tuple(x.shape)}")
    return (x.numel() // (G * d) if G * d else 0), G, d


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, y=None, stream=None):
    """Layer norm over the last axis (kdn_layer_norm); returns (y, mean, rstd), mean and rstd fp32 of
    x.shape[:-1].  weight, bias: fp32 [d], or [G, d] for x [..., G, d] (a row for each head), or None.
    (``layer_norm_backward`` returns the bias's gradient beside the weight's: a norm that trains a bias alone has
    a weight of ones.)"""
    if stream is None:
        done = (_native_mod or _native()).layer_norm(x, weight, bias, eps, y)
        if done is not None:
            return done
    torch = _mod or _cuda()
    code = _type_of(torch, "x", x)
    dev = _device_of("x", x)
    _expect("x", x, x.shape, x.dtype, dev)
    param = weight if weight is not None else bias
    n, G, d = _norm_rows(x, param)
    wp = bp = None
    if param is not None:
        shape = (G, d) if param.dim() == 2 else (d,)
        if weight is not None:
            _expect("weight", weight, shape, torch.float32, dev)
            wp = weight.data_ptr()
        if bias is not None:
            _expect("bias", bias, shape, torch.float32, dev)
            bp = bias.data_ptr()
    if y is not None:
        _expect("y", y, x.shape, x.dtype, dev)

    def run(handle):
        out = torch.empty_like(x) if y is None else y
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
        st = _lib.kdn_layer_norm(n, G, d, code, eps, x.data_ptr(), wp, bp, out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), handle)
        if st != KDN_OK:
            raise KdnError(st, "kdn_layer_norm")
        return out, mean, rstd

    load()
    return _launch(torch, dev, stream, run)


def layer_norm_backward(dy, x, weight, mean, rstd, workspace=None, stream=None):
    """Gradients of <y, dy> for ``layer_norm`` (kdn_layer_norm_backward), mean and rstd as it returned
    them: a dict of dx and, with a weight, dweight and dbias (fp32, the weight's shape)."""
    if stream is None and workspace is None:
        done = (_native_mod or _native()).layer_norm_backward(dy, x, weight, mean, rstd)
        if done is not None:
            return done
    torch = _mod or _cuda()
    code = _type_of(torch, "x", x)
    dev = _device_of("x", x)
    shape = x.shape
    _expect("x", x, shape, x.dtype, dev)
    _expect("dy", dy, shape, x.dtype, dev)
    n, G, d = _norm_rows(x, weight)
    wp = None
    if weight is not None:
        _expect("weight", weight, (G, d) if weight.dim() == 2 else (d,), torch.float32, dev)
        wp = weight.data_ptr()
    _expect("mean", mean, shape[:-1], torch.float32, dev)
    _expect("rstd", rstd, shape[:-1], torch.float32, dev)

    def run(handle):
        dx = torch.empty_like(x)
        out = {"dx": dx}
        dwp = dbp = sp = None
        sb = 0
        if weight is not None:
            out["dweight"], out["dbias"] = torch.empty_like(weight), torch.empty_like(weight)
            dwp, dbp = out["dweight"].data_ptr(), out["dbias"].data_ptr()
            key = ("norm", n, G, d)
            need = _sizes.get(key)
            if need is None:
                if len(_sizes) > 4096:
                    _sizes.clear()
                need = _sizes[key] = kdn_layer_norm_backward_workspace_size(n, G, d)
            ws, sp, sb = _work(torch, "layer_norm_backward", workspace, need, dev)
        st = _lib.kdn_layer_norm_backward(n, G, d, code, dy.data_ptr(), x.data_ptr(), wp, mean.data_ptr(), rstd.data_ptr(),
                                          dx.data_ptr(), dwp, dbp, sp, sb, handle)
        if st != KDN_OK:
            raise KdnError(st, "kdn_layer_norm_backward")
        return out

    load()
    return _launch(torch, dev, stream, run)


PATH_NAMES = {0: "recurrent", 1: "chunk_fp32", 3: "chunk_tcgen05_two_phase"}


def execution_path(q, v, cu_seqlens=None, mu: float = 1.0, chunk: int = 64, variant: str = "diagonal",
                   workspace: bool = True) -> str:
    """Name of the kernel path kdn_forward_chunkwise takes for these tensors (``workspace``:
    whether the call gets a workspace of kdn_workspace_size() bytes; the tensor-core path
    needs one, and without it the call runs the fp32 chunk kernel)."""
    p = make_problem(q, v, cu_seqlens=cu_seqlens, mu=mu, chunk=chunk, variant=variant)
    code = kdn_execution_path(p)
    if code == 3 and not workspace:
        code = 1
    return PATH_NAMES.get(code, "invalid")


def selftest_bounded_wait(limit_cycles: int = 2_000_000, stream=None):
    """Launch the failure-detection self-test (bounded waits that run out); the device error
    word then holds KDN_ERR_TIMEOUT, which last_device_error() raises."""
    _check(load().kdn_selftest_bounded_wait(int(limit_cycles), _stream_handle(stream)), "kdn_selftest_bounded_wait")


def last_device_error(stream=None):
    """Synchronise and raise if a kernel recorded a device-side condition."""
    _check(kdn_last_device_error(_stream_handle(stream)), "device")


def available_chunks(dtype=None):
    """The `chunk` values of kdn_forward_chunkwise with a built execution path."""
    return [0, 16, 32, 64]
