"""GPU tests of what the wrappers do when a call of the library fails: one call, an exception, and no second application
of a decode step to its state.  The failures are made on the host; nothing faults."""
import ctypes
import importlib.util
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.gpu


def token(seed=1):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen).cuda()   # noqa: E731
    return rn(2, 3, 64).bfloat16(), rn(2, 3, 64).bfloat16(), rn(2, 3, 32).bfloat16(), -rn(2, 3).abs(), rn(2, 3, 64, 32)


def stubs(kdn, status, calls):
    """Functions of the ABI's types that count their calls; the sizes are the library's own."""
    names = ("linear_workspace_size", "linear_forward", "linear_decode_tokens", "linear_backward_workspace_size",
             "linear_backward", "layer_norm", "layer_norm_backward_workspace_size", "layer_norm_backward")
    made, keep = [], []
    for n in names:
        fn = getattr(kdn.load(), "kdn_" + n)
        if not n.endswith("size"):
            fn = ctypes.CFUNCTYPE(fn.restype, *fn.argtypes)(lambda *a, n=n: calls.append(n) or status)
            keep.append(fn)
        made.append(ctypes.cast(fn, ctypes.c_void_p).value)
    return made, keep


def failing(kdn, monkeypatch, tmp_path, status):
    """The wrappers on an extension module of their own (a copy of the file: its bound functions are its own)."""
    path = str(tmp_path / "_kdn_marshal.so")
    shutil.copy(os.path.join(kdn.PKG, "_kdn_marshal.so"), path)
    spec = importlib.util.spec_from_file_location("_kdn_marshal", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    calls = []
    made, keep = stubs(kdn, status, calls)
    kdn._native()                       # what the wrappers know about the module is set up
    if hasattr(mod, "raise_with"):
        mod.raise_with(kdn.KdnError)
    mod.bind(*made)
    monkeypatch.setattr(kdn, "_native_mod", mod)
    return calls, keep


def test_a_failed_launch_is_reported_and_not_repeated(kdn, monkeypatch, tmp_path):
    q, k, v, g, S = token()
    before = S.clone()
    calls, keep = failing(kdn, monkeypatch, tmp_path, kdn.KDN_ERR_CUDA)
    with pytest.raises(kdn.KdnError) as err:
        kdn.linear_decode_step(q, k, v, g, S)
    assert err.value.code == kdn.KDN_ERR_CUDA and "kdn_linear_decode_tokens" in str(err.value)
    a = [t.unsqueeze(1) for t in (q, k, v, g)]
    with pytest.raises(kdn.KdnError):
        kdn.linear_decode_tokens(*a, S)
    with pytest.raises(kdn.KdnError):
        kdn.linear_forward(*a)
    with pytest.raises(kdn.KdnError):
        kdn.linear_backward(*a, a[2])
    with pytest.raises(kdn.KdnError):
        kdn.layer_norm(v)
    stat = torch.ones(v.shape[:-1], device="cuda")
    with pytest.raises(kdn.KdnError):
        kdn.layer_norm_backward(v, v, None, stat, stat)
    assert calls == ["linear_decode_tokens"] * 2 + ["linear_forward", "linear_backward", "layer_norm", "layer_norm_backward"]
    assert torch.equal(S, before)


def test_an_earlier_failure_is_not_a_launch_s(kdn):
    """A call of the library that failed leaves CUDA's last error behind (here: synchronising a stream that is being captured,
    which only ends the capture).  The decode step after it succeeds, and the state takes its token once."""
    q, k, v, g, S = token(2)
    want_S = S.clone()
    want = kdn.linear_decode_step(q, k, v, g, want_S)
    rt = None
    for line in open("/proc/self/maps"):
        if "libcudart.so" in line:
            rt = ctypes.CDLL(line.split()[-1])
            break
    if rt is None:
        pytest.skip("torch's CUDA runtime is not a shared library here")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = ctypes.c_void_p(side.cuda_stream)
    assert rt.cudaStreamBeginCapture(s, 2) == 0          # relaxed: other streams' calls stay allowed
    st = kdn.kdn_last_device_error(side.cuda_stream)
    graph = ctypes.c_void_p()
    ended = rt.cudaStreamEndCapture(s, ctypes.byref(graph))
    rt.cudaGetLastError()                                # (torch's own copy of the error)
    assert st == kdn.KDN_ERR_CUDA and ended != 0 and not graph.value
    o = kdn.linear_decode_step(q, k, v, g, S)
    assert torch.equal(o, want) and torch.equal(S, want_S)
    kdn.last_device_error()
