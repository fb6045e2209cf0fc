"""The linear-attention and layer-norm entry points on the CPU: bad arguments are refused before any
CUDA call (the fake addresses are never dereferenced), sizes are host-only."""
import ctypes

import pytest

from kalman_delta_rule_b200 import binding as B

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    from kalman_delta_rule_b200 import build
    build.build()
    return B.load()


def problem(**kw):
    p = B.kdn_linear_problem_t()
    p.B, p.T, p.H, p.d_k, p.d_v, p.in_dtype, p.scale, p.decay = 2, 128, 4, 128, 128, B.KDN_DTYPE_BF16, 1.0, B.KDN_DECAY_TOKEN
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD = [(dict(d_k=48), B.KDN_ERR_UNSUPPORTED), (dict(d_v=96), B.KDN_ERR_UNSUPPORTED), (dict(d_k=256), B.KDN_ERR_UNSUPPORTED),
       (dict(H=0), B.KDN_ERR_INVALID_ARG), (dict(B=-1), B.KDN_ERR_INVALID_ARG), (dict(T=-5), B.KDN_ERR_INVALID_ARG),
       (dict(in_dtype=2), B.KDN_ERR_INVALID_ARG), (dict(decay=3), B.KDN_ERR_INVALID_ARG), (dict(decay=-1), B.KDN_ERR_INVALID_ARG),
       (dict(scale=float("nan")), B.KDN_ERR_INVALID_ARG), (dict(scale=float("inf")), B.KDN_ERR_INVALID_ARG),
       (dict(cu_seqlens=FAKE, B=2, num_seqs=3), B.KDN_ERR_INVALID_ARG), (dict(cu_seqlens=FAKE, B=1, num_seqs=-1), B.KDN_ERR_INVALID_ARG),
       (dict(B=1 << 15, T=1 << 16), B.KDN_ERR_UNSUPPORTED), (dict(B=1 << 20, T=1, H=1 << 12), B.KDN_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD)
def test_problem_validation(lib, kw, code):
    p, n = problem(**kw), ctypes.c_size_t(0)
    assert lib.kdn_linear_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.kdn_linear_backward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert B.kdn_linear_forward(p, *[FAKE] * 4, None, FAKE, None, FAKE, 1 << 40, None) == code
    assert B.kdn_linear_backward(p, *[FAKE] * 4, None, FAKE, None, *[FAKE + 4096] * 3, FAKE, None, FAKE, 1 << 40, None) == code


def test_null_problem(lib):
    n = ctypes.c_size_t(0)
    assert lib.kdn_linear_workspace_size(None, ctypes.byref(n)) == B.KDN_ERR_INVALID_ARG
    assert lib.kdn_linear_workspace_size(ctypes.byref(problem()), None) == B.KDN_ERR_INVALID_ARG
    assert lib.kdn_linear_backward_workspace_size(None, ctypes.byref(n)) == B.KDN_ERR_INVALID_ARG


def test_forward_pointers_and_workspace(lib):
    p = problem()
    need = B.kdn_linear_workspace_size(p)
    call = lambda q=FAKE, k=FAKE, v=FAKE, g=FAKE, S0=None, o=FAKE, S=None, ws=FAKE, wb=need, p=p: \
        B.kdn_linear_forward(p, q, k, v, g, S0, o, S, ws, wb, None)      # noqa: E731
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(o=None), dict(q=FAKE + 2), dict(g=FAKE + 4),
                dict(o=FAKE + 8), dict(S0=FAKE + 4), dict(S=FAKE + 8), dict(S0=FAKE, S=FAKE)):
        assert call(**bad) == B.KDN_ERR_INVALID_ARG, bad
    if need:
        for bad in (dict(ws=None), dict(wb=need - 1), dict(ws=FAKE + 16)):
            assert call(**bad) == B.KDN_ERR_WORKSPACE, bad
    # nothing to do: no pointer is looked at
    assert call(p=problem(B=0), q=None, ws=None) == B.KDN_OK
    assert call(p=problem(T=0), q=None, ws=None) == B.KDN_OK
    assert call(p=problem(cu_seqlens=FAKE, B=1, num_seqs=0), ws=None) == B.KDN_OK


def test_backward_pointers_and_workspace(lib):
    p = problem()
    need = B.kdn_linear_backward_workspace_size(p)
    assert need > 0
    names = ["q", "k", "v", "g", "S0", "d_o", "dS_T", "dq", "dk", "dv", "dg", "dS0"]
    good = dict(zip(names, [FAKE, FAKE, FAKE, FAKE, None, FAKE, None, FAKE + 256, FAKE + 512, FAKE + 768, None, None]))

    def call(p=p, ws=FAKE, wb=need, **kw):
        a = {**good, **kw}
        return B.kdn_linear_backward(p, *[a[n] for n in names], ws, wb, None)
    for n in ("q", "k", "v", "g", "d_o", "dq", "dk", "dv"):
        assert call(**{n: None}) == B.KDN_ERR_INVALID_ARG, n
    for n in names:
        assert call(**{n: FAKE + 4}) == B.KDN_ERR_INVALID_ARG, n
    assert call(dS_T=FAKE, dS0=FAKE) == B.KDN_ERR_INVALID_ARG
    assert call(p=problem(decay=B.KDN_DECAY_NONE), g=None, dg=FAKE) == B.KDN_ERR_INVALID_ARG
    for bad in (dict(ws=None), dict(wb=need - 1), dict(ws=FAKE + 16)):
        assert call(**bad) == B.KDN_ERR_WORKSPACE, bad
    assert call(p=problem(T=0), q=None, ws=None) == B.KDN_OK


def test_decode_arguments(lib):
    ok = dict(N=2, n=1, H=2, dk=64, dv=64, dt=B.KDN_DTYPE_BF16, scale=1.0, decay=B.KDN_DECAY_TOKEN)

    def call(ptrs=(FAKE,) * 6, **kw):
        a = {**ok, **kw}
        return B.kdn_linear_decode_tokens(a["N"], a["n"], a["H"], a["dk"], a["dv"], a["dt"], a["scale"], a["decay"], *ptrs, None)
    assert call(dk=48) == B.KDN_ERR_UNSUPPORTED and call(dv=512) == B.KDN_ERR_UNSUPPORTED
    for bad in (dict(N=-1), dict(n=-1), dict(H=0), dict(dt=5), dict(scale=float("nan")), dict(decay=9)):
        assert call(**bad) == B.KDN_ERR_INVALID_ARG, bad
    assert call(N=1 << 20, n=1 << 12) == B.KDN_ERR_UNSUPPORTED
    assert call(N=0, ptrs=(None,) * 6) == B.KDN_OK and call(n=0, ptrs=(None,) * 6) == B.KDN_OK
    for i in range(6):
        for bad in (None, FAKE + 4):
            p = [FAKE] * 6
            p[i] = bad
            assert call(ptrs=p) == B.KDN_ERR_INVALID_ARG, (i, bad)


def test_norm_arguments(lib):
    f = lambda n=4, G=2, d=64, dt=1, eps=1e-5, x=FAKE, w=None, b=None, y=FAKE, m=None, r=None: \
        B.kdn_layer_norm(n, G, d, dt, eps, x, w, b, y, m, r, None)       # noqa: E731
    for bad in (dict(n=-1), dict(G=0), dict(d=0), dict(dt=3), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")),
                dict(x=None), dict(y=None), dict(x=FAKE + 2), dict(w=FAKE + 4), dict(m=FAKE + 8)):
        assert f(**bad) == B.KDN_ERR_INVALID_ARG, bad
    for bad in (dict(d=16385), dict(G=65536), dict(n=1 << 50)):
        assert f(**bad) == B.KDN_ERR_UNSUPPORTED, bad
    assert f(n=0, x=None, y=None) == B.KDN_OK
    need = B.kdn_layer_norm_backward_workspace_size(4, 2, 64)
    assert 0 < need < 1 << 24
    assert B.kdn_layer_norm_backward_workspace_size(4, 60000, 16) >= 60000 * 2 * 16 * 4
    g = lambda dy=FAKE, x=FAKE, w=None, m=FAKE, r=FAKE, dx=FAKE, dw=FAKE, db=None, ws=FAKE, wb=need, **kw: \
        B.kdn_layer_norm_backward(kw.get("n", 4), 2, kw.get("d", 64), 1, dy, x, w, m, r, dx, dw, db, ws, wb, None)   # noqa: E731
    for bad in (dict(dy=None), dict(x=None), dict(m=None), dict(r=None), dict(dx=None), dict(dx=FAKE + 4), dict(db=FAKE + 2), dict(d=-1)):
        assert g(**bad) == B.KDN_ERR_INVALID_ARG, bad
    for bad in (dict(ws=None), dict(wb=need - 1), dict(ws=FAKE + 16)):
        assert g(**bad) == B.KDN_ERR_WORKSPACE, bad
    assert g(d=20000) == B.KDN_ERR_UNSUPPORTED
    assert g(n=0, dy=None, x=None, dw=None, ws=None) == B.KDN_OK


def test_aliased_outputs(lib):
    """An output that is an input, or another output, is refused before anything is launched."""
    at = lambda i: FAKE + (i << 20)                                      # noqa: E731
    p = problem()
    need = max(B.kdn_linear_workspace_size(p), B.kdn_linear_backward_workspace_size(p))
    ws = (at(40), need, None)
    for i in range(5):             # q, k, v, g, S0
        for j in (5, 6):           # o, S_out
            a = [at(n) for n in range(7)]
            a[j] = a[i]
            assert B.kdn_linear_forward(p, *a, *ws) == B.KDN_ERR_INVALID_ARG, (i, j)
    for i in range(12):            # q, k, v, g, S0, d_o, dS_T, then the outputs
        for j in range(7, 12):
            if i != j:
                a = [at(n) for n in range(12)]
                a[j] = a[i]
                assert B.kdn_linear_backward(p, *a, *ws) == B.KDN_ERR_INVALID_ARG, (i, j)
    assert B.kdn_linear_backward(problem(T=0), *[None] * 6, at(1), *[None] * 4, at(1), *ws) == B.KDN_ERR_INVALID_ARG
    for i in range(4):             # q, k, v, g, S, o
        for j in (4, 5):
            a = [at(n) for n in range(6)]
            a[j] = a[i]
            assert B.kdn_linear_decode_tokens(2, 1, 2, 64, 64, 1, 1.0, 1, *a, None) == B.KDN_ERR_INVALID_ARG, (i, j)
    for i in range(3):             # x, weight, bias, y, mean, rstd
        for j in range(3, 6):
            a = [at(n) for n in range(6)]
            a[j] = a[i]
            assert B.kdn_layer_norm(4, 2, 64, 1, 1e-5, *a, None) == B.KDN_ERR_INVALID_ARG, (i, j)
    for i in range(5):             # dy, x, weight, mean, rstd, dx, dweight, dbias
        for j in range(5, 8):
            a = [at(n) for n in range(8)]
            a[j] = a[i]
            assert B.kdn_layer_norm_backward(4, 2, 64, 1, *a, *ws) == B.KDN_ERR_INVALID_ARG, (i, j)


def test_native_step_leaves_other_calls_alone(lib):
    """The wrappers' extension module: built, and None for what is not its call (here: tensors off the GPU, None, numbers)."""
    import importlib.util
    import os

    import torch
    spec = importlib.util.spec_from_file_location("_kdn_marshal", os.path.join(B.PKG, "_kdn_marshal.so"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    x, w = torch.zeros((1, 2, 2, 32)), torch.zeros(32)
    g, S = torch.zeros((1, 2, 2)), torch.zeros((1, 2, 32, 32))
    assert m.linear_forward(x, x, x, g, None, None, 1.0, None, None, True) is None
    assert m.linear_decode(x, x, x, g, S, 1.0, None, 4) is None and m.linear_decode(x, x, x, g, S, 1.0, None, 3) is None
    assert m.linear_backward(x, x, x, g, x, None, None, None, 1.0, True) is None
    assert m.layer_norm(x, w, w, 1e-5, None) is None and m.layer_norm_backward(x, x, w, g, g) is None
    for f in (m.linear_forward, m.linear_decode, m.linear_backward, m.layer_norm, m.layer_norm_backward):
        assert f() is None and f(1) is None and f(*[None] * 10) is None and f(*[None] * 5) is None and f(*[None] * 8) is None
    with pytest.raises(TypeError):
        m.bind(1, 2)
    with pytest.raises(TypeError):
        m.bind(*["x"] * 8)
