"""GPU tests of linear attention with a decay for each head: forward, recurrent form and gradients
against the plain fp64 forms of tests/linear_ref.py, with its elementwise error bounds."""
import itertools

import pytest
import torch

from tests import linear_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, B, T, H, dk, dv, dtype, decay="token", N=None, state=True, grads=False):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)   # noqa: E731
    x = {"q": rn(B, T, H, dk) / dk ** 0.5, "k": rn(B, T, H, dk) / dk ** 0.5, "v": rn(B, T, H, dv)}
    x = {n: t.to(DT[dtype]) for n, t in x.items()}
    x["g"] = {"token": lambda: -torch.nn.functional.softplus(-3.0 + rn(B, T, H)),
              "strong": lambda: -8.0 * torch.rand((B, T, H), generator=gen),
              "reset": lambda: torch.where(torch.rand((B, T, H), generator=gen) < 0.05, -float("inf"), -0.02 * torch.rand((B, T, H), generator=gen)),
              "head": lambda: -0.2 * torch.rand((H,), generator=gen),
              "none": lambda: None}[decay]()
    N = B if N is None else N
    x["S0"] = 0.3 * rn(N, H, dk, dv) if state else None
    if grads:
        x["do"] = rn(B, T, H, dv).to(DT[dtype])
        x["dS"] = 0.3 * rn(N, H, dk, dv) if state else None
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def offsets(lens):
    return torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32).cuda()


def check_forward(x, o, S, dtype, cu=None, scale=1.0, mask=None, state=True):
    r = R.forward(x["q"], x["k"], x["v"], x["g"], cu=cu, S0=x["S0"], scale=scale)
    T, dk, dv = x["q"].shape[1], x["q"].shape[-1], x["v"].shape[-1]
    n = R.terms(T, dk, dv) * R.U32
    bound = n * r["mag_o"]
    if dtype == "bf16":
        bound = bound * (1 + R.U16) + R.U16 * (r["o"].abs() + (1 + R.U16) * r["round_o"])
    rows = slice(None) if mask is None else mask
    R.assert_within(o.float().cpu()[:, rows], r["o"][:, rows], bound[:, rows], "o")
    if state:
        R.assert_within(S, r["S"], n * r["mag_S"], "S")


def check_backward(x, out, dtype, cu=None, scale=1.0):
    r = R.backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu=cu, S0=x["S0"], dS=x["dS"], scale=scale)
    T, dk, dv = x["q"].shape[1], x["q"].shape[-1], x["v"].shape[-1]
    n = R.terms(T, dk, dv) * R.U32
    for name in ("dq", "dk", "dv"):
        assert out[name].dtype == x["q"].dtype
        bound = n * r["mag_" + name]
        if dtype == "bf16":
            bound = bound * (1 + R.U16) + R.U16 * (r[name].abs() + (1 + R.U16) * r["round_" + name])
        R.assert_within(out[name].float(), r[name], bound, name)
    R.assert_within(out["dS0"], r["dS0"], n * r["mag_dS0"], "dS0")
    if x["g"] is None:
        assert "dg" not in out
    elif x["g"].dim() == 1:
        R.assert_within(out["dg"], r["dg"].sum((0, 1)), 2 * n * r["mag_dg"].sum((0, 1)), "dg")
    else:
        R.assert_within(out["dg"], r["dg"], 2 * n * r["mag_dg"], "dg")   # two chains of sums meet in it


SIZES = [(32, 32), (64, 64), (128, 128), (128, 32), (32, 256), (64, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("T", [1, 64, 129, 300])
def test_forward_dense(kdn, dtype, dk, dv, T):
    x = make(T + dk + dv, 2, T, 3, dk, dv, dtype)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], scale=0.7)
    kdn.last_device_error()
    check_forward(x, o, S, dtype, scale=0.7)


LENS = [0, 1, 64, 65, 0, 128, 130, 257, 2, 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 32), (128, 128), (128, 256)])
@pytest.mark.parametrize("decay", ["token", "strong", "reset", "head", "none"])
def test_forward_packed(kdn, dtype, dk, dv, decay):
    x = make(7, 1, sum(LENS), 2, dk, dv, dtype, decay, N=len(LENS))
    cu = offsets(LENS)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"])
    kdn.last_device_error()
    check_forward(x, o, S, dtype, cu=cu)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_defaults_and_no_state(kdn, dtype):
    x = make(11, 3, 70, 1, 64, 64, dtype, "token", state=False)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"])
    check_forward(x, o, S, dtype)
    o2, none = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], want_state=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_many_short_and_one_long(kdn, dtype):
    """Few chains with a long serial axis, and more sequences than the chip has SMs."""
    x = make(13, 1, 5001, 1, 128, 64, dtype, "head")
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    check_forward(x, o, S, dtype)
    x = make(17, 200, 3, 2, 32, 64, dtype)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    check_forward(x, o, S, dtype)
    kdn.last_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_other_sequences_and_rows_behind_the_last(kdn, dtype):
    """NaN and infinity in one sequence stay there; rows behind the last sequence keep what they held."""
    lens = [130, 40, 100]
    T = sum(lens) + 30
    x = make(19, 1, T, 2, 128, 64, dtype, N=3, grads=True)
    for n in ("q", "k", "v", "do"):
        x[n][0, 130:170] = float("nan")
        x[n][0, 150] = float("inf")
        x[n][0, 270:] = float("nan")
    cu = offsets(lens)
    o = torch.full_like(x["v"], 7.0)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"], o=o)
    assert (o[0, 270:] == 7.0).all()
    assert S[1].isnan().any() and not S[0].isnan().any() and not S[2].isnan().any()
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    kdn.last_device_error()
    keep = [i for i in range(270) if not 130 <= i < 170]
    clean = {n: (None if t is None else t.clone()) for n, t in x.items()}
    for n in ("q", "k", "v", "do"):
        clean[n][0, 130:170] = 0.0
        clean[n][0, 270:] = 0.0
    want, wantS = kdn.linear_forward(clean["q"], clean["k"], clean["v"], clean["g"], cu_seqlens=cu, S0=x["S0"])
    assert torch.equal(o[0, keep], want[0, keep]) and torch.equal(S[0], wantS[0]) and torch.equal(S[2], wantS[2])
    ref = kdn.linear_backward(clean["q"], clean["k"], clean["v"], clean["g"], clean["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    for n in ("dq", "dk", "dv", "dg"):
        assert torch.equal(out[n][0, keep], ref[n][0, keep]), n
    assert torch.equal(out["dS0"][0], ref["dS0"][0]) and torch.equal(out["dS0"][2], ref["dS0"][2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 128), (128, 256)])
@pytest.mark.parametrize("N,n", [(1, 1), (3, 5), (90, 2), (400, 1)])
def test_decode_tokens(kdn, dtype, dk, dv, N, n):
    """Every tile width; the state in place."""
    for decay in ("token", "head", "none", "reset"):
        x = make(N + n + dk, N, n, 3, dk, dv, dtype, decay)
        S = x["S0"].clone()
        o = kdn.linear_decode_tokens(x["q"], x["k"], x["v"], x["g"], S, scale=0.5)
        check_forward(x, o, S, dtype, scale=0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_steps_equal_tokens_and_continue_a_prompt(kdn, dtype):
    x = make(23, 2, 140, 2, 128, 128, dtype)
    _, S = kdn.linear_forward(x["q"][:, :136].contiguous(), x["k"][:, :136].contiguous(), x["v"][:, :136].contiguous(),
                              x["g"][:, :136].contiguous(), S0=x["S0"])
    T1, T2 = S.clone(), S.clone()
    tail = [x[n][:, 136:].contiguous() for n in ("q", "k", "v", "g")]
    o1 = kdn.linear_decode_tokens(*tail, T1)
    o2 = torch.stack([kdn.linear_decode_step(*(t[:, i].contiguous() for t in tail), T2) for i in range(4)], 1)
    assert torch.equal(o1, o2) and torch.equal(T1, T2)
    r = R.forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    n = R.terms(140, 128, 128) * R.U32
    R.assert_within(T1, r["S"], n * r["mag_S"], "S")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("T", [1, 65, 128, 300])
def test_backward_dense(kdn, dtype, dk, dv, T):
    x = make(T + dk - dv, 2, T, 2, dk, dv, dtype, grads=True)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS=x["dS"], scale=0.7)
    kdn.last_device_error()
    check_backward(x, out, dtype, scale=0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 32), (128, 128), (128, 256)])
@pytest.mark.parametrize("decay", ["token", "strong", "reset", "head", "none"])
def test_backward_packed(kdn, dtype, dk, dv, decay):
    x = make(29, 1, sum(LENS), 2, dk, dv, dtype, decay, N=len(LENS), grads=True)
    cu = offsets(LENS)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    kdn.last_device_error()
    check_backward(x, out, dtype, cu=cu)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_defaults(kdn, dtype):
    x = make(31, 2, 200, 1, 64, 64, dtype, "token", state=False, grads=True)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"])
    check_backward(x, out, dtype)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], want_initial=False)
    assert "dS0" not in out


def test_gradients_against_differences(kdn):
    """Directional derivatives of the plain form's <o, d_o> + <S, dS>, central differences in fp64: the
    scalar is linear in q, k, v and S0 (exact up to 2^-53 / h), and for g the cubic term of the difference is
    h^2 / 6 of the third derivative, below 1e-6 of the sum of magnitudes at h = 1e-4 and 40 tokens."""
    x = make(37, 2, 40, 2, 32, 64, "f32", grads=True)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS=x["dS"])
    gen = torch.Generator().manual_seed(1)
    args = {n: R.f64(x[n]) for n in ("q", "k", "v", "g", "S0")}

    def scalar(a):
        r = R.forward(a["q"], a["k"], a["v"], a["g"], S0=a["S0"])
        return float((r["o"] * R.f64(x["do"])).sum() + (r["S"] * R.f64(x["dS"])).sum())

    mag = R.backward(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS=x["dS"])
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("S0", "dS0")):
        way = torch.randn(args[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        up, dn = dict(args), dict(args)
        up[n], dn[n] = args[n] + h * way, args[n] - h * way
        diff = (scalar(up) - scalar(dn)) / (2 * h)
        got = float((R.f64(out[d]) * way).sum())
        total = float((mag["mag_" + d] * way.abs()).sum())
        assert abs(got - diff) <= (2 * R.terms(40, 32, 64) * R.U32 + 1e-6) * total, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeatable_streams_and_graphs(kdn, dtype):
    """The same bits again; on another stream; captured, replayed on new inputs, and captured twice with
    one workspace replayed in turn."""
    x = make(41, 2, 333, 4, 128, 128, dtype, grads=True)
    y = make(43, 2, 333, 4, 128, 128, dtype, grads=True)
    fwd = lambda z, **kw: kdn.linear_forward(z["q"], z["k"], z["v"], z["g"], S0=z["S0"], **kw)              # noqa: E731
    bwd = lambda z, **kw: kdn.linear_backward(z["q"], z["k"], z["v"], z["g"], z["do"], S0=z["S0"], dS=z["dS"], **kw)   # noqa: E731
    o, S = fwd(x)
    grads = bwd(x)
    oy, _ = fwd(y)
    gy = bwd(y)
    for _ in range(3):
        o2, S2 = fwd(x)
        g2 = bwd(x)
        assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(grads[n], g2[n]) for n in grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, S3 = fwd(x, stream=side)
    g3 = bwd(x, stream=side)
    side.synchronize()
    assert torch.equal(o, o3) and torch.equal(S, S3) and all(torch.equal(grads[n], g3[n]) for n in grads)

    z = {n: t.clone() for n, t in x.items()}
    q, v = x["q"], x["v"]
    p = kdn.kdn_linear_problem_t()
    p.B, p.T, p.H, p.d_k, p.d_v, p.scale, p.decay = *q.shape, v.shape[-1], 1.0, 1
    p.in_dtype = 1 if dtype == "bf16" else 0
    ws = torch.empty(max(kdn.kdn_linear_workspace_size(p), kdn.kdn_linear_backward_workspace_size(p)), dtype=torch.uint8,
                     device="cuda")
    gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gf):
        og, Sg = fwd(z, workspace=ws)
    with torch.cuda.graph(gb):
        gg = bwd(z, workspace=ws)
    for src, wo, wg in ((x, o, grads), (y, oy, gy), (x, o, grads)):
        for n in z:
            z[n].copy_(src[n])
        gf.replay()
        gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, wo) and all(torch.equal(gg[n], wg[n]) for n in gg)
    kdn.last_device_error()


def test_two_calls_at_once(kdn):
    """Two streams, each with a workspace of its own."""
    xs = [make(50 + i, 2, 700, 2, 128, 128, "bf16", grads=True) for i in range(2)]
    fwd = lambda z, **kw: kdn.linear_forward(z["q"], z["k"], z["v"], z["g"], S0=z["S0"], **kw)   # noqa: E731
    want = [fwd(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(fwd(xs[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(S, want[i][1]) for o, S in got[i])


def test_empty_problems(kdn):
    x = make(53, 2, 0, 2, 64, 64, "bf16")
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    assert o.numel() == 0 and torch.equal(S, x["S0"])
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"])
    assert (S == 0).all()
    x = make(53, 1, 5, 2, 64, 64, "f32", "head", N=0, state=False, grads=True)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu)
    assert S.shape[0] == 0
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu)
    assert (out["dg"] == 0).all()
    x = make(53, 2, 0, 2, 64, 64, "f32", "head", grads=True)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS=x["dS"])
    assert torch.equal(out["dS0"], x["dS"]) and (out["dg"] == 0).all()


def test_malformed_offsets_stay_inside(kdn):
    """Offsets that overrun the tokens, run backwards or start below zero are cut to the token tensors:
    no row outside them is touched, and the call returns."""
    x = make(59, 1, 100, 2, 64, 64, "f32", N=3, grads=True)
    for bad in ([0, 500, 90, 130], [-7, 50, 20, 100], [0, 0, 2 ** 30, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"])
        kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    torch.cuda.synchronize()


def test_refusals(kdn):
    x = make(61, 2, 10, 2, 64, 64, "bf16", grads=True)
    a = (x["q"], x["k"], x["v"], x["g"])
    with pytest.raises(kdn.KdnError):
        kdn.linear_forward(*(t[..., :48].contiguous() for t in a[:2]), a[2], a[3])
    with pytest.raises(ValueError, match="contiguous"):
        kdn.linear_forward(a[0].transpose(1, 2), a[1].transpose(1, 2), a[2].transpose(1, 2), a[3].transpose(1, 2))
    with pytest.raises(TypeError):
        kdn.linear_forward(a[0], a[1].float(), a[2], a[3])
    with pytest.raises(TypeError):
        kdn.linear_forward(a[0].half(), a[1].half(), a[2].half(), a[3])
    with pytest.raises(TypeError):
        kdn.linear_forward(a[0], a[1], a[2], a[3].double())
    with pytest.raises(ValueError):
        kdn.linear_forward(a[0], a[1], a[2], a[3][:, :5].contiguous())
    with pytest.raises(ValueError):
        kdn.linear_forward(*a, S0=x["S0"][:1])
    with pytest.raises(ValueError, match="B = 1"):
        kdn.linear_forward(*a, cu_seqlens=offsets([5, 5]))
    with pytest.raises(ValueError):
        kdn.linear_forward(a[0], a[1], a[2].cpu(), a[3])
    with pytest.raises(kdn.KdnError):
        kdn.linear_forward(*a, scale=float("inf"))
    with pytest.raises(kdn.KdnError):
        kdn.linear_forward(*a, S0=x["S0"], S_out=x["S0"])
    with pytest.raises(kdn.KdnError):
        y = make(61, 2, 200, 2, 64, 64, "bf16")     # (a few tokens need no workspace)
        kdn.linear_forward(y["q"], y["k"], y["v"], y["g"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kdn.linear_backward(*a, x["do"][:, :4].contiguous())
    with pytest.raises(TypeError):
        kdn.linear_backward(*a, x["do"].float())
    with pytest.raises(ValueError):
        kdn.linear_decode_tokens(*a, x["S0"][..., :32].contiguous())


# Few sequences and heads: bf16 sequences of 2048 tokens and more are cut into segments that are walked at once, from
# totals of the earlier ones; fp32 ones are scanned, but for those of a few chunks (packed: on average).
LONG = [(1, 2304, 1, 128, 128, None), (2, 4100, 1, 64, 64, None), (1, 3400, 2, 32, 256, [1, 3000, 0, 399]),
        (1, 2600, 1, 128, 256, [2600]), (1, 2500, 3, 128, 64, [0, 2499, 1]), (1, 2410, 1, 64, 64, [1000, 1010, 400]),
        (1, 1500, 2, 64, 128, [0, 700, 3, 64, 65, 128, 129, 200, 1, 210])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv,lens", LONG)
@pytest.mark.parametrize("decay", ["token", "reset", "head", "none"])
def test_long_sequences(kdn, dtype, B, T, H, dk, dv, lens, decay):
    cu = offsets(lens) if lens else None
    x = make(T + dv, B, T, H, dk, dv, dtype, decay, N=len(lens) if lens else B, grads=True)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"], scale=0.5)
    check_forward(x, o, S, dtype, cu=cu, scale=0.5)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"], scale=0.5)
    check_backward(x, out, dtype, cu=cu, scale=0.5)
    kdn.last_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("B,T,lens", [(3, 1, None), (5, 16, None), (2, 17, None), (2, 24, None), (2, 32, None), (2, 33, None), (1, 32, [0, 30, 0, 2]), (1, 16, [0, 5, 0, 10, 1, 0]),
                                      (1, 16, [3, 4, 2]), (1, 24, [7, 0, 16]), (2, 64, None), (2, 65, None)])
@pytest.mark.parametrize("decay", ["token", "reset", "head", "none"])
def test_short_sequences(kdn, dtype, dk, dv, B, T, lens, decay):
    """Around the lengths at which the path changes; packed ones with empty sequences and rows behind the last."""
    cu = offsets(lens) if lens else None
    end = sum(lens) if lens else T
    x = make(T + dk, B, T, 3, dk, dv, dtype, decay, N=len(lens) if lens else B, grads=True)
    if end < T:
        for m in ("q", "k", "v", "do"):
            x[m][:, end:] = float("nan")
    o = torch.full_like(x["v"], 7.0)
    _, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"], scale=0.8, o=o)
    check_forward(x, o, S, dtype, cu=cu, scale=0.8, mask=slice(0, end))
    assert (o[:, end:] == 7.0).all()
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"], scale=0.8)
    cut = {m: t[:, :end].contiguous() if m in ("q", "k", "v", "do") or m == "g" and t is not None and t.dim() == 3 else t for m, t in x.items()}
    out = {m: t[:, :end].contiguous() if m in ("dq", "dk", "dv") or m == "dg" and t.dim() == 3 else t for m, t in out.items()}
    check_backward(cut, out, dtype, cu=cu, scale=0.8)
    plain, none = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, want_state=False)
    assert none is None
    check_forward({**x, "S0": None}, plain, torch.zeros(0), dtype, cu=cu, mask=slice(0, end), state=False)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, want_initial=False)
    assert "dS0" not in out
    kdn.last_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 16, 40])
def test_bad_values_in_short_sequences(kdn, dtype, T):
    """A NaN log decay, and infinities and NaN in one sequence: the others' results keep their bits."""
    x = make(79 + T, 3, T, 2, 64, 64, dtype, grads=True)
    run = lambda: (kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"]),                        # noqa: E731
                   kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS=x["dS"]))
    (o, S), g = run()
    x["g"][1, T // 2] = float("nan")
    x["v"][1, 0] = float("inf")
    x["do"][1, T - 1] = float("nan")
    (o2, S2), g2 = run()
    for i in (0, 2):
        assert torch.equal(o[i], o2[i]) and torch.equal(S[i], S2[i])
        assert all(torch.equal(g[n][i], g2[n][i]) for n in g)
    assert o2[1, T // 2:].isnan().all() and S2[1].isnan().all()


@pytest.mark.parametrize("scale", [-0.7, 0.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_other_scales(kdn, dtype, scale):
    x = make(67, 1, 200, 2, 64, 64, dtype, grads=True)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], scale=scale)
    check_forward(x, o, S, dtype, scale=scale)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS=x["dS"], scale=scale)
    check_backward(x, out, dtype, scale=scale)


def test_malformed_offsets_stay_inside_bf16(kdn):
    """As above on the tensor cores; one long enough to be cut into segments."""
    for T, bads in ((300, ([0, 500, 90, 330], [-7, 250, 20, 300], [0, 0, 2 ** 30, 300])), (2400, ([0, 2400, 90, 5000], [-7, 2300, 20, 2400]))):
        x = make(59, 1, T, 1, 64, 128, "bf16", N=3, grads=True)
        for bad in bads:
            cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
            kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"])
            kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    torch.cuda.synchronize()
    kdn.last_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_past_32_bits(kdn, dtype):
    """The last of two packed sequences lies behind 2^31 elements of q; its results are those it has alone."""
    H, d, n = 64, 32, 300
    T = (1 << 31) // (H * d) + n + 77
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    x = make(71, 1, n, H, d, d, dtype, N=1, grads=True)
    big = {m: torch.zeros((1, T) + x[m].shape[2:], dtype=x[m].dtype, device="cuda") for m in ("q", "k", "v", "g", "do")}
    for m in big:
        big[m][:, T - n:] = x[m]
    cu = offsets([T - n, n])
    S0, dS = (torch.cat([torch.zeros_like(x[m]), x[m]]) for m in ("S0", "dS"))
    o, S = kdn.linear_forward(big["q"], big["k"], big["v"], big["g"], cu_seqlens=cu, S0=S0)
    check_forward(x, o[:, T - n:].contiguous(), S[1:], dtype)
    assert not o[:, :T - n].any()
    del o
    out = kdn.linear_backward(big["q"], big["k"], big["v"], big["g"], big["do"], cu_seqlens=cu, S0=S0, dS=dS)
    tail = {m: out[m][:, T - n:].contiguous() for m in ("dq", "dk", "dv", "dg")}
    check_backward(x, {**tail, "dS0": out["dS0"][1:]}, dtype)
    kdn.last_device_error()
    del big, out, tail
    torch.cuda.empty_cache()


def test_decode_states_past_32_bits(kdn):
    """More than 2^31 elements of state."""
    N, H, d = 2100, 64, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    x = make(73, 2, 1, H, d, d, "bf16")
    q, k, v, g, S = (torch.zeros((N,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in (x["q"], x["k"], x["v"], x["g"], x["S0"]))
    for big, t in ((q, x["q"]), (k, x["k"]), (v, x["v"]), (g, x["g"]), (S, x["S0"])):
        big[0], big[-1] = t[0], t[1]
    o = kdn.linear_decode_tokens(q, k, v, g, S)
    check_forward(x, torch.stack([o[0], o[-1]]), torch.stack([S[0], S[-1]]), "bf16")
    assert not S[1:-1].any() and not o[1:-1].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_both_ways_to_the_abi(kdn, dtype):
    """The wrappers' native step takes the common call and leaves any other to Python (here: a stream, a workspace of
    the caller's, an integer factor): the same bits, the same shapes, and the caller's outputs are the ones written."""
    x = make(83, 2, 70, 2, 64, 32, dtype, grads=True)
    a, st = (x["q"], x["k"], x["v"], x["g"]), torch.cuda.current_stream()
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    o, S = kdn.linear_forward(*a, S0=x["S0"])
    mine = torch.empty_like(o), torch.empty_like(S)
    for kw in (dict(stream=st), dict(workspace=ws), dict(scale=1), dict(o=mine[0], S_out=mine[1])):
        o2, S2 = kdn.linear_forward(*a, S0=x["S0"], **kw)
        assert torch.equal(o, o2) and torch.equal(S, S2)
    assert o2 is mine[0] and S2 is mine[1]
    assert kdn.linear_forward(*a, want_state=False)[1] is None and kdn.linear_forward(*a, want_state=0, stream=st)[1] is None
    g = kdn.linear_backward(*a, x["do"], S0=x["S0"], dS=x["dS"])
    for kw in (dict(stream=st), dict(workspace=ws), dict(scale=1)):
        g2 = kdn.linear_backward(*a, x["do"], S0=x["S0"], dS=x["dS"], **kw)
        assert g.keys() == g2.keys() and all(torch.equal(g[n], g2[n]) and g[n].dtype == g2[n].dtype for n in g)
    assert "dg" not in kdn.linear_backward(*a[:3], None, x["do"], want_initial=False)
    T1 = [t[:, 0].contiguous() for t in a]
    S1, S2, S3 = x["S0"].clone(), x["S0"].clone(), x["S0"].clone()
    o1, o2 = kdn.linear_decode_step(*T1, S1), kdn.linear_decode_step(*T1, S2, stream=st)
    o3 = kdn.linear_decode_tokens(*(t.unsqueeze(1) for t in T1), S3)
    assert o1.shape == (2, 2, 32) and torch.equal(o1, o2) and torch.equal(o1, o3.squeeze(1)) and torch.equal(S1, S2) and torch.equal(S1, S3)
    w = torch.randn((2, 32), device="cuda")
    for args in ((x["v"], w, w), (x["v"], None, w), (x["v"], w[0].contiguous(), None), (x["v"][0, 0, 0].contiguous(), None, None)):
        y, m, r = kdn.layer_norm(*args)
        y2, m2, r2 = kdn.layer_norm(*args, stream=st)
        assert torch.equal(y, y2) and torch.equal(m, m2) and torch.equal(r, r2) and m.shape == m2.shape == args[0].shape[:-1]
        d, d2 = (kdn.layer_norm_backward(y, args[0], args[1], m, r, **kw) for kw in ({}, dict(stream=st)))
        assert d.keys() == d2.keys() and all(torch.equal(d[n], d2[n]) for n in d)
    kdn.last_device_error()


FIRST_USE = """
import sys, torch
import kalman_delta_rule_b200.binding as kdn
dt = getattr(torch, sys.argv[1])
torch.manual_seed(0)
r = lambda *s: torch.randn(s, device="cuda").to(dt)
q, k, v, do = r(1, 2300, 1, 64), r(1, 2300, 1, 64), r(1, 2300, 1, 64), r(1, 2300, 1, 64)
g = -torch.rand((1, 2300, 1), device="cuda")
S = torch.zeros((1, 1, 64, 64), device="cuda")
w = torch.ones(64, device="cuda")
def calls():
    o, last = kdn.linear_forward(q, k, v, g)
    y, mean, rstd = kdn.layer_norm(o, w, w)
    n = kdn.layer_norm_backward(do, o, w, mean, rstd)
    b = kdn.linear_backward(q, k, v, g, n["dx"])
    t = kdn.linear_decode_tokens(q[:, :1].contiguous(), k[:, :1].contiguous(), v[:, :1].contiguous(), g[:, :1].contiguous(), S)
    return [last, y, n["dweight"], b["dq"], b["dg"], t]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
S.zero_()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
S.zero_()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
kdn.last_device_error()
print("same")
"""


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_first_use_inside_a_capture(kdn, dtype):
    """The process's first call of every operator is captured; its replay gives the eager calls' bits."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_USE, dtype], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
