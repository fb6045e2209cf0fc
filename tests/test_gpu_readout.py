"""GPU test of the operators together, as a layer uses them: linear attention, the layer norm of each head's
readout, the gradients of both, and single tokens that continue the prompt."""
import pytest
import torch

from tests import linear_ref as R
from tests import test_gpu_linear as TL
from tests import test_gpu_norm as TN

pytestmark = pytest.mark.gpu
EPS = 1e-5


def layer(kdn, x, w, b, dy, cu=None):
    """(o, S), (y, mean, rstd), the norm's gradients, the attention's"""
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"])
    y, mean, rstd = kdn.layer_norm(o, w, b, eps=EPS)
    n = kdn.layer_norm_backward(dy, o, w, mean, rstd)
    a = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], n["dx"], cu_seqlens=cu, S0=x["S0"])
    return (o, S), (y, mean, rstd), n, a


def make(seed, B, T, H, dk, dv, dtype, decay, N):
    x = TL.make(seed, B, T, H, dk, dv, dtype, decay, N=N)
    _, dy, w, b = TN.make(seed + 1, (B, T, H, dv), dtype, G=H)
    return x, w, b, dy


CASES = [(2, 200, 3, 64, 128, "token", None), (1, 333, 2, 128, 256, "head", [130, 3, 200]), (1, 2400, 1, 64, 64, "token", None)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv,decay,lens", CASES)
def test_each_stage_on_what_the_one_before_left(kdn, dtype, B, T, H, dk, dv, decay, lens):
    cu = TL.offsets(lens) if lens else None
    x, w, b, dy = make(T, B, T, H, dk, dv, dtype, decay, len(lens) if lens else B)
    (o, S), (y, mean, rstd), n, a = layer(kdn, x, w, b, dy, cu)
    TL.check_forward(x, o, S, dtype, cu=cu)
    TN.check_forward(o, w, b, EPS, (y, mean, rstd))
    TN.check_backward(dy, o, w, mean, rstd, n)
    TL.check_backward({**x, "do": n["dx"], "dS": None}, a, dtype, cu=cu)
    kdn.last_device_error()


@pytest.mark.parametrize("B,T,H,dk,dv,decay,lens", CASES[:2])
def test_gradients_of_the_whole(kdn, B, T, H, dk, dv, decay, lens):
    """fp32 against the fp64 gradients of the composition, with the error bound carried through it.  An error e of a
    row of the readout (2-norms over d) moves xh = (x - m) r by at most 2 r |e| and r by r^2 |e| / sqrt(d); with
    |xh| <= sqrt(d) and |mean(u xh)| <= |u| / sqrt(d) the norm's gradient r (u - mean u - xh mean(u xh)) moves by at
    most 6 r^2 |e| |u| / sqrt(d) to first order.  Its own roundings stay below 4 (d + 32) 2^-24 r |u|.  The
    attention's gradients are linear in it: the sum of both goes through them with every input's magnitude (a
    row's 2-norm bounds each of its elements)."""
    cu = TL.offsets(lens) if lens else None
    x, w, b, dy = make(T + 5, B, T, H, dk, dv, "f32", decay, len(lens) if lens else B)
    a = layer(kdn, x, w, b, dy, cu)[3]
    f = R.forward(x["q"], x["k"], x["v"], x["g"], cu=cu, S0=x["S0"])
    _, m, r = R.norm_forward(f["o"], w, b, EPS)
    dx, _ = R.norm_backward(dy, f["o"], w, m, r)
    want = R.backward(x["q"], x["k"], x["v"], x["g"], dx, cu=cu, S0=x["S0"])
    t = R.terms(T, dk, dv) * R.U32
    e = (t * f["mag_o"]).norm(dim=-1, keepdim=True)
    u = (R.f64(dy) * R.f64(w)).norm(dim=-1, keepdim=True)
    r = r[..., None]
    moved = 1.01 * (6 * r * r * e * u / dv ** 0.5 + 4 * (dv + 32) * R.U32 * r * u)
    far = R.backward(*(x[n].abs() for n in ("q", "k", "v")), x["g"], moved.expand_as(dx), cu=cu, S0=x["S0"].abs())
    for name in ("dq", "dk", "dv", "dS0"):
        R.assert_within(a[name], want[name], t * want["mag_" + name] + far["mag_" + name], name)
    dg, bound = want["dg"], 2 * t * want["mag_dg"] + far["mag_dg"]
    if x["g"].dim() == 1:
        dg, bound = dg.sum((0, 1)), bound.sum((0, 1))
    R.assert_within(a["dg"], dg, bound, "dg")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_single_tokens_continue_the_prompt(kdn, dtype):
    """Prompt and single tokens, the norm behind each: the same rows as the whole sequence at once, up to the roundings of
    its readout (to the type: half a step each way; sums in fp32) through the norm."""
    B, T, H, d, n = 2, 140, 2, 64, 6
    x, w, b, _ = make(3, B, T, H, d, d, dtype, "token", B)
    cut = {m: x[m][:, :T - n].contiguous() for m in ("q", "k", "v", "g")}
    _, S = kdn.linear_forward(cut["q"], cut["k"], cut["v"], cut["g"], S0=x["S0"])
    f = R.forward(x["q"], x["k"], x["v"], x["g"], S0=x["S0"])
    for t in range(T - n, T):
        o = kdn.linear_decode_step(*(x[m][:, t].contiguous() for m in ("q", "k", "v", "g")), S)
        y, mean, rstd = kdn.layer_norm(o, w, b, eps=EPS)
        bound = R.terms(T, d, d) * R.U32 * f["mag_o"][:, t]
        if dtype == "bf16":
            bound = bound * (1 + R.U16) + R.U16 * f["o"][:, t].abs()
        R.assert_within(o.float(), f["o"][:, t], bound, f"o at {t}")
        TN.check_forward(o, w, b, EPS, (y, mean, rstd))
    R.assert_within(S, f["S"], R.terms(T, d, d) * R.U32 * f["mag_S"], "S")
