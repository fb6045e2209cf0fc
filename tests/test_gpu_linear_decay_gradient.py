"""GPU tests of the log decay's gradient, whose four sums are formed from their own terms: no larger sum is subtracted, so a
reset's gradient is zero and a strong decay's keeps its bits, at every length.  Bounds: as in tests/linear_ref.py, with the
magnitudes of the gradient's own terms only."""
import pytest
import torch

from tests import linear_ref as R
from tests import test_gpu_linear as TL

pytestmark = pytest.mark.gpu


def before(x, dim):
    """Sums of the entries before each one along dim (as a difference of inclusive sums a term of 1e-22 would be lost)."""
    return torch.cat([torch.zeros_like(x.narrow(dim, 0, 1)), x.cumsum(dim).narrow(dim, 0, x.shape[dim] - 1)], dim)


def one_head(Q, K, V, dO, G, S0, dT):
    since, until = G.exp()[:, None], torch.exp(G[-1] - G)[:, None]
    Z = (Q @ K.T) * (dO @ V.T) * torch.exp((G[:, None] - G[None]).clamp(max=0.0)).tril()
    pairs = before(Z, 1).flip(0).cumsum(0).flip(0).diagonal()
    queries = (Q * since * (dO @ S0.T)).sum(1).flip(0).cumsum(0).flip(0)
    return pairs + queries + before((K * until * (V @ dT.T)).sum(1), 0) + (G[-1].exp() * S0 * dT).sum()


def own_terms(x, cu=None):
    """dg [B, T, H] in fp64 and the sum of its terms' magnitudes: pairs (query at or behind t, key before t), the initial
    state with the queries from t on, the last state's gradient with the keys before t, and the two states."""
    q, k, v, do, S0, dS = (R.f64(x[n]) for n in ("q", "k", "v", "do", "S0", "dS"))
    gt = R.token_decay(x["g"], q.shape[:3])
    out = [torch.zeros_like(gt), torch.zeros_like(gt)]
    for n, (b, t0, t1) in enumerate(R.sequences(q, cu)):
        if t1 == t0:
            continue
        for h in range(q.shape[2]):
            a = [t[b, t0:t1, h] for t in (q, k, v, do)]
            G = gt[b, t0:t1, h].cumsum(0)
            out[0][b, t0:t1, h] = one_head(*a, G, S0[n, h], dS[n, h])
            out[1][b, t0:t1, h] = one_head(*(t.abs() for t in a), G, S0[n, h].abs(), dS[n, h].abs())
    return out


def check(kdn, x, cu=None):
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    kdn.last_device_error()
    dg, mag = own_terms(x, cu)
    T, dk, dv = x["q"].shape[1], x["q"].shape[-1], x["v"].shape[-1]
    n = 2 * R.terms(T, dk, dv) * R.U32                  # two chains of sums meet in it
    if x["g"].dim() == 1:
        dg, mag = dg.sum((0, 1)), mag.sum((0, 1))
    R.assert_within(out["dg"], dg, n * mag, "dg")
    return out["dg"]


LENGTHS = [5, 16, 32, 33, 64, 65, 128, 129, 200, 300]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 256)])
@pytest.mark.parametrize("T", LENGTHS)
def test_resets_have_no_gradient(kdn, dtype, dk, dv, T):
    x = TL.make(T + dk, 2, T, 2, dk, dv, dtype, "token", grads=True)
    at = [t for t in (0, 1, 4, 15, 31, 32, 40, 63, 64, 100, 127, 128, 131, 190, 299) if t < T]
    x["g"][:, at] = -float("inf")
    dg = check(kdn, x)
    assert (dg[:, at] == 0).all(), f"{int((dg[:, at] != 0).sum())} of {dg[:, at].numel()} resets have a gradient"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_a_strong_decay_keeps_its_bits(kdn, dtype, T):
    """Tokens of e^-25 and e^-50 among weak ones: their gradients are 1e-11 and 1e-22 of the other tokens' terms."""
    x = TL.make(T, 2, T, 2, 64, 64, dtype, "token", grads=True)
    for t in range(3, T, 7):
        x["g"][:, t] = -25.0 if t % 2 else -50.0
    check(kdn, x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_and_per_head(kdn, dtype):
    lens = [0, 40, 1, 130, 129, 0, 300]
    cu = TL.offsets(lens)
    x = TL.make(5, 1, sum(lens), 2, 64, 128, dtype, "token", N=len(lens), grads=True)
    x["g"][:, ::9] = -float("inf")
    dg = check(kdn, x, cu)
    assert (dg[:, ::9] == 0).all()
    x["g"] = torch.tensor([-float("inf"), -0.01], device="cuda")
    assert check(kdn, x, cu)[0] == 0
    x["g"] = torch.tensor([-18.0, -0.3], device="cuda")
    check(kdn, x, cu)
