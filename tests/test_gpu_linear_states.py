"""GPU tests of the precision of linear attention's states: 24 bits through bf16 products, and over long sequences."""
import pytest
import torch

from tests import linear_ref as R

pytestmark = pytest.mark.gpu


def one_hot(T, d):
    """Row t is the unit vector t mod d: an element of the state sums one product per d tokens."""
    return torch.eye(d)[torch.arange(T) % d][None, :, None].bfloat16().cuda()


def last_states(x, chunk=512):
    """The last state and the first state's gradient in fp64, chunk by chunk as the recurrence unrolls; B = H = 1."""
    q, k, v, do = (x[n][0, :, 0].double() for n in ("q", "k", "v", "do"))
    T = q.shape[0]
    g = x["g"].double().reshape(-1).expand(T)
    S, D = (torch.zeros(q.shape[1], v.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    starts = range(0, T, chunk)
    for t in starts:
        G = g[t:t + chunk].cumsum(0)
        S = G[-1].exp() * S + (k[t:t + chunk] * (G[-1] - G).exp()[:, None]).T @ v[t:t + chunk]
    for t in reversed(starts):
        G = g[t:t + chunk].cumsum(0)
        D = G[-1].exp() * D + (q[t:t + chunk] * G.exp()[:, None]).T @ do[t:t + chunk]
    return S, D


def check_states(kdn, T, g, limit):
    gen = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(s, generator=gen).bfloat16().cuda()   # noqa: E731
    x = {"q": one_hot(T, 128), "k": one_hot(T, 128), "v": rn(1, T, 1, 64), "do": rn(1, T, 1, 64), "g": g}
    _, S = kdn.linear_forward(x["q"], x["k"], x["v"], g)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], g, x["do"])
    kdn.last_device_error()
    wantS, wantD = last_states(x)
    R.close_2norm(S[0, 0], wantS.cpu(), limit, "S")
    R.close_2norm(out["dS0"][0, 0], wantD.cpu(), limit, "dS0")


@pytest.mark.parametrize("T", [100, 128])
def test_a_chunk_s_weighted_rows_keep_24_bits(kdn, T):
    """One product per element of the state: its error is that of the token's decay (an exponential, the chunk's factor and
    their product, three units of 2^-24 each at most but rarely together), the product's and the sum's roundings: 8 units bound
    the 2-norm.  Rows weighted in two bf16 terms leave 2.4e-6 (41 units; measured on such products)."""
    gen = torch.Generator().manual_seed(T)
    check_states(kdn, T, -0.05 * torch.rand((1, T, 1), generator=gen).cuda(), 8 * R.U32)


def test_a_constant_decay_near_one_over_a_long_sequence(kdn):
    """65536 tokens of one decay, a factor f = 0.9946 per chunk of 128: the state remembers some 93 chunks (1 / (1 - f^2)).  Two
    roundings per chunk, at random: sqrt(186) 0.4 units; the weights' common error, two units: 8 units, with as much again to
    spare, bound the 2-norm.  f in one float would be off by 2.6e-8 of itself, the same way in every chunk: sqrt(2) 93 of
    that, 3.4e-6."""
    check_states(kdn, 65536, torch.tensor([-2.0 ** -15 * (1 + 6 / 16)], device="cuda"), 16 * R.U32)
