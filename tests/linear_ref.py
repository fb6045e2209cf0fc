"""Plain fp64 forms of linear attention with a decay for each head and of layer norm, and the error
bounds that the kernels are held to.

A kernel's error has two parts.  Sums of n fp32 products are off by at most n 2^-24 times the sum of the
products' magnitudes: ``mag_*`` below are the outputs with every input replaced by its magnitude, so
n 2^-24 mag bounds them.  Roundings to bf16 are off by at most 2^-8 of the rounded value each: the
output, and for bf16 inputs the matrix products' operands that are not inputs -- the decayed scores and
the chunk's initial state or state gradient, once each; ``round_*`` are the sums of magnitudes that
these carry into an output."""
import torch

U32 = 2.0 ** -24
U16 = 2.0 ** -8
CHUNK = 128      # the longest chunk of any path: bounds what a rounded operand can reach


def f64(x):
    return None if x is None else x.detach().double().cpu()


def token_decay(g, shape):
    """g as [B, T, H] in fp64 (resets as a decay of e^-2000: exactly zero in products with normal values)."""
    if g is None:
        return torch.zeros(shape, dtype=torch.float64)
    return f64(g).clamp(min=-2000.0).expand(shape).contiguous()


def sequences(q, cu):
    B, T = q.shape[:2]
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = cu.cpu().tolist()
    return [(0, c[i], c[i + 1]) for i in range(len(c) - 1)]


def forward(q, k, v, g, cu=None, S0=None, scale=1.0):
    """dict of o, S and the magnitudes mag_o, mag_S, round_o; the recurrence, token by token."""
    q, k, v, S0 = f64(q), f64(k), f64(v), f64(S0)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    gt = token_decay(g, (B, T, H))
    seqs = sequences(q, cu)
    out = {n: torch.zeros(v.shape, dtype=torch.float64) for n in ("o", "mag_o", "round_o")}
    out["S"], out["mag_S"] = (torch.zeros((len(seqs), H, dk, dv), dtype=torch.float64) for _ in range(2))
    for n, (b, t0, t1) in enumerate(seqs):
        S = torch.zeros((H, dk, dv), dtype=torch.float64) if S0 is None else S0[n].clone()
        M = S.abs()
        for c0 in range(t0, t1, CHUNK):
            c1 = min(c0 + CHUNK, t1)
            start = S.abs()
            for t in range(c0, c1):
                f = gt[b, t].exp()[:, None, None]
                S = f * S + k[b, t][:, :, None] * v[b, t][:, None, :]
                M = f * M + (k[b, t][:, :, None] * v[b, t][:, None, :]).abs()
                out["o"][b, t] = scale * torch.einsum("hi,hij->hj", q[b, t], S)
                out["mag_o"][b, t] = abs(scale) * torch.einsum("hi,hij->hj", q[b, t].abs(), M)
            G = gt[b, c0:c1].cumsum(0)
            D = torch.exp((G[:, None] - G[None]).clamp(max=0.0)) * torch.ones(c1 - c0, c1 - c0).tril()[:, :, None]
            P = torch.einsum("thi,shi->tsh", q[b, c0:c1], k[b, c0:c1]) * D * scale
            out["round_o"][b, c0:c1] = torch.einsum("tsh,shj->thj", P.abs(), v[b, c0:c1].abs()) + \
                abs(scale) * G.exp()[:, :, None] * torch.einsum("thi,hij->thj", q[b, c0:c1].abs(), start)
        out["S"][n], out["mag_S"][n] = S, M
    return out


def backward(q, k, v, g, do, cu=None, S0=None, dS=None, scale=1.0):
    """dict of dq, dk, dv, dg [B,T,H], dS0, their mag_* and round_*; whole sequences as triangular products."""
    q, k, v, do, S0, dS = (f64(x) for x in (q, k, v, do, S0, dS))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    gt = token_decay(g, (B, T, H))
    seqs = sequences(q, cu)
    out = {}
    for p in ("", "mag_", "round_"):
        out[p + "dq"], out[p + "dk"], out[p + "dv"] = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        out[p + "dg"], out[p + "dS0"] = torch.zeros_like(gt), torch.zeros((len(seqs), H, dk, dv), dtype=torch.float64)
    for n, (b, t0, t1) in enumerate(seqs):
        for h in range(H):
            s0 = torch.zeros((dk, dv), dtype=torch.float64) if S0 is None else S0[n, h]
            ds = torch.zeros((dk, dv), dtype=torch.float64) if dS is None else dS[n, h]
            a = [x[b, t0:t1, h] for x in (q, k, v, do)]
            G = gt[b, t0:t1, h].cumsum(0)
            r = _backward_one(*a, G, s0, ds, scale)
            m = _backward_one(*(x.abs() for x in a), G, s0.abs(), ds.abs(), abs(scale), magnitudes=True)
            w = _operand_roundings(*a, G, s0, ds, scale)
            for name in ("dq", "dk", "dv", "dg"):
                out[name][b, t0:t1, h], out["mag_" + name][b, t0:t1, h] = r[name], m[name]
            for name in ("dq", "dk", "dv"):
                out["round_" + name][b, t0:t1, h] = w[name]
            out["dS0"][n, h], out["mag_dS0"][n, h] = r["dS0"], m["dS0"]
    return out


def _backward_one(Q, K, V, dO, G, S0, dT, scale, magnitudes=False):
    L = len(G)
    D = torch.exp((G[:, None] - G[None]).clamp(max=0.0)).tril()
    since = G.exp()[:, None]
    until = torch.exp(G[-1] - G)[:, None] if L else since
    whole = G[-1].exp() if L else torch.tensor(1.0, dtype=torch.float64)
    P, R = scale * (Q @ K.T) * D, scale * (dO @ V.T) * D
    qf, kl = scale * since * (dO @ S0.T), until * (V @ dT.T)
    Z = P * (dO @ V.T)
    ends, starts = (Q * qf).sum(1), (K * kl).sum(1)
    # pairs (query i >= t, key j < t): the strictly-before-t columns of the rows from t on
    rect = ((Z.cumsum(1) - Z).flip(0).cumsum(0).flip(0)).diagonal() if L else G
    dg = rect + ends.flip(0).cumsum(0).flip(0) + (starts.cumsum(0) - starts) + (whole * S0 * dT).sum()
    if magnitudes and L:       # what an implementation may sum before it subtracts: the chunk's whole triangle
        dg = dg + torch.stack([Z[t // CHUNK * CHUNK:(t // CHUNK + 1) * CHUNK].sum() for t in range(L)])
    return {"dq": R @ K + qf, "dk": R.T @ Q + kl, "dv": P.T @ dO + until * (K @ dT), "dg": dg,
            "dS0": scale * (Q * since).T @ dO + whole * dT}


def _operand_roundings(Q, K, V, dO, G, S0, dT, scale):
    """Magnitudes that one rounding of the chunk's decayed score matrices, of the states at the chunks'
    starts and of the state gradients at their ends carry into dq, dk and dv."""
    L = len(G)
    out = {"dq": torch.zeros_like(Q), "dk": torch.zeros_like(K), "dv": torch.zeros_like(V)}
    cuts = list(range(0, L, CHUNK))
    S, states = S0, []
    for c in cuts:
        states.append(S)
        g = G[c:c + CHUNK] - (G[c - 1] if c else 0.0)
        S = g[-1].exp() * S + (K[c:c + CHUNK] * (g[-1] - g).exp()[:, None]).T @ V[c:c + CHUNK]
    R = dT
    for c, S in reversed(list(zip(cuts, states))):
        sl = slice(c, c + CHUNK)
        g = G[sl] - (G[c - 1] if c else 0.0)
        D = torch.exp((g[:, None] - g[None]).clamp(max=0.0)).tril()
        P, dA = (scale * (Q[sl] @ K[sl].T) * D).abs(), (scale * (dO[sl] @ V[sl].T) * D).abs()
        since, until = abs(scale) * g.exp()[:, None], (g[-1] - g).exp()[:, None]
        out["dq"][sl] = dA @ K[sl].abs() + since * (dO[sl].abs() @ S.abs().T)
        out["dk"][sl] = dA.T @ Q[sl].abs() + until * (V[sl].abs() @ R.abs().T)
        out["dv"][sl] = P.T @ dO[sl].abs() + until * (K[sl].abs() @ R.abs())
        R = g[-1].exp() * R + scale * (Q[sl] * g.exp()[:, None]).T @ dO[sl]
    return out


def terms(T, dk, dv):
    """Products and factors on the longest path of additions into an output: two inner products over the
    head sizes, two over a chunk, the scan over the chunks (of 64 tokens at least), and the decay factors
    (a dozen units in the last place)."""
    return 2 * max(dk, dv) + 2 * CHUNK + T // 64 + 32


def assert_within(got, want, bound, what):
    """Elementwise |got - want| <= bound (plus the smallest normal fp32 value: products may underflow)."""
    err = (f64(got) - want).abs()
    bad = ~(err <= bound + 2.0 ** -126)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst {float((err - bound).max()):.3e} "
                           f"over its bound, relative 2-norm {float(err.norm() / want.norm().clamp(min=1e-300)):.2e}")


def close_2norm(got, want, tol, what):
    err = float((f64(got) - want).norm() / want.norm().clamp(min=1e-300))
    assert err <= tol, f"{what}: relative 2-norm error {err:.3e} > {tol:.1e}"


def norm_forward(x, w, b, eps):
    x = f64(x)
    m = x.mean(-1, keepdim=True)
    r = ((x - m).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - m) * r
    if w is not None:
        y = y * f64(w)
    if b is not None:
        y = y + f64(b)
    return y, m.squeeze(-1), r.squeeze(-1)


def norm_backward(dy, x, w, mean, rstd):
    x, dy, mean, r = f64(x), f64(dy), f64(mean).unsqueeze(-1), f64(rstd).unsqueeze(-1)
    xh = (x - mean) * r
    u = dy if w is None else dy * f64(w)
    dx = r * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    return dx, xh
