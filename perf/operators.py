"""Measured cases of the linear-attention and layer-norm operators: inputs, plain forms, exact values and floors.

Plain forms are elementary torch operations in 32 bits (angles of the decay -- sums of log decays -- in 64), rounded
once at the end; with ``own`` set, ``run`` makes the calls a user makes of ``kalman_delta_rule_b200.binding``.

Linear attention with a decay for each head:  S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t, with the log
decay g per token and head [B, T, H], per head [H], or none.  Layer norm over the last axis with one weight and bias
row for all rows ([d]) or one for each head ([H, d], the norm of a layer's readout)."""
import math
import random

import torch

own = False

CHUNK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: one short prompt of a test-sized model, fp32; all latency
        dict(name="forward tiny fp32", op="forward", dtype="f32", B=1, T=256, H=2, dk=32, dv=32, decay="token", seqs=0, state=False),
        # a batch of prompts or the forward of a training step
        dict(name="forward prefill", op="forward", dtype="bf16", B=4, T=4096, H=16, dk=128, dv=128, decay="token", seqs=0, state=False),
        # one very long document, fixed decay for each head: few chains, a long serial axis
        dict(name="forward long", op="forward", dtype="bf16", B=1, T=65536, H=32, dk=128, dv=128, decay="head", seqs=0, state=False),
        # ragged prompts packed into one row, wide values, states carried in from earlier calls
        dict(name="forward packed", op="forward", dtype="bf16", B=1, T=65533, H=16, dk=128, dv=256, decay="token", seqs=12, state=True),
        # interactive serving: a handful of sequences, one token
        dict(name="decode few", op="decode", dtype="bf16", B=4, T=1, H=16, dk=128, dv=128, decay="token", seqs=0, state=True),
        # full serving batch, one token: the state is the traffic
        dict(name="decode many", op="decode", dtype="bf16", B=256, T=1, H=32, dk=128, dv=128, decay="token", seqs=0, state=True),
        # the backward of a training step
        dict(name="backward train", op="backward", dtype="bf16", B=4, T=4096, H=16, dk=128, dv=128, decay="token", seqs=0, state=False),
        # packed short documents in fp32, with gradients of the carried states
        dict(name="backward ragged fp32", op="backward", dtype="f32", B=1, T=5003, H=4, dk=64, dv=64, decay="token", seqs=24, state=True),
        # the readout's norm of the prefill: a weight row for each head
        dict(name="norm heads", op="norm", dtype="bf16", n=16384, G=16, d=128, affine=True),
        # odd width, few rows, fp32
        dict(name="norm odd fp32", op="norm", dtype="f32", n=1021, G=1, d=1001, affine=True),
        # the gradient of the readout's norm
        dict(name="norm backward heads", op="norm_backward", dtype="bf16", n=16384, G=16, d=128, affine=True),
        # the gradient of a norm over the whole width
        dict(name="norm backward wide", op="norm_backward", dtype="bf16", n=16384, G=1, d=4096, affine=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "decode", "backward", "backward", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        G = rng.choice([1, 1, rng.randint(2, 32)])
        d = _log(rng, 32, 8192 // G)
        n = _log(rng, 1, max(1, (1 << (25 if dtype == "bf16" else 24)) // (G * d)))
        return dict(op=op, dtype=dtype, n=n, G=G, d=d, affine=rng.random() < 0.8)
    dk, dv = rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128, 256])
    H = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
    decay = rng.choice(["token", "token", "head", "none"])
    if op == "decode":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 8192 // H), T=rng.choice([1, 1, 1, 2, 4, 7]), H=H, dk=dk, dv=dv,
                    decay=decay, seqs=0, state=True)
    most = (1 << (18 if dtype == "bf16" else 16)) // H           # tokens of the whole batch
    T = _log(rng, 1, min(most, 16384))
    if rng.random() < 0.4:                                       # packed: T tokens in all
        return dict(op=op, dtype=dtype, B=1, T=T, H=H, dk=dk, dv=dv, decay=decay, seqs=_log(rng, 1, min(T, 40)),
                    state=rng.random() < 0.6)
    return dict(op=op, dtype=dtype, B=_log(rng, 1, max(1, min(64, most // T))), T=T, H=H, dk=dk, dv=dv, decay=decay,
                seqs=0, state=rng.random() < 0.5)


def _lengths(case, seed):
    """Ragged lengths that sum to T: shares of an exponential law, some of them one or zero tokens."""
    r, n, T = random.Random(seed * 7919 + 17), case["seqs"], case["T"]
    cuts = [r.expovariate(1.0) ** 1.3 + 1e-3 for _ in range(n)]
    if n > 4:
        cuts[1] = 0.0                                            # a request whose tokens were all cached
    total, acc, ends = sum(cuts), 0.0, []
    for c in cuts:
        acc += c
        ends.append(min(T, int(round(acc / total * T))))
    ends[-1] = T
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    if case["op"].startswith("norm"):
        n, G, d = case["n"], case["G"], case["d"]
        shape = (n, G, d) if G > 1 else (n, d)
        wshape = (G, d) if G > 1 else (d,)
        x = (0.7 * randn(*shape) + 0.3 * randn(*shape[:-1], 1)).to(dt)
        st = dict(op=case["op"], x=x, eps=1e-5, weight=None, bias=None)
        if case["affine"]:
            st["weight"], st["bias"] = 1.0 + 0.1 * randn(*wshape), 0.1 * randn(*wshape)
        if case["op"] == "norm_backward":
            st["dy"] = randn(*shape).to(dt)
            xd = x.double()                                      # what the forward call left
            mean = xd.mean(-1)
            st["mean"] = mean.float()
            st["rstd"] = ((xd - mean.unsqueeze(-1)).square().mean(-1) + st["eps"]).rsqrt().float()
        return st
    B, T, H, dk, dv = (case[x] for x in ("B", "T", "H", "dk", "dv"))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)            # noqa: E731  (keys and queries are L2-normalised)
    st = dict(op=case["op"], scale=1.0, cu=None, lens=None, S0=None, dS=None)
    st["q"], st["k"] = unit(randn(B, T, H, dk)).to(dt), unit(randn(B, T, H, dk)).to(dt)
    st["v"] = randn(B, T, H, dv).to(dt)
    st["g"] = None
    if case["decay"] == "token":                                 # log of a sigmoid gate around 0.98
        st["g"] = -torch.nn.functional.softplus(-4.0 - randn(B, T, H))
    elif case["decay"] == "head":                                # 1 - 2^-5 ... 1 - 2^-12 over the heads, with a little spread
        at = torch.linspace(5.0, 12.0, H, device="cuda") + 0.1 * randn(H)
        st["g"] = torch.log1p(-torch.exp2(-at))
    N = B
    if case["seqs"]:
        lens = _lengths(case, seed)
        N = len(lens)
        ends = torch.tensor([0] + lens).cumsum(0)
        st["cu"], st["longest"] = ends.to(torch.int32).cuda(), max(lens)
    if case["state"]:
        st["S0"] = 0.1 * randn(N, H, dk, dv)
    if case["op"] == "backward":
        st["do"] = randn(B, T, H, dv).to(dt)
        if case["state"]:
            st["dS"] = 0.1 * randn(N, H, dk, dv)
    return st


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        rows, d, G = case["n"] * case["G"], case["d"], case["G"]
        par = 4 * G * d * (2 if case["affine"] else 0)
        if case["op"] == "norm":
            return dict(bytes=rows * (2 * e * d + 8) + par, flops=8 * rows * d)
        return dict(bytes=rows * (3 * e * d + 8) + par * 3 // 2, flops=14 * rows * d)
    B, T, H, dk, dv = (case[x] for x in ("B", "T", "H", "dk", "dv"))
    th, N = B * T * H, case["seqs"] or B
    states = 4 * N * H * dk * dv
    g = {"token": 4 * th, "head": 4 * H, "none": 0}[case["decay"]]
    if case["op"] == "backward":
        return dict(bytes=th * e * (4 * dk + 3 * dv) + 2 * g + (3 if case["state"] else 1) * states, flops=10 * th * dk * dv)
    return dict(bytes=th * e * 2 * (dk + dv) + g + (2 if case["state"] else 1) * states, flops=4 * th * dk * dv)


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        from kalman_delta_rule_b200 import binding as kdn
        op = st["op"]
        if op == "forward":
            return kdn.linear_forward(st["q"], st["k"], st["v"], st["g"], cu_seqlens=st["cu"], S0=st["S0"], scale=st["scale"])
        if op == "decode":
            o = kdn.linear_decode_tokens(st["q"], st["k"], st["v"], st["g"], st["S0"], scale=st["scale"])
            return o, st["S0"]
        if op == "backward":
            return kdn.linear_backward(st["q"], st["k"], st["v"], st["g"], st["do"], cu_seqlens=st["cu"], S0=st["S0"],
                                       dS=st["dS"], scale=st["scale"])
        if op == "norm":
            return kdn.layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"])
        return kdn.layer_norm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"])
    return {"forward": _forward, "decode": _decode, "backward": _backward, "norm": _norm, "norm_backward": _norm_backward}[st["op"]](st)


# ------------------------------------------------------------------ plain forms
def _norm(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + st["eps"]).rsqrt()
    y = (x - mean) * rstd
    if st["weight"] is not None:
        y = y * st["weight"] + st["bias"]
    return y.to(st["x"].dtype), mean.squeeze(-1), rstd.squeeze(-1)


def _norm_backward(st):
    x, dy = st["x"].float(), st["dy"].float()
    rstd = st["rstd"].unsqueeze(-1)
    xh = (x - st["mean"].unsqueeze(-1)) * rstd
    wdy = dy if st["weight"] is None else dy * st["weight"]
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    out = {"dx": dx.to(st["x"].dtype)}
    if st["weight"] is not None:
        out["dweight"], out["dbias"] = (dy * xh).sum(0), dy.sum(0)
    return out


def _log_decay(st, dtype):
    """g as [B, T, H]."""
    q = st["q"]
    if st["g"] is None:
        return torch.zeros(q.shape[:3], dtype=dtype, device=q.device)
    return st["g"].to(dtype).expand(q.shape[:3])


def _unpack_index(st):
    """Packed rows as [sequence, position]: index of each place, which of them hold a token, and each token's place."""
    cu, T = st["cu"].long(), st["q"].shape[1]
    at = cu[:-1, None] + torch.arange(st["longest"], device=cu.device)
    there = at < cu[1:, None]
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return at.clamp(max=T - 1), there, (seq, t - cu[seq])


def _dense(st, names):
    """The named token tensors and g as [N, H, chunks, C, d] in 32 bits (g in 64, [N, H, chunks, C]); zeros behind each end."""
    xs = [st[n].float() for n in names] + [_log_decay(st, torch.float64)]
    back = None
    if st["cu"] is not None:
        at, there, back = _unpack_index(st)
        xs = [x[0][at] * there.reshape(there.shape + (1,) * (x.dim() - 2)) for x in xs]
    T = xs[0].shape[1]
    C = max(1, min(CHUNK, T))
    pad = -T % C
    out = []
    for x in xs:
        x = torch.nn.functional.pad(x.transpose(1, 2), (0, 0) * (x.dim() - 3) + (0, pad))
        out.append(x.reshape(x.shape[:2] + ((T + pad) // C, C) + x.shape[3:]))
    return out, T, back


def _tokens(x, T, back):
    """[N, H, chunks, C, ...] -> the inputs' layout."""
    x = x.flatten(2, 3)[:, :, :T].transpose(1, 2)
    return x.contiguous() if back is None else x[back].unsqueeze(0)


def _decays(g):
    """Of [N, H, n, C] log decays: G within a chunk, pairwise D, decay to the chunk's end, log decay before and behind each chunk."""
    C = g.shape[-1]
    G = g.cumsum(-1)
    tri = torch.ones(C, C, dtype=torch.bool, device=g.device).tril()
    D = torch.where(tri, (G.unsqueeze(-1) - G.unsqueeze(-2)).float(), -math.inf).exp()
    end = (G[..., -1:] - G).exp().float().unsqueeze(-1)
    total = G[..., -1].cumsum(-1)
    return G, D, end, total - G[..., -1], total


def _carried(U, before, behind, first, reverse=False):
    """States at each chunk's start, sum_{j<c} exp(before_c - behind_j) U_j + exp(before_c) first, and the last one; with
    ``reverse`` the mirror image: gradients at each chunk's end, from the chunks after it and the last state's."""
    n = U.shape[2]
    if reverse:
        L = before[..., None, :] - behind[..., :, None]          # chunk j > c reaches back to c's end
        ok = torch.ones(n, n, dtype=torch.bool, device=U.device).triu(1)
        whole = behind[..., -1:] - behind
    else:
        L = before[..., :, None] - behind[..., None, :]
        ok = torch.ones(n, n, dtype=torch.bool, device=U.device).tril(-1)
        whole = before
    S = (torch.where(ok, L, -math.inf).exp().float() @ U.flatten(3)).reshape(U.shape)
    if first is not None:
        S = S + whole.exp().float()[..., None, None] * first.unsqueeze(2)
    return S


def _forward(st):
    (q, k, v, g), T, back = _dense(st, ("q", "k", "v"))
    if T == 0:
        return st["v"].clone(), st["S0"].clone()
    G, D, end, before, behind = _decays(g)
    U = (k * end).transpose(-1, -2) @ v
    S = _carried(U, before, behind, st["S0"])
    a = G.exp().float().unsqueeze(-1)
    o = st["scale"] * (((q @ k.transpose(-1, -2)) * D) @ v + a * (q @ S))
    S_out = G[:, :, -1, -1].exp().float()[..., None, None] * S[:, :, -1] + U[:, :, -1]
    return _tokens(o, T, back).to(st["v"].dtype), S_out


def _decode(st):
    o, S = _forward(st)
    st["S0"].copy_(S)
    return o, st["S0"]


def _backward(st):
    (q, k, v, do, g), T, back = _dense(st, ("q", "k", "v", "do"))
    scale = st["scale"]
    G, D, end, before, behind = _decays(g)
    a = scale * G.exp().float().unsqueeze(-1)
    U = (k * end).transpose(-1, -2) @ v
    S = _carried(U, before, behind, st["S0"])
    E = (q * a).transpose(-1, -2) @ do
    dS = _carried(E, before, behind, st["dS"], reverse=True)     # gradient of the state behind each chunk
    A = scale * (q @ k.transpose(-1, -2)) * D
    dP = do @ v.transpose(-1, -2)
    dA = scale * dP * D
    dq_in, dk_in = a * (do @ S.transpose(-1, -2)), end * (v @ dS.transpose(-1, -2))
    dq, dk = dA @ k + dq_in, dA.transpose(-1, -2) @ q + dk_in
    dv = A.transpose(-1, -2) @ do + end * (k @ dS)
    step = G[..., -1].exp().float()[..., None, None]
    dS0 = step[:, :, 0] * dS[:, :, 0] + E[:, :, 0]
    # the decay's gradient: pairs (later query, earlier key) that the token's decay lies between
    Z = (A * dP).double()
    x = Z.sum(-1) + (q * dq_in).double().sum(-1)
    y = Z.sum(-2) + (k * dk_in).double().sum(-1)
    after = step * S + U
    dg = (x - y).flip(-1).cumsum(-1).flip(-1) + (after.double() * dS.double()).sum((-1, -2)).unsqueeze(-1)
    dt = st["q"].dtype
    out = {"dq": _tokens(dq, T, back).to(dt), "dk": _tokens(dk, T, back).to(dt), "dv": _tokens(dv, T, back).to(dt), "dS0": dS0}
    if st["g"] is not None:
        dg = _tokens(dg, T, back)
        out["dg"] = (dg.sum((0, 1)) if st["g"].dim() == 1 else dg).float()
    return out


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(st)
    steps = st["longest"] if st["cu"] is not None else case["T"]
    if case["op"] == "backward":
        N = case["seqs"] or case["B"]
        if N * case["H"] * float(steps) ** 2 > 3e9:
            return None
        return _exact_backward(st)
    return _exact_forward(st)


def _exact_norm(st):
    x = st["x"].double()
    n = x.shape[-1]
    if st["op"] == "norm":
        mean = x.sum(-1) / n
        dev = x - mean[..., None]
        rstd = 1.0 / torch.sqrt((dev * dev).sum(-1) / n + st["eps"])
        y = dev * rstd[..., None]
        if st["weight"] is not None:
            y = y * st["weight"].double() + st["bias"].double()
        return y, mean, rstd
    # the same scalar <y, dy> differentiated by hand: y = (x - m) r w + b with m and r as given by the forward
    dy, r = st["dy"].double(), st["rstd"].double()
    xh = (x - st["mean"].double()[..., None]) * r[..., None]
    up = dy if st["weight"] is None else dy * st["weight"].double()
    dot = torch.einsum("...d,...d->...", up, xh) / n
    dx = (up - up.sum(-1)[..., None] / n - dot[..., None] * xh) * r[..., None]
    out = {"dx": dx}
    if st["weight"] is not None:
        out["dweight"] = torch.einsum("n...d,n...d->...d", dy, xh)
        out["dbias"] = dy.sum(0)
    return out


def _sequences(st, names):
    """The named tensors one row per sequence in 64 bits, [N, steps, H, ...], zeros behind each end (a decay of 1 there)."""
    xs = [st[n].double() for n in names] + [_log_decay(st, torch.float64)]
    if st["cu"] is None:
        return xs
    cu = st["cu"].tolist()
    rows = []
    for x in xs:
        r = torch.zeros((len(cu) - 1, st["longest"]) + x.shape[2:], dtype=torch.float64, device=x.device)
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            r[i, : b - a] = x[0, a:b]
        rows.append(r)
    return rows


def _flat(st, x):
    if st["cu"] is None:
        return x
    cu = st["cu"].tolist()
    return torch.cat([x[i, : b - a] for i, (a, b) in enumerate(zip(cu, cu[1:]))]).unsqueeze(0)


def _exact_forward(st):
    """The recurrence, token by token."""
    q, k, v, g = _sequences(st, ("q", "k", "v"))
    N, steps, H, dk = q.shape
    S = torch.zeros((N, H, dk, v.shape[-1]), dtype=torch.float64, device=q.device) if st["S0"] is None else st["S0"].double()
    f = g.exp()
    o = torch.empty_like(v)
    for t in range(steps):
        S = torch.addcmul(S * f[:, t, :, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
        o[:, t] = torch.matmul(q[:, t, :, None, :], S).squeeze(-2)
    return _flat(st, o) * st["scale"], S


def _exact_backward(st):
    """The whole sequence as one lower-triangular product, sequence by sequence and head by head."""
    q, k, v, do, g = _sequences(st, ("q", "k", "v", "do"))
    N, steps, H, dk = q.shape
    scale, dv = st["scale"], v.shape[-1]
    zero = torch.zeros((dk, dv), dtype=torch.float64, device=q.device)
    outs = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v), "dg": torch.zeros_like(g),
            "dS0": torch.zeros((N, H, dk, dv), dtype=torch.float64, device=q.device)}
    for i in range(N):
        for h in range(H):
            Q, K, V, dO, G = q[i, :, h], k[i, :, h], v[i, :, h], do[i, :, h], g[i, :, h].cumsum(0)
            S0 = zero if st["S0"] is None else st["S0"][i, h].double()
            dT = zero if st["dS"] is None else st["dS"][i, h].double()
            D = torch.exp((G[:, None] - G[None, :]).tril()).tril()
            P, R = scale * (Q @ K.T) * D, scale * (dO @ V.T) * D
            since, until = torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None]
            from_first, to_last = scale * since * (dO @ S0.T), until * (V @ dT.T)
            outs["dq"][i, :, h] = R @ K + from_first
            outs["dk"][i, :, h] = R.T @ Q + to_last
            outs["dv"][i, :, h] = P.T @ dO + until * (K @ dT)
            outs["dS0"][i, h] = scale * (Q * since).T @ dO + torch.exp(G[-1]) * dT
            Z = P * (dO @ V.T)                                   # each pair's share of the scalar; g_t is in those that span t
            ends = Z.sum(1) + (Q * from_first).sum(1)
            starts = Z.sum(0) + (K * to_last).sum(1)
            kept = (torch.exp(G[-1]) * S0 * dT).sum() + (K * to_last).sum()
            outs["dg"][i, :, h] = (ends - starts).flip(0).cumsum(0).flip(0) + kept
    out = {n: _flat(st, outs[n]) for n in ("dq", "dk", "dv")}
    out["dS0"] = outs["dS0"]
    if st["g"] is not None:
        dg = _flat(st, outs["dg"])
        out["dg"] = dg.sum((0, 1)) if st["g"].dim() == 1 else dg
    return out
