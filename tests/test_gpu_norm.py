"""GPU tests of layer norm's forward and backward pass against the plain fp64 forms."""
import pytest
import torch

from tests import linear_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# every width class: parts of a warp, a warp, a CTA of 256 and of 512 threads; vector and element loads
WIDTHS = [1, 7, 32, 63, 64, 100, 128, 129, 256, 300, 512, 777, 1000, 1001, 1024, 1031, 2048, 2050, 4096, 4100, 8192, 8195, 16383, 16384,
          2, 6, 62, 126, 254, 510, 514, 1022, 1502, 4094, 8190, 12002]


def make(seed, shape, dtype, G=None, affine=True, offset=0.5):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(shape, generator=gen) + offset).to(DT[dtype]).cuda()
    dy = torch.randn(shape, generator=gen).to(DT[dtype]).cuda()
    w = b = None
    if affine:
        ws = (G, shape[-1]) if G else (shape[-1],)
        w, b = (1.0 + 0.2 * torch.randn(ws, generator=gen)).cuda(), torch.randn(ws, generator=gen).cuda()
    return x, dy, w, b


def check_forward(x, w, b, eps, got):
    y, mean, rstd = got
    want, m, r = R.norm_forward(x, w, b, eps)
    x64, d = R.f64(x), x.shape[-1]
    n = (d + 8) * R.U32
    top = x64.abs().amax(-1)
    # the mean of d values: d roundings of partial sums that are at most d max|x|
    em = n * x64.abs().mean(-1)
    R.assert_within(mean, m, em, "mean")
    # the variance moves by 2 |mean error| mean|x - m| + (mean error)^2 and its own sum's roundings; r by half its relative change
    dev = (x64 - m[..., None]).abs()
    var = dev.square().mean(-1)
    ev = em.square() + n * var + 4 * R.U32 * top * dev.mean(-1)
    er = r * (0.5 * ev * r.square() + 4 * R.U32)
    R.assert_within(rstd, r, 1.01 * er, "rstd")
    ww = 1.0 if w is None else R.f64(w).abs()
    bound = ww * ((em + 2 * R.U32 * top)[..., None] * r[..., None] + dev * (er + 2 * R.U32 * r)[..., None]) * 1.01
    bound = bound + 2 * R.U32 * (want.abs() + (0.0 if b is None else R.f64(b).abs()))
    if x.dtype == torch.bfloat16:
        bound = bound * (1 + R.U16) + R.U16 * want.abs()
    R.assert_within(y.float(), want, bound, "y")


def check_backward(dy, x, w, mean, rstd, out):
    want, xh = R.norm_backward(dy, x, w, mean, rstd)
    d = x.shape[-1]
    n = (d + 16) * R.U32
    g = R.f64(dy) if w is None else R.f64(dy) * R.f64(w)
    r = R.f64(rstd)[..., None]
    # x - mean is exact to one rounding of its operands' size; xh carries it into every term
    dxh = R.U32 * (2 * xh.abs() + 2 * r * (R.f64(x).abs() + R.f64(mean)[..., None].abs()))
    s2, m2 = (g * xh).mean(-1, keepdim=True), (g * xh).abs().mean(-1, keepdim=True)
    es2 = n * m2 + (g.abs() * dxh).mean(-1, keepdim=True)
    bound = r * (8 * R.U32 * (g.abs() + g.abs().mean(-1, keepdim=True) + (xh * s2).abs()) + n * g.abs().mean(-1, keepdim=True)
                 + xh.abs() * es2 + dxh * (s2.abs() + es2)) * 1.01
    if x.dtype == torch.bfloat16:
        bound = bound * (1 + R.U16) + R.U16 * want.abs()
    R.assert_within(out["dx"].float(), want, bound, "dx")
    if w is None:
        assert "dweight" not in out and "dbias" not in out
        return
    lead = tuple(range(x.dim() - w.dim()))
    dy64 = R.f64(dy)
    rows = max(1, x.numel() // w.numel())
    R.assert_within(out["dweight"], (dy64 * xh).sum(lead),
                    (rows + 16) * R.U32 * (dy64 * xh).abs().sum(lead) + (dy64.abs() * dxh).sum(lead), "dweight")
    R.assert_within(out["dbias"], dy64.sum(lead), (rows + 16) * R.U32 * dy64.abs().sum(lead), "dbias")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(kdn, dtype, d):
    for rows in (1, 37):
        x, dy, w, b = make(d + rows, (rows, d), dtype)
        got = kdn.layer_norm(x, w, b)
        check_forward(x, w, b, 1e-5, got)
        check_backward(dy, x, w, got[1], got[2], kdn.layer_norm_backward(dy, x, w, got[1], got[2]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 50, 4, 64), (1, 1, 16, 128), (3, 700, 3, 256), (5, 1, 1, 33), (2, 9, 33, 40), (700, 2, 1100)])
def test_heads(kdn, dtype, shape):
    """A weight row for each head; more rows than the launch has row places."""
    x, dy, w, b = make(3, shape, dtype, G=shape[-2])
    got = kdn.layer_norm(x, w, b, eps=1e-3)
    assert got[1].shape == shape[:-1]
    check_forward(x, w, b, 1e-3, got)
    out = kdn.layer_norm_backward(dy, x, w, got[1], got[2])
    assert out["dweight"].shape == w.shape
    check_backward(dy, x, w, got[1], got[2], out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_parameters_and_many_rows(kdn, dtype):
    x, dy, _, _ = make(5, (30011, 96), dtype, affine=False)
    got = kdn.layer_norm(x)
    check_forward(x, None, None, 1e-5, got)
    check_backward(dy, x, None, got[1], got[2], kdn.layer_norm_backward(dy, x, None, got[1], got[2]))
    x, dy, w, b = make(6, (30011, 96), dtype)
    for ww, bb in ((w, None), (None, b)):
        check_forward(x, ww, bb, 1e-5, kdn.layer_norm(x, ww, bb))
    _, mean, rstd = kdn.layer_norm(x, w, b)
    check_backward(dy, x, w, mean, rstd, kdn.layer_norm_backward(dy, x, w, mean, rstd))


def test_a_large_mean_and_a_constant_row(kdn):
    """The variance is formed from deviations: a mean of 1000 standard deviations costs it nothing more than
    the inputs' own rounding; a constant row normalises to the bias."""
    x, dy, w, b = make(7, (9, 1000), "f32", offset=1000.0)
    check_forward(x, w, b, 1e-5, kdn.layer_norm(x, w, b))
    x.fill_(3.0)
    y, mean, rstd = kdn.layer_norm(x, w, b, eps=1e-4)
    assert torch.equal(y, b.expand_as(y)) and (mean == 3.0).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)


def test_a_bad_row_stays_alone(kdn):
    x, dy, w, b = make(8, (40, 128), "bf16")
    y, mean, rstd = kdn.layer_norm(x, w, b)
    x2 = x.clone()
    x2[3, 5], x2[17, 0] = float("nan"), float("inf")
    y2, m2, r2 = kdn.layer_norm(x2, w, b)
    keep = [i for i in range(40) if i not in (3, 17)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(mean[keep], m2[keep]) and y2[3].isnan().all()
    g = kdn.layer_norm_backward(dy, x, w, mean, rstd)["dx"]
    g2 = kdn.layer_norm_backward(dy, x2, w, m2, r2)["dx"]
    assert torch.equal(g[keep], g2[keep])


def test_gradient_against_differences(kdn):
    """Central differences of the plain form's <y, dy> in fp64 at h = 1e-4: the cubic term is h^2 / 6 of third
    derivatives of size (1 / std)^3, below 1e-7 of the magnitudes here."""
    x, dy, w, b = make(9, (6, 50), "f32")
    y, mean, rstd = kdn.layer_norm(x, w, b)
    out = kdn.layer_norm_backward(dy, x, w, mean, rstd)
    gen = torch.Generator().manual_seed(2)
    scalar = lambda xx, ww, bb: float((R.norm_forward(xx, ww, bb, 1e-5)[0] * R.f64(dy)).sum())   # noqa: E731
    base = [R.f64(t) for t in (x, w, b)]
    for i, name in enumerate(("dx", "dweight", "dbias")):
        way = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + 1e-4 * way, base[i] - 1e-4 * way
        diff = (scalar(*up) - scalar(*dn)) / 2e-4
        got = float((R.f64(out[name]) * way).sum())
        assert abs(got - diff) <= 1e-5 * float((R.f64(out[name]) * way).abs().sum()), name


def test_repeatable_streams_and_graphs(kdn):
    x, dy, w, b = make(10, (5000, 4, 128), "bf16", G=4)
    y, mean, rstd = kdn.layer_norm(x, w, b)
    out = kdn.layer_norm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        again = kdn.layer_norm_backward(dy, x, w, mean, rstd)
        assert all(torch.equal(out[n], again[n]) for n in out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = kdn.layer_norm(x, w, b, stream=s)[0]
    o2 = kdn.layer_norm_backward(dy, x, w, mean, rstd, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(out[n], o2[n]) for n in out)
    xs, gr = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        yg, mg, rg = kdn.layer_norm(xs, w, b)
        og = kdn.layer_norm_backward(dy, xs, w, mg, rg)
    for scale in (0.5, 1.0):
        xs.copy_(x * scale)
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(yg, y) and all(torch.equal(out[n], og[n]) for n in out)


def test_empty_and_refusals(kdn):
    x, dy, w, b = make(11, (0, 64), "bf16")
    y, mean, rstd = kdn.layer_norm(x, w, b)
    assert y.shape == (0, 64) and mean.shape == (0,)
    out = kdn.layer_norm_backward(dy, x, w, mean, rstd)
    assert (out["dweight"] == 0).all() and (out["dbias"] == 0).all()
    x, dy, w, b = make(11, (3, 64), "bf16")
    y, mean, rstd = kdn.layer_norm(x, w, b)
    with pytest.raises(ValueError, match="contiguous"):
        kdn.layer_norm(x.t().contiguous().t(), w, b)
    with pytest.raises(TypeError):
        kdn.layer_norm(x.half())
    with pytest.raises(TypeError):
        kdn.layer_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        kdn.layer_norm(x, w[:32].contiguous())
    with pytest.raises(ValueError):
        kdn.layer_norm(x, w, b.cpu())
    with pytest.raises(ValueError):
        kdn.layer_norm(x, w.expand(2, 64).contiguous())
    with pytest.raises(kdn.KdnError):
        kdn.layer_norm(x, w, b, eps=-1.0)
    with pytest.raises(kdn.KdnError):
        kdn.layer_norm(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(TypeError):
        kdn.layer_norm_backward(dy.float(), x, w, mean, rstd)
    with pytest.raises(ValueError):
        kdn.layer_norm_backward(dy, x, w, mean[:2], rstd)
    with pytest.raises(kdn.KdnError):
        kdn.layer_norm_backward(dy, x, w, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
