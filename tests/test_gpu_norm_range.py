"""GPU test of layer norm's gradient where (0 - mean) rstd leaves fp32's range: a width that leaves places of a row's threads
without an element must not see it."""
import pytest
import torch

from tests import linear_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [24, 33, 72, 100, 200, 510, 600, 1001, 1500, 3001, 5000, 9000])
def test_a_constant_row_of_large_values(kdn, dtype, d):
    """x = mean = 2^105 and rstd = 2^25 (an eps of 2^-50): xh is 0, dx = rstd (u - mean u) and dweight is 0."""
    x = torch.full((5, d), 2.0 ** 105, device="cuda", dtype=dtype)
    gen = torch.Generator().manual_seed(d)
    dy = torch.randn((5, d), generator=gen).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=gen)).cuda()
    mean, rstd = torch.full((5,), 2.0 ** 105, device="cuda"), torch.full((5,), 2.0 ** 25, device="cuda")
    out = kdn.layer_norm_backward(dy, x, w, mean, rstd)
    u = R.f64(dy) * R.f64(w)
    want = 2.0 ** 25 * (u - u.mean(-1, keepdim=True))
    bound = 2.0 ** 25 * ((d + 16) * R.U32 * u.abs().mean(-1, keepdim=True) + 4 * R.U32 * u.abs())
    if dtype == torch.bfloat16:
        bound = bound * (1 + R.U16) + R.U16 * want.abs()
    R.assert_within(out["dx"].float(), want, bound, "dx")
    assert (out["dweight"] == 0).all()
    R.assert_within(out["dbias"], R.f64(dy).sum(0), 21 * R.U32 * R.f64(dy).abs().sum(0), "dbias")
