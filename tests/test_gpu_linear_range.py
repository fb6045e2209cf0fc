"""GPU tests of the range of linear attention's chunked forms: scores and decays whose product is ordinary although their
factors are not."""
import pytest

from tests import test_gpu_linear as TL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk", [64, 128])
def test_large_scores_under_a_decay(kdn, dtype, dk):
    """Scores of 2^76, values of 2^-70 and gradients of 2^30 with decays that sum to e^-40 over a chunk: every product of the operator's
    definition is far inside the range, so is every output."""
    x = TL.make(3 + dk, 2, 300, 2, dk, 64, dtype, "token", grads=True, state=False)
    x["q"], x["k"], x["v"] = x["q"] * 2.0 ** 38, x["k"] * 2.0 ** 38, x["v"] * 2.0 ** -70
    x["do"] = x["do"] * 2.0 ** 30
    x["g"] = x["g"].new_full(x["g"].shape, -40.0 / 128)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"])
    kdn.last_device_error()
    assert o.isfinite().all()
    TL.check_forward(x, o, S, dtype)
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"])
    assert all(t.isfinite().all() for t in out.values())
    TL.check_backward(x, out, dtype)
