"""GPU test of packed fp32 problems whose tokens are nearly all one sequence's: right, and no slower than that sequence alone."""
import pytest
import torch

from tests import linear_ref as R
from tests import test_gpu_linear as TL

pytestmark = pytest.mark.gpu


def best_us(f, turns=5):
    f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    us = []
    for _ in range(turns):
        a.record()
        f()
        b.record()
        b.synchronize()
        us.append(1e3 * a.elapsed_time(b))
    return min(us)


def test_one_long_sequence_among_single_tokens(kdn):
    """8170 tokens and 16 sequences of one, 16 heads of 128 x 256: milliseconds of work.  Against the same tokens as one dense
    sequence (128 chunks scanned once) the extra sequences cost 17 chunks in 145 and their states; a path that reads every
    earlier chunk's contribution again takes twice as long."""
    lens = [8170] + [1] * 16
    T = sum(lens)
    x = TL.make(1, 1, T, 16, 128, 256, "f32", "token", N=len(lens), grads=True)
    cu = TL.offsets(lens)
    a = (x["q"], x["k"], x["v"], x["g"])
    one, ds = x["S0"][:1].contiguous(), x["dS"][:1].contiguous()
    packed, dense = best_us(lambda: kdn.linear_forward(*a, cu_seqlens=cu, S0=x["S0"])), best_us(lambda: kdn.linear_forward(*a, S0=one))
    assert packed <= 1.4 * dense, (packed, dense)
    packed = best_us(lambda: kdn.linear_backward(*a, x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"]))
    dense = best_us(lambda: kdn.linear_backward(*a, x["do"], S0=one, dS=ds))
    assert packed <= 1.4 * dense, (packed, dense)
    kdn.last_device_error()


# around the rule's bounds: folded, and scanned
@pytest.mark.parametrize("lens,H,dk,dv", [([4990] + [1] * 11, 1, 64, 64), ([1500] + [1] * 5, 2, 128, 128), ([700, 3, 900], 2, 128, 64),
                                          ([1024] + [64, 63], 3, 32, 32), ([600] + [0] * 7, 2, 128, 256)])
def test_results_around_the_bounds(kdn, lens, H, dk, dv):
    x = TL.make(sum(lens), 1, sum(lens), H, dk, dv, "f32", "token", N=len(lens), grads=True)
    cu = TL.offsets(lens)
    o, S = kdn.linear_forward(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, S0=x["S0"])
    TL.check_forward(x, o, S, "f32", cu=cu)
    r = R.backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu=cu, S0=x["S0"], dS=x["dS"])
    out = kdn.linear_backward(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu, S0=x["S0"], dS=x["dS"])
    kdn.last_device_error()
    n = R.terms(sum(lens), dk, dv) * R.U32
    for name in ("dq", "dk", "dv", "dS0"):
        R.assert_within(out[name], r[name], n * r["mag_" + name], name)
    R.assert_within(out["dg"], r["dg"], 2 * n * r["mag_dg"], "dg")
