"""GPU test of the two launches of layer norm's gradient: the second starts while the first still writes the shares of dweight
and dbias that it reads."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d", [(300, 128), (5000, 1024), (4000, 4096)])
def test_calls_in_a_row_on_one_workspace(kdn, n, d):
    """Whole numbers, whose sums are exact in any order: dweight and dbias of calls that follow one another on one workspace
    are each its own inputs', never the shares of the call before."""
    gen = torch.Generator().manual_seed(d)
    x = (torch.randint(0, 2, (n, d), generator=gen) * 2.0 - 1.0).cuda()
    dys = [torch.randint(-3, 4, (n, d), generator=gen).float().cuda() for _ in range(4)]
    w, mean, rstd = torch.ones(d, device="cuda"), torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    ws = torch.empty(kdn.kdn_layer_norm_backward_workspace_size(n, 1, d), dtype=torch.uint8, device="cuda")
    got = [kdn.layer_norm_backward(dys[i % 4], x, w, mean, rstd, workspace=ws) for i in range(40)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        dy = dys[i % 4]
        assert torch.equal(out["dweight"], (dy * x).sum(0)) and torch.equal(out["dbias"], dy.sum(0)), i
