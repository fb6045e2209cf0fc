"""Outputs that share some bytes with an input, another output or the workspace are refused before anything is launched (the
fake addresses are never dereferenced)."""
import pytest

from kalman_delta_rule_b200 import binding as B

BASE = 0x7F0000000000
STEP = 1 << 24                     # further apart than any of the arrays is long


@pytest.fixture(scope="module", autouse=True)
def lib():
    from kalman_delta_rule_b200 import build
    build.build()
    return B.load()


def overlapping(sizes, outs, call):
    """Every pair with an output in it, one array beginning 16 bytes before the other one's end."""
    for o in outs:
        for other in range(len(sizes)):
            if other == o:
                continue
            for first, second in ((o, other), (other, o)):
                at = [BASE + i * STEP for i in range(len(sizes))]
                at[second] = (at[first] + sizes[first] - 16) // 256 * 256 if sizes[first] > 256 else at[first]
                if at[second] < at[first]:
                    at[second] = at[first]
                assert call(at) == B.KDN_ERR_INVALID_ARG, (o, other, first)


@pytest.mark.parametrize("dtype,e", [(B.KDN_DTYPE_F32, 4), (B.KDN_DTYPE_BF16, 2)])
@pytest.mark.parametrize("decay", [B.KDN_DECAY_TOKEN, B.KDN_DECAY_HEAD])
def test_linear(dtype, e, decay):
    p = B.kdn_linear_problem_t(2, 200, 4, 64, 32, None, 2, dtype, 1.0, decay)
    rows = 2 * 200 * 4
    qk, vo, g, state = rows * 64 * e, rows * 32 * e, 4 * (rows if decay == B.KDN_DECAY_TOKEN else 4), 2 * 4 * 64 * 32 * 4
    need = B.kdn_linear_workspace_size(p)
    overlapping([qk, qk, vo, g, state, vo, state, need], (5, 6, 7), lambda a: B.kdn_linear_forward(p, *a, need, None))
    need = B.kdn_linear_backward_workspace_size(p)
    overlapping([qk, qk, vo, g, state, vo, state, qk, qk, vo, g, state, need], (7, 8, 9, 10, 11, 12),
                lambda a: B.kdn_linear_backward(p, *a, need, None))
    overlapping([qk, qk, vo, g, state, vo], (4, 5),
                lambda a: B.kdn_linear_decode_tokens(2, 200, 4, 64, 32, dtype, 1.0, decay, *a, None))


@pytest.mark.parametrize("dtype,e", [(B.KDN_DTYPE_F32, 4), (B.KDN_DTYPE_BF16, 2)])
def test_norm(dtype, e):
    n, G, d = 300, 4, 96
    x, par, stat = n * G * d * e, G * d * 4, n * G * 4
    overlapping([x, par, par, x, stat, stat], (3, 4, 5), lambda a: B.kdn_layer_norm(n, G, d, dtype, 1e-5, *a, None))
    need = B.kdn_layer_norm_backward_workspace_size(n, G, d)
    overlapping([x, x, par, stat, stat, x, par, par, need], (5, 6, 7, 8),
                lambda a: B.kdn_layer_norm_backward(n, G, d, dtype, *a, need, None))
