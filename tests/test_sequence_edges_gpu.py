"""Corners of the sequence operators on the GPU: what lies behind a sequence
while its data are not finite, plans that only large problems choose, every form
of the convolution's step."""
import pytest
import torch

from oracle import seq

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


def _gpu(d):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def _scan(N, L, H, P, G, S, dtype, **kw):
    from convolution_forward_implicit_amd import SelectiveScan
    return SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype, **kw)


def _conv(N, L, C, F, dtype, **kw):
    from convolution_forward_implicit_amd import CausalConv
    return CausalConv({"N": N, "L": L, "C": C, "F": F}, dtype, **kw)


def _scan_case(N, L, H, P, G, S, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = TYPE[dtype]
    a = dict(x=r(N, L, H, P).to(t), dt=r(N, L, H).to(t), A=-torch.rand(H, generator=g) * 4 - 0.1, B=r(N, L, G, S).to(t),
             C=r(N, L, G, S).to(t), D=r(H), dt_bias=r(H) - 2, state=r(N, H, P, S))
    return a, r(N, L, H, P).to(t), r(N, H, P, S), g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(4, 32, 1, 32), (4, 32, 4, 32), (2, 20, 1, 20), (2, 72, 2, 128)], ids=str)
def test_rows_behind_a_sequence_are_zeros_whatever_comes_before(dims, dtype):
    """NaN and infinities in the state, its gradient and the last token: rows behind the length stay zeros and the
    other sequence keeps its bits."""
    H, P, G, S = dims
    N, L = 3, 150
    a, dy, dlast, _ = _scan_case(N, L, H, P, G, S, dtype, 3)
    n = torch.tensor([100, 130, 5], dtype=torch.int32)
    p = _scan(N, L, H, P, G, S, dtype)
    run = lambda v: p(**_gpu(v), lengths=n.to(DEV))
    back = lambda v, u: p.backward(dy.to(DEV), **_gpu(v), lengths=n.to(DEV), dstate_out=u.to(DEV))
    y, grads = run(a), back(a, dlast)
    bad, u = dict(a, x=a["x"].clone(), state=a["state"].clone()), dlast.clone()
    bad["state"][0, :, 1], bad["state"][0, :, 2], u[0, :, 3] = float("nan"), float("inf"), float("-inf")
    bad["x"][2, 4, 0, 0] = float("inf")
    got, gbad = run(bad), back(bad, u)
    for i in (0, 2):
        assert (got[i, n[i]:] == 0).all(), i
        for k in ("dx", "ddt", "dB", "dC"):
            assert (gbad[k][i, n[i]:] == 0).all(), (k, i)
    assert torch.equal(got[1], y[1])
    for k in ("dx", "ddt", "dB", "dC", "dstate"):
        assert torch.equal(gbad[k][1], grads[k][1]), k
