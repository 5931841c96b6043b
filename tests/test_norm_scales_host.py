"""The tolerances of the group norm's tests of large means are small enough to tell statistics that
lose the spread, and gradients that are none.  No GPU needed."""
import pytest
import torch

from oracle import norm as ref
from test_norm_means_gpu import CASES, MEANS, allowed, check, inputs


def _rejected(got, want, tol, k):
    with pytest.raises(AssertionError):
        check(got, want, tol, k)


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("mean", MEANS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_planted_mistakes_are_rejected(case, mean, per_token):
    a, dy = inputs(case, mean)
    kw = dict(act="silu", per_token=per_token)
    tol = allowed(a, dy, per_token)
    y, (want, _) = ref.norm(**a, **kw)[0], ref.norm_grad(dy, **a, **kw)
    check(y, y, tol, "y")
    for k in ("dx", "dw", "dbias"):
        check(want[k], want[k], tol, k)
        _rejected(torch.zeros_like(want[k]), want[k], tol, k)
        half = want[k].clone()
        half[..., ::2] = 0
        _rejected(half, want[k], tol, k)
    cut = want["dx"].clone()
    cut[:, -1] = 0
    _rejected(cut, want["dx"], tol, "dx")
    # the mean of squares less the square of the mean, in fp32
    dims = (3,) if per_token else (1, 3)
    x = a["x"]
    m = x.mean(dims, keepdim=True)
    var = (x.square().mean(dims, keepdim=True) - m.square()).clamp(min=0)
    v = (x - m) / (var + 1e-5).sqrt() * a["w"] + a["bias"]
    _rejected(v * torch.sigmoid(v), y, tol, "y")
