"""The gradient of the gated delta rule on the GPU against the double-precision reference, every
gradient with the scale of its own errors and no wider one: dg's is that of the terms that cross the
token's decay.  Cases and inputs are those of the other tests of the gradient.

Tolerance: a rounding of the result, and 2^-13 of the scale, as derived there.
"""
import pytest
import torch

from oracle import delta as ref
from test_delta_gpu import CASES, CG, DEV, HALF, TYPE, _case, _gpu, _near, _plan

pytestmark = pytest.mark.gpu

ALL = CASES + [(1, 70, 12, 16, 1, 24, True, None), (2, 65, 48, 40, 4, 24, True, "most"), (5, 66, 27, 33, 9, 128, True, "zero"),
               (1, 260, 2, 48, 2, 64, True, None), (1, 260, 4, 130, 2, 128, True, None), (2, 200, 3, 16, 1, 256, True, "most")]


def check(got, want, mag, dtype, only=None):
    for k, t in got.items():
        if t is not None and only in (None, k):
            _near(t, want[k], mag[k], HALF["f32" if k in ("dg", "dstate") else dtype], CG, k)


def inputs(case, dtype, keys):
    N, L, H, P, G, S, state, lengths = case
    a, s0, n = _case(N, L, H, P, G, S, dtype, state, lengths, 23 + L, keys)
    g = torch.Generator().manual_seed(L)
    dy = torch.randn(N, L, H, P, generator=g).to(TYPE[dtype])
    return dy, dict(a, scale=S ** -0.5, state=s0, lengths=n, dstate_out=torch.randn(N, H, P, S, generator=g) if state else None)


@pytest.mark.parametrize("keys", ["random", "same", "few"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ALL, ids=str)
def test_gradient(case, dtype, keys):
    dy, a = inputs(case, dtype, keys)
    want, mag = ref.delta_grad(dy, **a)
    scale = a.pop("scale")
    check(_plan(*case[:6], dtype, scale=scale).backward(dy.to(DEV), **_gpu(a)), want, mag, dtype)
