"""The group norm on the GPU with means far larger than the spread, every result held to what fp32
leaves of the spread.

Errors, of fp32 tensors.  In these cases a thread takes one batch of 16 values at most, or 8 tokens; what
goes over threads and slabs is fp64.  Partial sums of k values around a mean are k times as large, so a
batch's mean is off by (2 + .. + 16) / 16 roundings of it and two more, 2^-20 |mean|: delta.  x less the
mean is one rounding, so xhat is off by delta r, the same for all of a group, and by the relative error of
r, rho: half of the squares' 16 roundings and two more (2^-20), and delta^2 r^2, by which squares around a
mean that is delta away are too large.  All else follows to first order (silu' is at most 1.1, silu'' at
most 0.5), with 2^-20 of the terms for the sigmoid, single roundings and sums of 16.  A mean enters
linearly: nothing grows with its square but rho's second part.
"""
import pytest
import torch

from oracle import norm as ref
from test_norm_gpu import DEV, _gpu, _plan

pytestmark = pytest.mark.gpu

CASES = [(2, 200, 4, 64), (1, 4096, 1, 48), (3, 37, 2, 33)]
MEANS = [1000.0, -8000.0]


def inputs(case, mean):
    N, L, G, Ch = case
    g = torch.Generator().manual_seed(L)
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(x=r(N, L, G, Ch) + r(G, Ch) + mean, w=1 + 0.3 * r(G, Ch), bias=r(G, Ch), gate=None, lengths=None), r(N, L, G, Ch)


def allowed(a, dy, per_token, eps=1e-5):
    """The errors of y, dx, dw and dbias that fp32 allows, for act silu."""
    dims = (3,) if per_token else (1, 3)
    x, w, b, dy = (t.double() for t in (a["x"], a["w"], a["bias"], dy))
    mean = x.mean(dims, keepdim=True)
    r = 1 / ((x - mean).square().mean(dims, keepdim=True) + eps).sqrt()
    xh = (x - mean) * r
    delta = 2.0 ** -20 * mean.abs()
    rho = 2.0 ** -20 + (delta * r) ** 2
    e = delta * r + xh.abs() * rho
    v = xh * w + b
    s = torch.sigmoid(v)
    slope = s + v * s * (1 - s)
    y = 1.1 * w.abs() * e + 2.0 ** -20 * (v.abs() + w.abs() * xh.abs())
    d, ed = dy * slope, dy.abs() * (0.5 * w.abs() * e + 2.0 ** -20)
    D, eD = d * w, w.abs() * ed + 2.0 ** -20 * (d * w).abs()
    avg = lambda t: t.mean(dims, keepdim=True)
    a1, a2 = avg(D), avg(D * xh)
    e1, e2 = avg(eD) + 2.0 ** -20 * avg(D.abs()), avg(eD * xh.abs() + D.abs() * e) + 2.0 ** -20 * avg((D * xh).abs())
    terms = D.abs() + a1.abs() + (xh * a2).abs()
    dx = r * (eD + e1 + e * a2.abs() + xh.abs() * e2 + (rho + 2.0 ** -20) * terms)
    dw = (ed * xh.abs() + d.abs() * e + 2.0 ** -20 * (d * xh).abs()).sum((0, 1))
    return {"y": y, "dx": dx, "dw": dw, "dbias": (ed + 2.0 ** -20 * d.abs()).sum((0, 1))}


def check(got, want, tol, k):
    over = (got.detach().cpu().double() - want).abs() - (2.0 ** -24 * want.abs() + tol[k])
    assert (over <= 0).all(), (k, float(over.max()), float(tol[k].median()))


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("mean", MEANS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_means_far_larger_than_the_spread(case, mean, per_token):
    a, dy = inputs(case, mean)
    kw = dict(act="silu", per_token=per_token)
    p, tol = _plan(*case, "f32", a, **kw), allowed(a, dy, per_token)
    check(p(**_gpu(a)), ref.norm(**a, **kw)[0], tol, "y")
    want, _ = ref.norm_grad(dy, **a, **kw)
    got = p.backward(dy.to(DEV), **_gpu(a))
    for k in ("dx", "dw", "dbias"):
        check(got[k], want[k], tol, k)
