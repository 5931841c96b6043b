"""States of the gated delta rule keep fp32's digits, also in bf16 calls, and y and the gradients have
theirs where their terms cancel.

Keys are unit vectors along one axis and g is 0, so that every column of a state is a running mean of
its own, S = (1 - beta) S + beta v where its key comes up, and a sum has few terms that are not zero.

Tolerances.  A chunk takes a column from S to S + beta (v - S) in at most 8 roundings of |S| + |v| for
each time its key comes up (v - S, beta times it, the three terms that each of S, Z, U and N is held
in, N's own, the sum): 2^-21 (|S| + |v|) once a chunk, 2^-19 four times.  What is off fades by 1 - beta <= 1/2 at each
time, so in all it is twice that at most.  Two terms instead of three would be off by 2^-17.
"""
import pytest
import torch

from test_delta_gpu import DEV, HALF, TYPE, _plan

pytestmark = pytest.mark.gpu

# S, L, times that a key comes up in a chunk, tolerance
STATES = [(128, 448, 1, 2.0 ** -20), (64, 448, 1, 2.0 ** -20), (256, 640, 1, 2.0 ** -20), (16, 300, 4, 2.0 ** -18)]


def inputs(S, L, dtype, H=2, P=24):
    g = torch.Generator().manual_seed(S + L)
    t = TYPE[dtype]
    key = torch.eye(S)[torch.arange(L) % S].expand(1, 1, L, S).transpose(1, 2).contiguous()
    beta = (0.5 + 0.5 * torch.rand(1, L, H, generator=g)).to(t)
    v = torch.randn(1, L, H, P, generator=g).to(t)
    return dict(q=key.to(t), k=key.to(t), v=v, g=torch.zeros(1, L, H), beta=beta), torch.randn(1, H, P, S, generator=g)


def exact(a, s0):
    """The last state and, by element, the largest |S| + |v| on the way."""
    s, most = s0.double().clone(), s0.double().abs()
    S = s.shape[-1]
    for t in range(a["v"].shape[1]):
        j, b, v = t % S, a["beta"][0, t].double()[:, None], a["v"][0, t].double()
        most[0, :, :, j] = torch.maximum(most[0, :, :, j], s[0, :, :, j].abs() + v.abs())
        s[0, :, :, j] = s[0, :, :, j] + b * (v - s[0, :, :, j])
    return s, most


def near(got, want, most, tol):
    over = (got.detach().cpu().double() - want).abs() - tol * most
    assert (over <= 0).all(), float(((got.detach().cpu().double() - want).abs() / most).max() / tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", STATES, ids=str)
def test_states(case, dtype):
    S, L, _, tol = case
    a, s0 = inputs(S, L, dtype)
    out = torch.empty_like(s0, device=DEV)
    _plan(1, L, 2, 24, 1, S, dtype)(**{k: t.to(DEV) for k, t in a.items()}, state=s0.to(DEV), state_out=out)
    near(out, *exact(a, s0), tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", STATES, ids=str)
def test_gradients_of_states(case, dtype):
    """Without dy a state's gradient goes back through every token: a column of it times 1 - beta where its key comes
    up, which takes the same roundings of it alone."""
    S, L, _, tol = case
    a, s0 = inputs(S, L, dtype)
    last = torch.randn(s0.shape, generator=torch.Generator().manual_seed(1))
    d = {k: t.to(DEV) for k, t in a.items()}
    got = _plan(1, L, 2, 24, 1, S, dtype).backward(torch.zeros_like(d["v"]), **d, state=s0.to(DEV), dstate_out=last.to(DEV))
    want = last.double().clone()
    for t in range(L):
        want[0, :, :, t % S] *= 1 - a["beta"][0, t].double()[:, None]
    near(got["dstate"], want, last.double().abs(), tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [32, 64, 128, 256])
def test_what_is_left_of_terms_that_cancel(S, dtype):
    """y of two columns' difference, dq of two channels' difference: 2^-10 of the columns.  Without rates no token
    changes the state: both are a difference of two of its elements in 4 roundings of them, 2^-22, and one of the
    result (scale is a power of two).  Two terms would be off by 2^-17."""
    N, L, H, P = 1, 70, 1, 32
    g = torch.Generator().manual_seed(S)
    t = TYPE[dtype]
    base = 1 + torch.rand(1, H, P, 1, generator=g)
    s0 = base * (1 + 2.0 ** -10 * torch.randn(1, H, P, S, generator=g))         # columns of a channel nearly equal
    q = torch.zeros(N, L, 1, S)
    rows = torch.arange(L)
    q[0, rows, 0, rows % S], q[0, rows, 0, (rows + 1) % S] = 1, -1
    z = lambda *s: torch.zeros(*s, dtype=t, device=DEV)
    p = _plan(N, L, H, P, 1, S, dtype, scale=0.5)
    k = torch.randn(N, L, 1, S, generator=g).to(t).to(DEV)
    y = p(q.to(t).to(DEV), k, z(N, L, H, P), torch.zeros(N, L, H, device=DEV), z(N, L, H), state=s0.to(DEV))
    want = 0.5 * torch.einsum("hps,ls->lhp", s0[0].double(), q[0, :, 0].double())
    over = (y[0].cpu().double() - want).abs() - HALF[dtype] * (1 + 2 ** -8) * want.abs() - 2.0 ** -22 * s0[0].double().abs().amax(-1)
    assert (over <= 0).all(), float(over.max())
    s1 = (1 + torch.rand(1, H, 1, S, generator=g)) * (1 + 2.0 ** -10 * torch.randn(1, H, P, S, generator=g))     # rows nearly equal
    dy = torch.zeros(N, L, H, P)
    dy[0, rows, 0, rows % P], dy[0, rows, 0, (rows + 1) % P] = 1, -1
    got = p.backward(dy.to(t).to(DEV), q.to(t).to(DEV), k, z(N, L, H, P), torch.zeros(N, L, H, device=DEV), z(N, L, H),
                     state=s1.to(DEV))["dq"]
    want = 0.5 * torch.einsum("ps,lp->ls", s1[0, 0].double(), dy[0, :, 0].double())
    over = (got[0, :, 0].cpu().double() - want).abs() - HALF[dtype] * (1 + 2 ** -8) * want.abs() - 2.0 ** -22 * s1.double().abs().max()
    assert (over <= 0).all(), float(over.max())
