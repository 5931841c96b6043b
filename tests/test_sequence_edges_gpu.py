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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [16, 21])
def test_an_empty_sequence_adds_nothing_to_the_convolutions_gradient(C, dtype):
    """... whatever its state holds: no token reads it, and it is handed on."""
    g = torch.Generator().manual_seed(5)
    N, L, F, t = 3, 20, 4, TYPE[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(t)
    v = dict(x=r(N, L, C), w=r(C, F), bias=r(C), state=r(N, F - 1, C))
    dy, dlast = r(N, L, C), r(N, F - 1, C)
    n = torch.tensor([20, 0, 7], dtype=torch.int32)
    bad = dict(v, state=v["state"].clone())
    bad["state"][1] = float("nan")
    p = _conv(N, L, C, F, dtype, has_bias=True, silu=True)
    back = lambda a: p.backward(dy.to(DEV), **_gpu(a), lengths=n.to(DEV), dstate_out=dlast.to(DEV))
    want, got = back(v), back(bad)
    for k in ("dx", "dw", "dbias", "dstate"):
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(got["dstate"][1].cpu(), dlast[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [16, 21])
def test_a_last_token_reaches_only_the_tap_that_reads_it(C, dtype):
    """Without an activation: NaN in a sequence's last token meets w[F-1] alone, the tokens behind it are no terms."""
    g = torch.Generator().manual_seed(6)
    N, L, F, t = 2, 40, 4, TYPE[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(t)
    v = dict(x=r(N, L, C), w=r(C, F))
    dy = r(N, L, C).to(DEV)
    n = torch.tensor([18, 40], dtype=torch.int32, device=DEV)
    bad = dict(v, x=v["x"].clone())
    bad["x"][0, 17] = float("nan")
    p = _conv(N, L, C, F, dtype)
    want, got = p.backward(dy, **_gpu(v), lengths=n), p.backward(dy, **_gpu(bad), lengths=n)
    assert torch.equal(got["dx"], want["dx"])
    assert torch.equal(got["dw"][:, :F - 1], want["dw"][:, :F - 1]) and torch.isnan(got["dw"][:, F - 1]).all()


def test_the_widest_heads_take_a_state():
    """65536 channels of 128 states, 32 MiB a head: one token from a state, as a prompt, a step and a gradient, against
    the definitions in 64 bits on the GPU.  Sums of up to 128 terms and the decay, in fp32: 140 steps of 2^-24 < 2^-16
    of the terms; dB and dC over 65536 channels in a chain of 16-channel sums: under 2^13 steps of 2^-24, 2^-11."""
    H, P, S = 2, 65536, 128
    g = torch.Generator(device=DEV).manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, dt, A, B, C, D, h, dy = (r(1, 1, H, P), r(1, 1, H).abs() * 0.1, -r(H).abs(), r(1, 1, 1, S), r(1, 1, 1, S), r(H),
                                r(1, H, P, S), r(1, 1, H, P))
    p = _scan(1, 1, H, P, 1, S, "f32", softplus=False)
    last = torch.empty_like(h)
    y = p(x, dt, A, B, C, D, state=h, state_out=last)
    got = p.backward(dy, x, dt, A, B, C, D, state=h)
    one = h.clone()
    y1 = p.step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], one, D)
    x, dt, A, B, C, D, dy = (v.double() for v in (x[0, 0], dt[0, 0], A, B[0, 0, 0], C[0, 0, 0], D, dy[0, 0]))
    h = h[0].double()
    a = torch.exp(A * dt)[:, None]

    def near(got, want, mag, c, what):
        assert ((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + c * mag).all(), what

    xd = dt[:, None] * x
    new, top = a[..., None] * h + xd[..., None] * B, a[..., None] * h.abs() + xd.abs()[..., None] * B.abs()
    for state, out in ((last, y[0, 0]), (one, y1[0])):
        near(state[0], new, top, 2.0 ** -16, "state")
        near(out, new @ C + D[:, None] * x, top @ C.abs() + (D[:, None] * x).abs(), 2.0 ** -16, "y")
    into = dy * (C @ B)
    near(got["dx"][0, 0], dt[:, None] * into + D[:, None] * dy,
         dt[:, None] * dy.abs() * (C.abs() @ B.abs()) + (D[:, None] * dy).abs(), 2.0 ** -16, "dx")
    near(got["dstate"][0], a[..., None] * dy[..., None] * C, a[..., None] * dy.abs()[..., None] * C.abs(), 2.0 ** -16, "dstate")
    near(got["dC"][0, 0, 0], (dy[..., None] * new).sum((0, 1)), (dy.abs()[..., None] * top).sum((0, 1)), 2.0 ** -11, "dC")
    near(got["dB"][0, 0, 0], (xd * dy).sum() * C, (xd * dy).abs().sum() * C.abs(), 2.0 ** -11, "dB")
