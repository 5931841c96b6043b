"""How exactly the selective scan is computed, on inputs of few terms: the
tolerances are small enough to see an operand or an exponent that is held in
fewer than fp32's 24 bits.

Tolerances.  A result of type T is rounded once (half a step: 2^-8 in bf16,
2^-24 in fp32, of its value); before that it is off by c * sum |t_k| over its
terms, the sum being evaluated by the reference (oracle/seq.py).  dt is used as
it is (no softplus) and A and dt are exact, so a decay e^(A dt ..) has
  half a step of the exponent, |e| 2^-24 ln 2 < 2^-22 for |e| <= 6, and the
  exponential's own step, 2^-23: together under 2^-21.4,
and a product on its way two roundings of 2^-24.  All but two states and three
tokens are zeros, which add nothing: a sum has six terms at most, in three
matrix instructions, each off by a step (2^-23) of what it holds at most.
  one decay, one sum: 2^-21.4 + 2^-23 + 3 2^-23 < c = 2^-20
  states over four chunks: a decay (2^-21.4) and a sum (2^-23) each, then the
    product with C: 4 (2^-21.4 + 2^-23) + 2^-20 < c = 2^-18.2
  gradients: two such chains, c = 2^-17.2
An operand of two bf16 terms is off by up to 2^-18 by itself, and of 16 bits by
2^-17; cancelling sums have it all where half a step of the result is far less.
"""
import pytest
import torch

from oracle import seq

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"
# channels, states: whole 16-byte vectors in bf16 and not, few and many states
SHAPES = [(64, 8), (64, 5), (64, 128), (72, 100)]


def _near(got, want, mag, half, c, what):
    got, want, mag = got.detach().cpu().double(), want.double(), mag.double().abs()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - (half * want.abs() * (1 + 2 ** -8) + c * mag + 1e-37)
    assert (over <= 0).all(), "%s: error %.3g of the terms, %d of %d results over 2^%.1f" % (
        what, ((got - want).abs() - half * want.abs()).div(mag + 1e-37).max(), (over > 0).sum(), over.numel(),
        torch.tensor(c).log2())


def _gpu(d):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def _scan(N, L, H, P, G, S, dtype):
    from convolution_forward_implicit_amd import SelectiveScan
    return SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype, softplus=False)


def _two_states(g, S, *lead):
    """Values in two of S states, zeros in the others."""
    v = torch.zeros(*lead, S)
    v[..., [S // 3, S - 1]] = torch.randn(*lead, 2, generator=g)
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_a_state_enters_y_with_all_its_bits(P, S, dtype):
    """y = e^(A dt) (h_1 C_1 + h_2 C_2) where the two products cancel to the last bits of h."""
    g = torch.Generator().manual_seed(1)
    N, H, t = 8, 16, TYPE[dtype]
    C = _two_states(g, S, N, 1, 1).to(t)
    a, b = S // 3, S - 1
    h = torch.zeros(N, H, P, S)
    h[..., a] = torch.randn(N, H, P, generator=g)
    h[..., b] = -(h[..., a].double() * C[:, :, :, a].double() / C[:, :, :, b].double()).float()
    v = dict(x=torch.zeros(N, 1, H, P, dtype=t), dt=torch.full((N, 1, H), 0.25, dtype=t), A=torch.full((H,), -0.5),
             B=torch.ones(N, 1, 1, S, dtype=t), C=C, state=h)
    y, _ = seq.scan(**v, softplus=False)
    mag, _ = seq.scan(**v, softplus=False, magnitude=True)
    assert (y.abs() < 2.0 ** -22 * mag).all()
    _near(_scan(N, 1, H, P, 1, S, dtype)(**_gpu(v)), y, mag, HALF[dtype], 2.0 ** -20, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_tokens_enter_y_with_all_bits_of_their_weights(P, S, dtype):
    """y = sum_j (C_i . B_j) e^(c_i - c_j) dt_j x_j over three tokens: of many results some nearly cancel."""
    g = torch.Generator().manual_seed(2)
    N, L, H, t = 48, 3, 32, TYPE[dtype]
    v = dict(x=torch.randn(N, L, H, P, generator=g).to(t), dt=(0.1 + torch.rand(N, L, H, generator=g)).to(t),
             A=-torch.rand(H, generator=g) - 0.1, B=_two_states(g, S, N, L, 1).to(t), C=_two_states(g, S, N, L, 1).to(t),
             D=torch.randn(H, generator=g))
    y, _ = seq.scan(**v, softplus=False)
    mag, _ = seq.scan(**v, softplus=False, magnitude=True)
    assert (y.abs() < 2.0 ** -12 * mag).sum() > 10
    _near(_scan(N, L, H, P, 1, S, dtype)(**_gpu(v)), y, mag, HALF[dtype], 2.0 ** -20, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_tokens_behind_one_that_clears_the_state(P, S, dtype):
    """A step of 2^12 forgets all before it; the decays between the tokens behind it are as exact as without it."""
    g = torch.Generator().manual_seed(3)
    N, L, H, t = 4, 6, 8, TYPE[dtype]
    dt = torch.randint(1, 32, (N, L, H), generator=g) / 64
    dt[:, 1] = 4096.0
    v = dict(x=torch.randn(N, L, H, P, generator=g).to(t), dt=dt.to(t), A=-torch.rand(H, generator=g) - 1,
             B=_two_states(g, S, N, L, 1).to(t), C=_two_states(g, S, N, L, 1).to(t))
    v["x"][:, 1:3] = 0      # of three tokens, one before the step and two behind it
    v["x"][:, 5] = 0
    y, last = seq.scan(**v, softplus=False)
    mag, top = seq.scan(**v, softplus=False, magnitude=True)
    out = torch.empty(N, H, P, S, device=DEV)
    _near(_scan(N, L, H, P, 1, S, dtype)(**_gpu(v), state_out=out), y, mag, HALF[dtype], 2.0 ** -20, "y")
    _near(out, last, top, HALF["f32"], 2.0 ** -20, "state_out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_one_large_pair_leaves_the_other_tokens_gradients_alone(P, S, dtype):
    """Token 10's output meets token 9's input 2^30 times as strongly as any other pair, in a channel of its own.  Only
    the decay of token 10 lies between them; the others' ddt have no such term and must not be rounded as if they had.
    A term A W of ddt is off by 2^-21 (decay, products), a sum over 30 tokens in fp32 by 30 steps of 2^-24: c = 2^-18
    of the terms of each token alone."""
    g = torch.Generator().manual_seed(7)
    N, L, H, t = 2, 30, 3, TYPE[dtype]
    v = dict(x=torch.zeros(N, L, H, P), dt=torch.full((N, L, H), 2.0 ** -6), A=-torch.rand(H, generator=g) - 0.5,
             B=torch.zeros(N, L, 1, S), C=torch.zeros(N, L, 1, S))
    v["B"][..., S // 2] = v["C"][..., S // 2] = 1
    dy = torch.zeros(N, L, H, P)
    v["x"][..., P - 1], dy[..., P - 1] = torch.randn(N, L, H, generator=g), torch.randn(N, L, H, generator=g)
    v["x"][:, 9, :, 0], dy[:, 10, :, 0] = 2.0 ** 18, 2.0 ** 18
    for k in ("x", "dt", "B", "C"):
        v[k] = v[k].to(t)
    dy = dy.to(t)
    want = seq.scan_grad(dy, **v, softplus=False)
    mag = seq.scan_grad(dy, **v, softplus=False, magnitude=True)
    got = _scan(N, L, H, P, 1, S, dtype).backward(dy.to(DEV), **_gpu(v))
    _near(got["ddt"], want["ddt"], mag["ddt"], HALF[dtype], 2.0 ** -18, "ddt")


@pytest.mark.parametrize("step", [2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_a_step_of_any_size_clears_the_state(P, S, dtype, step):
    """As above with steps past the digits of fp64 sums, on tokens without an input; the gradients of what follows too."""
    g = torch.Generator().manual_seed(8)
    N, L, H, t = 4, 6, 8, TYPE[dtype]
    dt = torch.randint(1, 32, (N, L, H), generator=g) / 64
    dt[:, 1] = step
    v = dict(x=torch.randn(N, L, H, P, generator=g), dt=dt.to(t), A=-torch.rand(H, generator=g) - 1,
             B=_two_states(g, S, N, L, 1).to(t), C=_two_states(g, S, N, L, 1).to(t), state=_two_states(g, S, N, H, P))
    v["x"][:, 1:3] = 0
    v["x"][:, 5] = 0
    v["x"] = v["x"].to(t)
    y, last = seq.scan(**v, softplus=False)
    mag, top = seq.scan(**v, softplus=False, magnitude=True)
    out = torch.empty(N, H, P, S, device=DEV)
    p = _scan(N, L, H, P, 1, S, dtype)
    _near(p(**_gpu(v), state_out=out), y, mag, HALF[dtype], 2.0 ** -20, "y")
    _near(out, last, top, HALF["f32"], 2.0 ** -20, "state_out")
    dy = torch.zeros(N, L, H, P)
    dy[:, 4:, :, P // 3] = torch.randn(N, 2, H, generator=g)
    dy = dy.to(t)
    want = seq.scan_grad(dy, **v, softplus=False)
    mag = seq.scan_grad(dy, **v, softplus=False, magnitude=True)
    got = p.backward(dy.to(DEV), **_gpu(v))
    # sums over eight heads of one channel each: as a gradient's two chains, and eight steps of 2^-24
    for k in ("dx", "dB", "dC", "dstate"):
        _near(got[k], want[k], mag[k], HALF["f32" if k == "dstate" else dtype], 2.0 ** -17, k)


@pytest.mark.parametrize("step", [4096.0, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,S", SHAPES)
def test_a_clearing_step_has_no_gradient_by_its_decay(P, S, dtype, step):
    """Its decay is zero, and so is the gradient of A dt there, however large dt makes what is left of a sum.  The inputs
    differ by up to 2^16 in size, so that fp64 sums of them leave something.  c = 2^-17.2 as above and 30 steps of
    2^-24 for the sums over the tokens: 2^-16."""
    g = torch.Generator().manual_seed(9)
    N, L, H, t = 3, 30, 4, TYPE[dtype]
    dt = torch.randint(1, 32, (N, L, H), generator=g) / 64
    dt[:, 2] = step
    v = dict(x=torch.zeros(N, L, H, P), dt=dt.to(t), A=-torch.rand(H, generator=g) - 1, B=_two_states(g, S, N, L, 1).to(t),
             C=_two_states(g, S, N, L, 1).to(t), state=_two_states(g, S, N, H, P))
    dy = torch.zeros(N, L, H, P)
    wide = lambda: torch.randn(N, L, H, generator=g) * 2.0 ** torch.randint(-8, 9, (N, L, H), generator=g)
    v["x"][..., P // 3], dy[..., P // 3] = wide(), wide()
    v["x"][:, 2] = 0
    v["x"], dy = v["x"].to(t), dy.to(t)
    want = seq.scan_grad(dy, **v, softplus=False)
    mag = seq.scan_grad(dy, **v, softplus=False, magnitude=True)
    got = _scan(N, L, H, P, 1, S, dtype).backward(dy.to(DEV), **_gpu(v))
    _near(got["ddt"], want["ddt"], mag["ddt"], HALF[dtype], 2.0 ** -16, "ddt")
    _near(got["dA"], want["dA"], mag["dA"], HALF["f32"], 2.0 ** -16, "dA")
