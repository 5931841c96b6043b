"""The gated delta rule on the GPU against the double-precision reference
(oracle/delta.py): prompts and steps over the sizes where a tile or a chunk ends,
ragged and strided batches, keys that repeat, decays that clear the state.

Tolerances.  A result of type T is rounded once: half a step, 2^-8 (bf16) or
2^-24 (fp32) of its value.  Before that an error is at most c times the scale that
the reference gives (norms of what the tokens add): operands computed on the way
are off by 2^-16 at most (two bf16 terms; the kernels have three, 2^-23); sums over 256 keys, 64 tokens and the chunk's triangular system
add (256 + 64 + 64) 2^-24 < 2^-15; a decay is the exponential of a rounded
difference, 2^-24 of itself up to 2^7, two of them 2^-16.  Together under 2^-14.
"""
import pytest
import torch

from oracle import delta as ref

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"
C = 2.0 ** -14


def _near(got, want, mag, half, c, what):
    got, want, mag = got.detach().cpu().double(), want.double(), mag.double().abs().expand(want.shape)
    assert torch.isfinite(got).all(), what
    if not want.numel():
        return
    over = (got - want).abs() - (half * want.abs() * (1 + 2 ** -8) + c * mag + 1e-37)
    assert (over <= 0).all(), "%s: %g over at %r (got %g, want %g)" % (
        what, over.max(), tuple(torch.nonzero(over == over.max())[0].tolist()),
        got.flatten()[over.argmax()], want.flatten()[over.argmax()])


def _gpu(d):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def _lengths(kind, N, L, g):
    if kind is None:
        return None
    n = torch.randint(0, L + 1, (N,), generator=g, dtype=torch.int32)
    n[0] = {"zero": 0, "one": min(1, L), "most": max(0, L - 1)}[kind]
    return n


def _case(N, L, H, P, G, S, dtype, state, lengths, seed, keys="random"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = TYPE[dtype]
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()
    k = unit(r(N, L, G, S))
    if keys == "same":
        k = k[:, :1].expand(N, L, G, S)
    elif keys == "few":         # three keys in turn, and their opposites
        k = (k[:, :3] if L >= 3 else k).repeat(1, -(-L // 3), 1, 1)[:, :L] * (1 - 2 * (torch.arange(L) % 2))[None, :, None, None]
    a = dict(q=unit(r(N, L, G, S)).to(t), k=k.to(t).contiguous(), v=r(N, L, H, P).to(t), g=-r(N, L, H).abs() * 0.2,
             beta=(torch.rand(N, L, H, generator=g) * (1.9 if keys != "random" else 1)).to(t))
    return a, r(N, H, P, S) if state else None, _lengths(lengths, N, L, g)


def _plan(N, L, H, P, G, S, dtype, **kw):
    from convolution_forward_implicit_amd import DeltaRule
    return DeltaRule({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype, **kw)


CASES = [(1, 1, 1, 1, 1, 1, True, None), (2, 64, 2, 64, 1, 128, False, None), (2, 65, 4, 64, 2, 128, True, "most"),
         (1, 130, 3, 40, 3, 24, True, None), (3, 33, 2, 130, 1, 17, True, "zero"), (1, 200, 2, 16, 1, 64, False, None),
         (2, 63, 2, 128, 2, 100, True, "one"), (1, 300, 1, 64, 1, 256, True, None), (4, 70, 16, 8, 4, 16, True, "most"),
         (2, 0, 2, 16, 1, 16, True, None), (0, 9, 2, 16, 1, 16, False, None), (2, 192, 6, 24, 1, 33, True, "zero"),
         (1, 129, 2, 24, 1, 200, False, None)]


@pytest.mark.parametrize("keys", ["random", "same", "few"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompt(case, dtype, keys):
    N, L, H, P, G, S, state, lengths = case
    a, s0, n = _case(N, L, H, P, G, S, dtype, state, lengths, 17 + L, keys)
    p = _plan(N, L, H, P, G, S, dtype)
    y, last, my, ms = ref.delta(**a, scale=S ** -0.5, state=s0, lengths=n)
    out = torch.full((N, H, P, S), 7.0, device=DEV)
    got = p(**_gpu(a), state=None if s0 is None else s0.to(DEV), lengths=None if n is None else n.to(DEV), state_out=out)
    _near(got, y, my, HALF[dtype], C, "y")
    _near(out, last, ms, HALF["f32"], C, "state_out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (3, 4, 64, 2, 128), (2, 3, 40, 1, 24), (2, 2, 130, 2, 101),
                                  (5, 2, 33, 1, 8), (2, 4, 96, 4, 256)], ids=str)
def test_step(case, dtype):
    N, H, P, G, S = case
    a, s0, _ = _case(N, 1, H, P, G, S, dtype, True, None, 31)
    p = _plan(N, 1, H, P, G, S, dtype, scale=0.7)
    one = {k: v[:, 0] for k, v in a.items()}
    y, last, my, ms = ref.step(**one, scale=0.7, state=s0)
    state = s0.to(DEV)
    got = p.step(**_gpu(one), state=state)
    _near(got, y, my, HALF[dtype], C, "y")
    _near(state, last, ms, HALF["f32"], C, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_column_ranges(dtype):
    """The inputs as columns of one tensor, aligned and not, y into columns of another."""
    N, L, H, P, G, S = 2, 70, 4, 32, 2, 40
    a, _, _ = _case(N, L, H, P, G, S, dtype, False, None, 7)
    p = _plan(N, L, H, P, G, S, dtype)
    v = _gpu(a)
    want = p(**v)
    for extra in (0, 3):
        parts = [v[k].flatten(2) for k in ("q", "k", "v", "beta")]
        u = torch.cat([torch.zeros(N, L, extra, dtype=TYPE[dtype], device=DEV)] + parts, -1).contiguous()
        q, k, x, b = u[..., extra:].split([t.shape[2] for t in parts], -1)
        wide = torch.full((N, L, H * P + 8 + extra), 3.0, dtype=TYPE[dtype], device=DEV)
        g = torch.cat([v["g"], v["g"]], -1)[..., H:]
        p(q.unflatten(-1, (G, S)), k.unflatten(-1, (G, S)), x.unflatten(-1, (H, P)), g, b,
          out=wide[..., 8:8 + H * P].unflatten(-1, (H, P)))
        assert torch.equal(wide[..., 8:8 + H * P], want.flatten(2))
        assert (wide[..., :8] == 3).all() and (wide[..., 8 + H * P:] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_behind_a_sequence_is_read(dtype):
    """NaN and infinities in the rows behind the lengths reach nothing; lengths out of range are the nearer end."""
    N, L, H, P, G, S = 4, 130, 2, 24, 1, 20
    n = torch.tensor([130, 0, 37, 64], dtype=torch.int32)
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 9)
    bad = {k: v.clone() for k, v in a.items()}
    for i in range(N):
        for j, k in enumerate(bad):
            bad[k][i, n[i]:] = float("nan") if j % 2 else float("inf")
    p = _plan(N, L, H, P, G, S, dtype)
    one, two = torch.empty(N, H, P, S, device=DEV), torch.empty(N, H, P, S, device=DEV)
    y = p(**_gpu(a), state=s0.to(DEV), lengths=n.to(DEV), state_out=one)
    far = torch.tensor([999, -5, 37, 64], dtype=torch.int32)
    z = p(**_gpu(bad), state=s0.to(DEV), lengths=far.to(DEV), state_out=two)
    assert torch.equal(y, z) and torch.equal(one, two)
    assert torch.equal(one[1].cpu(), s0[1]) and (y[1] == 0).all() and (y[2, 37:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_that_clear_the_state(dtype):
    """A decay of minus infinity, and huge ones: what lies behind depends on nothing in front, and keeps its digits."""
    N, L, H, P, G, S = 1, 150, 3, 16, 1, 32
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 3)
    a["g"][:, 70, 0], a["g"][:, 70, 1], a["g"][:, :, 2] = -float("inf"), -1e30, -50.0
    y, last, my, ms = ref.delta(**a, scale=S ** -0.5, state=s0)
    p = _plan(N, L, H, P, G, S, dtype)
    out = torch.empty(N, H, P, S, device=DEV)
    got = p(**_gpu(a), state=s0.to(DEV), state_out=out)
    _near(got, y, my, HALF[dtype], C, "y")
    _near(out, last, ms, HALF["f32"], C, "state_out")
    tail = p.__class__(dict(p.problem, L=L - 70), dtype)({k: v[:, 70:].contiguous() for k, v in _gpu(a).items()}["q"],
                                                         *(_gpu(a)[k][:, 70:].contiguous() for k in ("k", "v", "g", "beta")))
    ty, _, tmy, _ = ref.delta(**{k: v[:, 70:] for k, v in a.items()}, scale=S ** -0.5)
    _near(tail[:, :, :2], ty[:, :, :2], tmy[:, :, :2], HALF[dtype], C, "behind")
    _near(got[:, 70:, :2], ty[:, :, :2], tmy[:, :, :2], HALF[dtype], C, "behind in place")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens_is_the_whole_sequence(dtype):
    N, L, H, P, G, S = 2, 75, 4, 40, 2, 48
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 5)
    v = _gpu(a)
    whole = torch.empty(N, H, P, S, device=DEV)
    y = _plan(N, L, H, P, G, S, dtype)(**v, state=s0.to(DEV), state_out=whole)
    state = torch.empty(N, H, P, S, device=DEV)
    cut = lambda lo, hi: {k: t[:, lo:hi].contiguous() for k, t in v.items()}
    ys = [_plan(N, 70, H, P, G, S, dtype)(**cut(0, 70), state=s0.to(DEV), state_out=state)]
    p = _plan(N, 1, H, P, G, S, dtype)
    for t in range(70, L):
        ys.append(p.step(**{k: x[:, t] for k, x in v.items()}, state=state)[:, None])
    want, last, my, ms = ref.delta(**a, scale=S ** -0.5, state=s0)
    _near(torch.cat(ys, 1), want, my, HALF[dtype], C, "y")
    _near(y, want, my, HALF[dtype], C, "whole y")
    _near(state, last, ms, HALF["f32"], C, "state")


# ---- the gradient ----------------------------------------------------------------
# It chains two products of what the forward pass and the pass behind it leave: twice the
# forward's error of terms that are products of both scales.  A decay's gradient sums, over
# the chunk, terms of the tokens on both sides: its scale is taken from the 127 tokens around.
CG = 2.0 ** -13


def _around(v):
    """Sums over the 127 tokens around each, [N, L, H]."""
    if v.shape[1] == 0:
        return v
    c = torch.nn.functional.pad(v.cumsum(1), (0, 0, 1, 0))
    t = torch.arange(v.shape[1])
    return c[:, (t + 64).clamp(max=v.shape[1])] - c[:, (t - 63).clamp(min=0)]


def _check_gradient(got, want, mag, dtype, what=""):
    mag = dict(mag, dg=mag["dg"] + _around(mag["dbeta"]))
    for k, t in got.items():
        if t is not None:
            _near(t, want[k], mag[k], HALF["f32" if k in ("dg", "dstate") else dtype], CG, what + k)


@pytest.mark.parametrize("keys", ["random", "same", "few"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES + [(1, 70, 12, 16, 1, 24, True, None)], ids=str)
def test_gradient(case, dtype, keys):
    N, L, H, P, G, S, state, lengths = case
    a, s0, n = _case(N, L, H, P, G, S, dtype, state, lengths, 23 + L, keys)
    g = torch.Generator().manual_seed(L)
    dy = torch.randn(N, L, H, P, generator=g).to(TYPE[dtype])
    dlast = torch.randn(N, H, P, S, generator=g) if state else None
    p = _plan(N, L, H, P, G, S, dtype)
    want, mag = ref.delta_grad(dy, **a, scale=S ** -0.5, state=s0, lengths=n, dstate_out=dlast)
    put = lambda t: None if t is None else t.to(DEV)
    got = p.backward(dy.to(DEV), **_gpu(a), state=put(s0), lengths=put(n), dstate_out=put(dlast))
    assert (got["dstate"] is not None) == state
    _check_gradient(got, want, mag, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_in_column_ranges_and_behind_lengths(dtype):
    """dq, dk and dv into columns of one tensor, odd ones too; NaN behind the lengths reaches nothing."""
    N, L, H, P, G, S = 3, 130, 4, 24, 2, 20
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 9)
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(N, L, H, P, generator=g).to(TYPE[dtype])
    n = torch.tensor([130, 0, 37], dtype=torch.int32)
    p = _plan(N, L, H, P, G, S, dtype)
    kw = dict(state=s0.to(DEV), lengths=n.to(DEV))
    want = p.backward(dy.to(DEV), **_gpu(a), **kw)
    for i in range(N):
        for k in a:
            a[k][i, n[i]:] = float("nan")
        dy[i, n[i]:] = float("nan")
        for k in ("dq", "dk", "dv", "dg", "dbeta"):
            assert (want[k][i, n[i]:] == 0).all(), k
    width = 2 * G * S + H * P
    for extra in (0, 3):
        u = torch.full((N, L, width + 2 * extra), 5.0, dtype=TYPE[dtype], device=DEV)
        q, k, v = u[..., extra:extra + width].split([G * S, G * S, H * P], -1)
        out = {"dq": q.unflatten(-1, (G, S)), "dk": k.unflatten(-1, (G, S)), "dv": v.unflatten(-1, (H, P))}
        got = p.backward(dy.to(DEV), **_gpu(a), **kw, out=out)
        for name, t in want.items():
            assert torch.equal(got[name], t), name
        assert (u[..., :extra] == 5).all() and (u[..., extra + width:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_decays_that_clear_the_state(dtype):
    """A decay of zero has no gradient and lets none through."""
    N, L, H, P, G, S = 1, 150, 3, 16, 1, 32
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 3)
    a["g"][:, 70, 0], a["g"][:, 70, 1], a["g"][:, :, 2] = -float("inf"), -1e30, -50.0
    dy = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(2)).to(TYPE[dtype])
    dlast = torch.randn(N, H, P, S, generator=torch.Generator().manual_seed(3))
    want, mag = ref.delta_grad(dy, **a, scale=S ** -0.5, state=s0, dstate_out=dlast)
    got = _plan(N, L, H, P, G, S, dtype).backward(dy.to(DEV), **_gpu(a), state=s0.to(DEV), dstate_out=dlast.to(DEV))
    _check_gradient(got, want, mag, dtype)
    assert (got["dg"][:, 70, :2] == 0).all()


def test_gradient_against_differences():
    """In fp32, along random directions, the gradients are the slope of the loss, which the reference evaluates in
    double precision on both sides of the point."""
    N, L, H, P, G, S = 2, 70, 4, 24, 2, 20
    a, s0, _ = _case(N, L, H, P, G, S, "f32", True, None, 4)
    g = torch.Generator().manual_seed(8)
    dy, dlast = torch.randn(N, L, H, P, generator=g), torch.randn(N, H, P, S, generator=g)
    got = _plan(N, L, H, P, G, S, "f32").backward(dy.to(DEV), **_gpu(a), state=s0.to(DEV), dstate_out=dlast.to(DEV))
    grad = {k: got["d" + k].cpu().double() for k in ("q", "k", "v", "g", "beta", "state")}
    v = {k: t.double() for k, t in dict(a, state=s0).items()}

    def loss(s, way):
        y, last, _, _ = ref.delta(**{k: t + s * way[k] for k, t in v.items()}, scale=S ** -0.5)
        return float((y * dy.double()).sum() + (last * dlast.double()).sum())

    eps = 1e-5
    for k in v:
        way = {j: torch.randn(t.shape, generator=g, dtype=torch.float64) * (j == k) for j, t in v.items()}
        slope = (loss(eps, way) - loss(-eps, way)) / (2 * eps)
        # fp32 gradients: 2^-13 of sums of terms that in norm are about the gradient's own
        scale = float(grad[k].norm() * way[k].norm())
        assert abs(float((grad[k] * way[k]).sum()) - slope) <= 2.0 ** -13 * scale + 1e-6 * abs(slope), (k, slope)
