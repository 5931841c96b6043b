"""The group norm on the GPU against the double-precision reference
(oracle/norm.py): every width of access, rows narrower and wider than a workgroup,
tokens by themselves and samples, ragged and strided batches, large means.

Tolerances.  A result of type T is rounded once: half a step, 2^-8 (bf16) or 2^-24
(fp32) of its value.  Before that fp32 arithmetic: x less its mean and its product
with r, w, b at 2^-24 of the scale that the reference gives each, the sigmoid's and
Phi's approximations (2^-22; in bf16 Phi is a fit within 2^-17.9), sums of at most
64 values in a register and then in fp64: under 16 x 2^-24 + 2^-17.9 < 2^-17 of the
scale.  The gradients chain two such results and sum up to 2^5 values a thread
beyond a batch: under 2^-15 of theirs.
"""
import pytest
import torch

from oracle import norm as ref

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"
C, CG = 2.0 ** -17, 2.0 ** -15


def _near(got, want, mag, half, c, what):
    got, want, mag = got.detach().cpu().double(), want.double(), mag.double().abs()
    assert torch.isfinite(got).all(), what
    if not want.numel():
        return
    over = (got - want).abs() - (half * want.abs() * (1 + 2 ** -8) + c * mag + 1e-37)
    assert (over <= 0).all(), "%s: %g over at %r (got %g, want %g)" % (
        what, over.max(), tuple(torch.nonzero(over == over.max())[0].tolist()),
        got.flatten()[over.argmax()], want.flatten()[over.argmax()])


def _gpu(d):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def _case(N, L, G, C, dtype, bias, gated, lengths, seed, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    t = TYPE[dtype]
    r = lambda *s: torch.randn(*s, generator=g)
    a = dict(x=(r(N, L, G, C) + r(G, C) + mean).to(t), w=(1 + 0.3 * r(G, C)).to(t), bias=r(G, C).to(t) if bias else None,
             gate=r(N, L, G, C).to(t) if gated else None, lengths=None)
    if lengths is not None and N:
        n = torch.randint(0, L + 1, (N,), generator=g, dtype=torch.int32)
        n[0] = {"zero": 0, "one": min(1, L), "most": max(0, L - 1)}[lengths]
        a["lengths"] = n
    return a, r(N, L, G, C).to(t)


def _plan(N, L, G, C, dtype, a, **kw):
    from convolution_forward_implicit_amd import GroupNorm
    return GroupNorm({"N": N, "L": L, "G": G, "C": C}, dtype, has_bias=a["bias"] is not None, gated=a["gate"] is not None, **kw)


# N, L, G, C, lengths
CASES = [(1, 1, 1, 1, None), (2, 49, 32, 8, None), (3, 37, 8, 48, "most"), (2, 130, 1, 40, "zero"), (2, 33, 4, 12, "one"),
         (1, 300, 3, 7, None), (2, 9, 1, 2050, "most"), (2, 5, 2, 2056, None), (0, 4, 2, 8, None), (2, 0, 2, 8, None),
         (1, 700, 2, 128, None), (2, 70, 5, 64, "most"), (1, 3, 70, 32, None), (4, 1, 6, 24, None)]
KINDS = [dict(act="none"), dict(act="silu"), dict(act="gelu"), dict(act="silu", gated=True), dict(act="gelu", gated=True, center=False),
         dict(act="none", center=False, bias=False), dict(act="none", gated=True, bias=False)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join("%s=%s" % i for i in k.items()))
@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_and_gradient(case, dtype, per_token, kind):
    N, L, G, Ch, lengths = case
    a, dy = _case(N, L, G, Ch, dtype, kind.get("bias", True), kind.get("gated", False), lengths, 3 + L)
    kw = dict(act=kind["act"], center=kind.get("center", True), per_token=per_token, eps=1e-3)
    p = _plan(N, L, G, Ch, dtype, a, **kw)
    y, my = ref.norm(**a, **kw)
    _near(p(**_gpu(a)), y, my, HALF[dtype], C, "y")
    want, mag = ref.norm_grad(dy, **a, **kw)
    got = p.backward(dy.to(DEV), **_gpu(a))
    assert (got["dgate"] is None) == (a["gate"] is None) and (got["dbias"] is None) == (a["bias"] is None)
    for k, t in got.items():
        if t is not None:
            _near(t, want[k], mag[k], HALF[dtype], CG, k)


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("mean", [1000.0, -3e4])
def test_means_far_larger_than_the_spread(per_token, mean):
    """Squares are summed around a mean: nothing of the spread is lost that x itself still holds."""
    N, L, G, Ch = 2, 200, 4, 64
    a, dy = _case(N, L, G, Ch, "f32", True, False, None, 1, mean)
    a["x"][:, 0] = 0 if not per_token else a["x"][:, 0]          # a first row unlike the others
    p = _plan(N, L, G, Ch, "f32", a, act="silu", per_token=per_token)
    y, my = ref.norm(**a, act="silu", per_token=per_token)
    _near(p(**_gpu(a)), y, my, HALF["f32"], C, "y")
    want, mag = ref.norm_grad(dy, **a, act="silu", per_token=per_token)
    for k, t in p.backward(dy.to(DEV), **_gpu(a)).items():
        if t is not None:
            _near(t, want[k], mag[k], HALF["f32"], CG, k)


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_column_ranges(dtype, per_token):
    """x, gate, y and the gradients as columns of wider tensors, aligned and not: the rest of the rows stays as it was.
    Other accesses add the same terms in another order: both results are within the tolerance of the exact one."""
    N, L, G, Ch = 2, 37, 4, 24
    W = G * Ch
    a, dy = _case(N, L, G, Ch, dtype, True, True, "most", 5)
    kw = dict(act="silu", per_token=per_token)
    p = _plan(N, L, G, Ch, dtype, a, **kw)
    v = _gpu(a)
    y, my = ref.norm(**a, **kw)
    want, mag = ref.norm_grad(dy, **a, **kw)
    for lo, wide in ((8, 2 * W + 8), (3, 2 * W + 3), (2, 2 * W + 4)):
        u = torch.full((N, L, wide), 5.0, dtype=TYPE[dtype], device=DEV)
        x, gate = u[..., lo:lo + W].unflatten(-1, (G, Ch)), u[..., wide - W:].unflatten(-1, (G, Ch))
        x.copy_(v["x"])
        if lo + W <= wide - W:
            gate.copy_(v["gate"])
        else:
            gate = v["gate"]
        both = torch.full((N, L, wide), 9.0, dtype=TYPE[dtype], device=DEV)
        out = both[..., lo:lo + W].unflatten(-1, (G, Ch))
        p(**dict(v, x=x, gate=gate), out=out)
        _near(out, y, my, HALF[dtype], C, "y")
        assert (both[..., :lo] == 9).all() and (both[..., lo + W:] == 9).all()
        got = p.backward(dy.to(DEV), **dict(v, x=x, gate=gate), out={"dx": out})
        for k in want:
            _near(got[k], want[k], mag[k], HALF[dtype], CG, k)
        assert (both[..., :lo] == 9).all() and (both[..., lo + W:] == 9).all()


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_behind_a_sample_is_read(dtype, per_token):
    N, L, G, Ch = 3, 70, 2, 24
    a, dy = _case(N, L, G, Ch, dtype, True, True, None, 7)
    a["lengths"] = torch.tensor([70, 0, 37], dtype=torch.int32)
    p = _plan(N, L, G, Ch, dtype, a, act="gelu", per_token=per_token)
    y, got = p(**_gpu(a)), p.backward(dy.to(DEV), **_gpu(a))
    bad = dict(a, x=a["x"].clone(), gate=a["gate"].clone(), lengths=torch.tensor([99, -3, 37], dtype=torch.int32))
    for i, n in enumerate((70, 0, 37)):
        bad["x"][i, n:], bad["gate"][i, n:], dy[i, n:] = float("nan"), float("inf"), float("nan")
        assert (y[i, n:] == 0).all() and (got["dx"][i, n:] == 0).all() and (got["dgate"][i, n:] == 0).all()
    assert torch.equal(p(**_gpu(bad)), y)
    for k, t in p.backward(dy.to(DEV), **_gpu(bad)).items():
        assert torch.equal(t, got[k]), k


def test_gradient_against_differences():
    """In fp32, along random directions, the gradients are the slope of the loss, which the reference evaluates in
    double precision on both sides of the point."""
    for per_token in (False, True):
        a, dy = _case(2, 30, 3, 20, "f32", True, True, None, 4)
        kw = dict(act="gelu", per_token=per_token)
        got = _plan(2, 30, 3, 20, "f32", a, **kw).backward(dy.to(DEV), **_gpu(a))
        names = {"x": "dx", "w": "dw", "bias": "dbias", "gate": "dgate"}
        v = {k: a[k].double() for k in names}
        g = torch.Generator().manual_seed(8)
        loss = lambda s, way: float((ref.norm(**{k: t + s * way[k] for k, t in v.items()}, **kw)[0] * dy.double()).sum())
        eps = 1e-5
        for k in v:
            way = {j: torch.randn(t.shape, generator=g, dtype=torch.float64) * (j == k) for j, t in v.items()}
            slope = (loss(eps, way) - loss(-eps, way)) / (2 * eps)
            grad = got[names[k]].cpu().double()
            scale = float(grad.norm() * way[k].norm())
            assert abs(float((grad * way[k]).sum()) - slope) <= 2.0 ** -15 * scale + 1e-6 * abs(slope), (k, slope)
