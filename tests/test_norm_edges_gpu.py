"""The group norm on the GPU at the ends of its range: means whose square is no fp32 number,
sums of thousands of equal terms a thread.  Reference: oracle/norm.py.
"""
import pytest
import torch

from oracle import norm as ref
from test_norm_gpu import C, CG, DEV, HALF, TYPE, _gpu, _near, _plan

pytestmark = pytest.mark.gpu


# N, L, G, C, per_token: several batches a thread, a row wider than a workgroup, one row, tokens in registers, tokens
# that are samples of their own
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mean", [2e19, -2e19])
@pytest.mark.parametrize("case", [(2, 300, 3, 40, False), (1, 9, 1, 2050, False), (3, 1, 2, 64, False), (2, 5, 2, 64, True),
                                  (1, 3, 1, 4100, True)], ids=str)
def test_means_whose_square_overflows(case, mean, dtype):
    """Only what is left of the mean is squared: 2e19 squared is beyond fp32, half of 2^-7 of it squared is 6e33 and
    12000 of these 7e37.  Both types hold the two values."""
    N, L, G, Ch, per_token = case
    g = torch.Generator().manual_seed(L)
    t = TYPE[dtype]
    a = dict(x=(mean * (1 + 2.0 ** -7 * torch.randint(0, 2, (N, L, G, Ch), generator=g))).to(t),
             w=(1 + 0.3 * torch.randn(G, Ch, generator=g)).to(t), bias=torch.randn(G, Ch, generator=g).to(t), gate=None,
             lengths=None)
    dy = torch.randn(N, L, G, Ch, generator=g).to(t)
    kw = dict(act="silu", per_token=per_token)
    p = _plan(N, L, G, Ch, dtype, a, **kw)
    y, my = ref.norm(**a, **kw)
    _near(p(**_gpu(a)), y, my, HALF[dtype], C, "y")
    want, mag = ref.norm_grad(dy, **a, **kw)
    for k, got in p.backward(dy.to(DEV), **_gpu(a)).items():
        if got is not None:
            _near(got, want[k], mag[k], HALF[dtype], CG, k)


@pytest.mark.parametrize("dims", [(1, (1 << 21) + 5, 32, 4), (3, (1 << 23) + 7, 1, 8)], ids=str)
def test_more_tokens_than_samples_could_be(dims):
    """Each token by itself: the first and the last tokens as in a call of their own, forward and gradient, padded too;
    dw and dbias as the sums of the terms.  bf16 tensors of one sign in dy."""
    N, L, G, Ch = dims
    n = 300
    g = torch.Generator(DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    x, dy, w, b = r(N, L, G, Ch), r(N, L, G, Ch).abs(), r(G, Ch), r(G, Ch)
    lengths = torch.full((N,), L, dtype=torch.int32, device=DEV)
    lengths[-1] = L - 100
    a = dict(bias=0, gate=None)
    p, q = (_plan(N, m, G, Ch, "bf16", a, per_token=True) for m in (L, n))
    y, got = p(x, w, b, lengths=lengths), p.backward(dy, x, w, b, lengths=lengths)
    for lo in (0, L - n):
        part = slice(lo, lo + n)
        short = (lengths - lo).clamp(max=n)
        cut, cdy = x[:, part].contiguous(), dy[:, part].contiguous()
        assert torch.equal(y[:, part], q(cut, w, b, lengths=short))
        assert torch.equal(got["dx"][:, part], q.backward(cdy, cut, w, b, lengths=short)["dx"])
    # the terms are dy, at most 512 of a thread in fp32: 2^-15 of their sum, and the result's rounding
    keep = torch.arange(L, device=DEV) < lengths[:, None]
    db = sum((dy[i].double() * keep[i, :, None, None]).sum(0) for i in range(N))
    assert ((got["dbias"].double() - db).abs() <= (2.0 ** -8 * (1 + 2 ** -8) + 2.0 ** -15) * db).all()


@pytest.mark.parametrize("dtype,Ch", [("bf16", 520), ("bf16", 2048), ("f32", 260), ("f32", 1024)])
def test_tokens_in_registers_and_columns_that_are_not(dtype, Ch):
    """The same plan over aligned tensors, whose groups stay in registers, and over columns from an odd one on, which
    go through slabs: forward and gradient, the rest of the rows as it was."""
    N, L, G = 2, 21, 3
    W, t = G * Ch, TYPE[dtype]
    g = torch.Generator().manual_seed(Ch)
    r = lambda *s: torch.randn(*s, generator=g)
    a = dict(x=r(N, L, G, Ch).to(t), w=(1 + 0.3 * r(G, Ch)).to(t), bias=r(G, Ch).to(t), gate=r(N, L, G, Ch).to(t),
             lengths=torch.tensor([L, 9], dtype=torch.int32))
    dy = r(N, L, G, Ch).to(t)
    kw = dict(act="silu", per_token=True)
    p = _plan(N, L, G, Ch, dtype, a, **kw)
    y, my = ref.norm(**a, **kw)
    want, mag = ref.norm_grad(dy, **a, **kw)
    v = _gpu(a)
    _near(p(**v), y, my, HALF[dtype], C, "y")
    wide = torch.full((N, L, 2 * W + 1), 5.0, dtype=t, device=DEV)
    x, out = (wide[..., i:i + W].unflatten(-1, (G, Ch)) for i in (1, W + 1))
    x.copy_(v["x"])
    _near(p(**dict(v, x=x), out=out), y, my, HALF[dtype], C, "y")
    for got in (p.backward(dy.to(DEV), **v), p.backward(dy.to(DEV), **dict(v, x=x), out={"dx": out})):
        for k in want:
            _near(got[k], want[k], mag[k], HALF[dtype], CG, k)
    assert (wide[..., 0] == 5).all() and torch.equal(x, v["x"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("per_token,Ch", [(False, 24), (True, 24), (True, 520)])
def test_what_is_no_number_reaches_its_group_and_no_other(per_token, Ch, bad):
    """All of its group's y and dx are NaN; every other group's are what they are without it, to the bit."""
    N, L, G = 2, 37, 3
    g = torch.Generator().manual_seed(Ch)
    x, dy, w = torch.randn(N, L, G, Ch, generator=g), torch.randn(N, L, G, Ch, generator=g).to(DEV), torch.ones(G, Ch, device=DEV)
    p = _plan(N, L, G, Ch, "f32", dict(bias=None, gate=None), per_token=per_token)
    out = []
    for value in (float(x[1, 5, 1, 7]), bad):
        x[1, 5, 1, 7] = value
        d = x.to(DEV)
        out.append((p(d, w), p.backward(dy, d, w)["dx"]))
    for clean, got in zip(*out):
        mine = torch.zeros(N, L, G, Ch, dtype=torch.bool, device=DEV)
        mine[1, 5:6, 1] = True
        if not per_token:
            mine[1, :, 1] = True
        assert torch.isnan(got[mine]).all() and torch.equal(got[~mine], clean[~mine])
