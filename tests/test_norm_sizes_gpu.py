"""The group norm on the GPU where offsets pass 32 bits, on other streams, and two calls at a
time: the same numbers as the same rows by themselves.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _plan(N, L, G, C, dtype, **kw):
    from convolution_forward_implicit_amd import GroupNorm
    return GroupNorm({"N": N, "L": L, "G": G, "C": C}, dtype, **kw)


def test_more_than_2_to_31_tokens_values():
    """Tokens past the 2^31st value, forward and gradient, are those of a call of their own: the same bits, each token
    by itself."""
    G, C, last = 2, 128, 300
    L = 2 ** 31 // (G * C) + last
    x = torch.empty(1, L, G, C, dtype=torch.bfloat16, device=DEV).normal_()
    w = torch.randn(G, C, device=DEV).to(torch.bfloat16)
    p, q = (_plan(1, n, G, C, "bf16", act="silu", per_token=True, center=False) for n in (L, last))
    end = x[:, -last:]
    assert torch.equal(p(x, w)[:, -last:], q(end.contiguous(), w))
    got = p.backward(x, x, w)["dx"]
    assert torch.equal(got[:, -last:], q.backward(end.contiguous(), end.contiguous(), w)["dx"])


def test_more_than_2_to_31_pixels_values():
    """A sample past the 2^31st value.  Its slabs are cut otherwise than in a call of its own, so a result may round
    the other way: by one step, 2^-7 of its value."""
    G, C = 8, 32
    L = 2 ** 30 // (G * C) + 3
    x = torch.empty(3, L, G, C, dtype=torch.bfloat16, device=DEV).normal_()
    w, b = torch.randn(2, G, C, device=DEV).to(torch.bfloat16).unbind()
    p, q = (_plan(n, L, G, C, "bf16", act="gelu", has_bias=True) for n in (3, 1))
    got, want = p(x, w, b)[2:], q(x[2:], w, b)
    for lo in (0, L // 2, L - 1000):
        a, e = got[:, lo:lo + 1000].double(), want[:, lo:lo + 1000].double()
        assert ((a - e).abs() <= 2.0 ** -7 * e.abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_calls_at_once(dtype, per_token):
    """On streams of their own, given and current."""
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    N, L, G, C = 3, 517, 6, 40
    g = torch.Generator().manual_seed(3)
    p = _plan(N, L, G, C, dtype, act="silu", has_bias=True, gated=True, per_token=per_token)
    r = lambda *s: torch.randn(*s, generator=g).to(t).to(DEV)
    calls = [dict(x=r(N, L, G, C), w=r(G, C), bias=r(G, C), gate=r(N, L, G, C)) for _ in range(2)]
    dys = [r(N, L, G, C) for _ in calls]
    want = [(p(**c), p.backward(d, **c)) for c, d in zip(calls, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for i, (s, c, d) in enumerate(zip(streams, calls, dys)):
            if i == 0:
                got.append((p(**c, stream=s), p.backward(d, **c, stream=s)))
            else:
                with torch.cuda.stream(s):
                    got.append((p(**c), p.backward(d, **c)))
        torch.cuda.synchronize()
        for (y, e), (z, f) in zip(got, want):
            assert torch.equal(y, z)
            for k in f:
                assert torch.equal(e[k], f[k]), k
