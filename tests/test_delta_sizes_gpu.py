"""The gated delta rule on the GPU at the sizes that take its other forms: more blocks of
channels than compute units, keys as wide as their operands, several heads of a group
in a workgroup, offsets past 32 bits, two calls at a time.  Reference and
tolerances are those of the tests of the smaller sizes.
"""
import pytest
import torch

from oracle import delta as ref
from test_delta_gpu import C, DEV, HALF, TYPE, _case, _check_gradient, _gpu, _near, _plan

pytestmark = pytest.mark.gpu


# more than 256 blocks of 16 channels: an odd number of them in a head, one, a last one that is not full
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(2, 65, 48, 40, 4, 24, True, "most"), (3, 70, 96, 32, 96, 64, False, None),
                                  (5, 66, 27, 33, 9, 128, True, "zero"), (2, 130, 135, 16, 5, 32, True, "one"),
                                  (3, 64, 12, 130, 4, 200, True, None)], ids=str)
def test_many_channels(case, dtype):
    N, L, H, P, G, S, state, lengths = case
    a, s0, n = _case(N, L, H, P, G, S, dtype, state, lengths, 41 + L)
    g = torch.Generator().manual_seed(L)
    dy = torch.randn(N, L, H, P, generator=g).to(TYPE[dtype])
    dlast = torch.randn(N, H, P, S, generator=g)
    put = lambda t: None if t is None else t.to(DEV)
    p = _plan(N, L, H, P, G, S, dtype)
    y, last, my, ms = ref.delta(**a, scale=S ** -0.5, state=s0, lengths=n)
    out = torch.full((N, H, P, S), 7.0, device=DEV)
    got = p(**_gpu(a), state=put(s0), lengths=put(n), state_out=out)
    _near(got, y, my, HALF[dtype], C, "y")
    _near(out, last, ms, HALF["f32"], C, "state_out")
    want, mag = ref.delta_grad(dy, **a, scale=S ** -0.5, state=s0, lengths=n, dstate_out=dlast)
    got = p.backward(dy.to(DEV), **_gpu(a), state=put(s0), lengths=put(n), dstate_out=put(dlast))
    _check_gradient(got, want, mag, dtype)


# the heads of a group in one workgroup of the gradient, and in several
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(4, 1025, 12, 8, 4, 16), (5, 1281, 8, 8, 1, 16), (3, 1400, 20, 8, 4, 40)], ids=str)
def test_gradient_of_shared_keys(case, dtype):
    N, L, H, P, G, S = case
    a, s0, n = _case(N, L, H, P, G, S, dtype, True, "most", 5 + L)
    dy = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(L)).to(TYPE[dtype])
    want, mag = ref.delta_grad(dy, **a, scale=S ** -0.5, state=s0, lengths=n)
    got = _plan(N, L, H, P, G, S, dtype).backward(dy.to(DEV), **_gpu(a), state=s0.to(DEV), lengths=n.to(DEV))
    _check_gradient(got, want, mag, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [32, 64, 128, 256])
def test_aligned_keys(S, dtype):
    """Keys as wide as their operands, as columns of one tensor, aligned and not: the same numbers; NaN behind the
    lengths."""
    N, L, H, P, G = 3, 150, 4, 24, 2
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 3 + S)
    n = torch.tensor([150, 0, 71], dtype=torch.int32)
    u = torch.cat([a["q"].flatten(2), a["k"].flatten(2)], -1).to(DEV)
    y, last, my, ms = ref.delta(**a, scale=S ** -0.5, state=s0, lengths=n)
    for i in range(N):
        u[i, n[i]:] = float("nan")
        a["v"][i, n[i]:] = float("inf")
    v = _gpu(a)
    v["q"], v["k"] = (t.unflatten(-1, (G, S)) for t in u.split([G * S, G * S], -1))
    out = torch.empty(N, H, P, S, device=DEV)
    got = _plan(N, L, H, P, G, S, dtype)(**v, state=s0.to(DEV), lengths=n.to(DEV), state_out=out)
    _near(got, y, my, HALF[dtype], C, "y")
    _near(out, last, ms, HALF["f32"], C, "state_out")
    w = torch.cat([torch.zeros(N, L, 1, dtype=TYPE[dtype], device=DEV), u], -1)
    v["q"], v["k"] = (t.unflatten(-1, (G, S)) for t in w[..., 1:].split([G * S, G * S], -1))
    assert torch.equal(got, _plan(N, L, H, P, G, S, dtype)(**v, state=s0.to(DEV), lengths=n.to(DEV)))


def test_offsets_past_32_bits():
    """Rows 16 MB apart, all in one tensor: those of the last sequence lie past the 2^32nd element."""
    N, L, H, P, G, S = 3, 192, 2, 32, 1, 32
    far = 1 << 23
    a, _, _ = _case(N, L, H, P, G, S, "bf16", False, None, 2)
    v = _gpu(a)
    p = _plan(N, L, H, P, G, S, "bf16")
    want = p(**v)
    wide = torch.zeros(N * L * far, dtype=torch.bfloat16, device=DEV).view(N, L, far)       # 9.7 GB
    q, k, x, y = wide[..., :S], wide[..., S:2 * S], wide[..., 2 * S:2 * S + H * P], wide[..., 512:512 + H * P]
    q.copy_(v["q"].flatten(2)), k.copy_(v["k"].flatten(2)), x.copy_(v["v"].flatten(2))
    got = p(q.unflatten(-1, (G, S)), k.unflatten(-1, (G, S)), x.unflatten(-1, (H, P)), v["g"], v["beta"],
            out=y.unflatten(-1, (H, P)))
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_calls_at_once(dtype):
    """Two plans on two streams, and the gradients of both, as each by itself."""
    N, L, H, P, G, S = 2, 200, 8, 64, 4, 64
    calls = []
    for seed in (1, 2):
        a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, seed)
        dy = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(seed)).to(TYPE[dtype])
        calls.append((_plan(N, L, H, P, G, S, dtype), _gpu(a), s0.to(DEV), dy.to(DEV)))
    run = lambda c: (c[0](**c[1], state=c[2]), c[0].backward(c[3], **c[1], state=c[2]))
    want = [run(c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(run(c))
        torch.cuda.synchronize()
        for (y, d), (z, e) in zip(got, want):
            assert torch.equal(y, z)
            for k in e:
                assert torch.equal(d[k], e[k]), k
