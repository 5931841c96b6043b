"""The operators of a mixer run together, as a model runs them: the short convolution,
unit keys and queries, the gated delta rule, and the norm of its heads with a gate;
over a padded batch, token by token, backwards, on other streams and in captured
graphs.

Tolerances: every operator is within a rounding (2^-8 in bf16, 2^-24 in fp32) and
2^-13 of its terms of the exact one (their own tests); norms that divide by a spread of
about one pass errors on.  Four of them chained, in 2-norm: 8 x 2^-8 in bf16, 2^-12 in
fp32.
"""
import pytest
import torch

from oracle import delta as rdelta, norm as rnorm, seq

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
FAR = {"bf16": 2.0 ** -5, "f32": 2.0 ** -12}
DEV = "cuda:0"
N, H, P, G, S, F = 2, 4, 32, 2, 24, 4
W = 2 * G * S + H * P


def _far(got, want):
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    assert torch.isfinite(got).all()
    return float((got - want).norm() / want.norm().clamp(min=1e-30))


def _cut(m):
    return (m[..., :G * S].unflatten(-1, (G, S)), m[..., G * S:2 * G * S].unflatten(-1, (G, S)),
            m[..., 2 * G * S:].unflatten(-1, (H, P)))


def _inputs(dtype, L, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = TYPE[dtype]
    return dict(u=r(N, L, W).to(t), w=(0.5 * r(W, F)).to(t), bias=(0.1 * r(W)).to(t), g=-0.2 * r(N, L, H).abs(),
                beta=torch.sigmoid(r(N, L, H)).to(t), z=r(N, L, H, P).to(t), unit=torch.full((G, S), S ** -0.5).to(t),
                scale=(1 + 0.1 * r(H, P)).to(t))


class Mixer:
    def __init__(self, dtype, L):
        from convolution_forward_implicit_amd import CausalConv, DeltaRule, GroupNorm
        self.conv = CausalConv({"N": N, "L": L, "C": W, "F": F}, dtype, has_bias=True, silu=True)
        self.unit = GroupNorm({"N": N, "L": L, "G": G, "C": S}, dtype, center=False, per_token=True, eps=1e-6)
        self.rule = DeltaRule({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype)
        self.norm = GroupNorm({"N": N, "L": L, "G": H, "C": P}, dtype, act="silu", gated=True, center=False, per_token=True)

    def forward(self, v, lengths=None, stream=None, conv_state=None, state=None, conv_out=None, state_out=None):
        c = self.conv(v["u"], v["w"], v["bias"], state=conv_state, lengths=lengths, state_out=conv_out, stream=stream)
        q0, k0, x = _cut(c)
        q = self.unit(q0, v["unit"], lengths=lengths, stream=stream)
        k = self.unit(k0, v["unit"], lengths=lengths, stream=stream)
        y = self.rule(q, k, x, v["g"], v["beta"], state=state, lengths=lengths, state_out=state_out, stream=stream)
        return self.norm(y, v["scale"], gate=v["z"], lengths=lengths, stream=stream), (c, q, k, y)

    def backward(self, dout, v, kept, lengths=None, stream=None):
        c, q, k, y = kept
        q0, k0, x = _cut(c)
        a = self.norm.backward(dout, y, v["scale"], gate=v["z"], lengths=lengths, stream=stream)
        dc = torch.empty_like(c)
        dq0, dk0, dx = _cut(dc)
        b = self.rule.backward(a["dx"], q, k, x, v["g"], v["beta"], lengths=lengths, out={"dv": dx}, stream=stream)
        d = self.unit.backward(b["dq"], q0, v["unit"], lengths=lengths, out={"dx": dq0}, stream=stream)
        e = self.unit.backward(b["dk"], k0, v["unit"], lengths=lengths, out={"dx": dk0}, stream=stream)
        f = self.conv.backward(dc, v["u"], v["w"], v["bias"], lengths=lengths, stream=stream)
        return {"u": f["dx"], "w": f["dw"], "bias": f["dbias"], "g": b["dg"], "beta": b["dbeta"], "z": a["dgate"],
                "scale": a["dw"], "unit": d["dw"] + e["dw"]}


def _reference(v, lengths):
    c, _, _ = seq.causal(v["u"], v["w"], v["bias"], True, lengths=lengths)
    q0, k0, x = _cut(c)
    unit = lambda t: rnorm.norm(t, v["unit"], lengths=lengths, center=False, per_token=True, eps=1e-6)[0]
    y, last, _, _ = rdelta.delta(unit(q0), unit(k0), x, v["g"], v["beta"], S ** -0.5, lengths=lengths)
    return rnorm.norm(y, v["scale"], None, v["z"], lengths, "silu", False, True)[0], last


def _gpu(d):
    return {k: t.to(DEV) for k, t in d.items()}


@pytest.mark.parametrize("lengths", [None, [70, 33]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_and_gradient(dtype, lengths):
    L = 70
    v = _inputs(dtype, L)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    nd = None if n is None else n.to(DEV)
    m, d = Mixer(dtype, L), _gpu(v)
    last = torch.empty(N, H, P, S, device=DEV)
    out, kept = m.forward(d, nd, state_out=last)
    want, rlast = _reference(v, n)
    assert _far(out, want) <= FAR[dtype] and _far(last, rlast) <= FAR[dtype]
    g = torch.Generator().manual_seed(5)
    dout = torch.randn(N, L, H, P, generator=g).to(TYPE[dtype])
    grad = {k: t.cpu().double() for k, t in m.backward(dout.to(DEV), d, kept, nd).items()}
    v64 = {k: t.double() for k, t in v.items()}
    eps = 1e-4
    for k in v:
        # the loss's slope along each gradient's own direction is that gradient's length
        way = grad[k] / grad[k].norm()
        loss = lambda s: float((_reference(dict(v64, **{k: v64[k] + s * way}), n)[0] * dout.double()).sum())
        slope = (loss(eps) - loss(-eps)) / (2 * eps)
        assert abs(slope - float(grad[k].norm())) <= FAR[dtype] * abs(slope), (k, slope, float(grad[k].norm()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(dtype):
    L = 72
    v = _inputs(dtype, L)
    d = _gpu(v)
    cut = lambda lo, hi: {k: t[:, lo:hi].contiguous() if t.dim() > 2 and t.shape[1] == L else t for k, t in d.items()}
    cs = torch.zeros(N, F - 1, W, dtype=TYPE[dtype], device=DEV)
    conv_out, state = torch.empty_like(cs), torch.empty(N, H, P, S, device=DEV)
    ys = [Mixer(dtype, 67).forward(cut(0, 67), conv_state=cs, conv_out=conv_out, state_out=state)[0]]
    m = Mixer(dtype, 1)
    for t in range(67, L):
        q0, k0, x = _cut(m.conv.step(d["u"][:, t], d["w"], conv_out, d["bias"]))
        q, k = (m.unit(a[:, None], d["unit"])[:, 0] for a in (q0, k0))
        y = m.rule.step(q, k, x, d["g"][:, t], d["beta"][:, t], state)
        ys.append(m.norm(y[:, None], d["scale"], gate=d["z"][:, t:t + 1].contiguous()))
    want, last = _reference(v, None)
    assert _far(torch.cat(ys, 1), want) <= FAR[dtype] and _far(state, last) <= FAR[dtype]


def _everything(dtype="bf16", L=130):
    m, d = Mixer(dtype, L), _gpu(_inputs(dtype, L))
    dout = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(4)).to(TYPE[dtype]).to(DEV)

    def run(stream=None):
        out, kept = m.forward(d, stream=stream)
        return [out] + list(m.backward(dout, d, kept, stream=stream).values())
    return d, run


def test_same_bits_every_time_and_on_two_streams_at_once():
    _, run = _everything()
    want = run()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (one, two):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for s in (one, two, one, two):
        with torch.cuda.stream(s):
            got.append(run())
    torch.cuda.synchronize()
    for other in [run()] + got:
        for a, b in zip(want, other):
            assert torch.equal(a, b)


def test_a_stream_that_is_not_the_current_one():
    """Calls that are given a stream launch and allocate there, step and norm among them."""
    m, d = Mixer("bf16", 130), _gpu(_inputs("bf16", 130))
    want, kept = m.forward(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = m.forward(d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_captured_and_replayed_with_new_inputs():
    """Two graphs of the same plans in turn, with eager work between: each replay is the eager result of its inputs."""
    d, run = _everything(L=70)
    _, other = _everything(L=70)
    run(), other()
    torch.cuda.synchronize()
    graphs = []
    for f in (run, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = f()
        graphs.append((g, outs, f))
    for k in range(3):
        with torch.no_grad():
            for t in ("u", "z"):
                d[t].mul_(0.9).add_(0.01 * k)
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, outs, f in graphs:
            for a, b in zip(outs, f()):
                assert torch.equal(a, b)


def test_norm_behind_a_convolution():
    """ConvFwd's result, channels innermost, normalised over its pixels as it stands."""
    from convolution_forward_implicit_amd import ConvFwd, GroupNorm
    import synthdata as sd
    p = sd.problem(2, 2, 16, 32, (1, 9, 11), (1, 3, 3), (1, 1, 1), (0, 1, 1), (1, 1, 1))
    x, w, _ = sd.random_inputs(p, "bf16", 3, False)
    put = lambda a: torch.from_numpy(a).to(DEV).to(torch.bfloat16).contiguous()
    conv = ConvFwd(p, "bf16")
    y = conv(put(x), put(w))
    norm = GroupNorm({"N": 2, "L": 99, "G": 8, "C": 8}, "bf16", act="silu", has_bias=True)
    scale, bias = torch.full((8, 8), 1.5).bfloat16(), torch.full((8, 8), 0.25).bfloat16()
    flat = y.view(2, 99, 8, 8)
    got = norm(flat, scale.to(DEV), bias.to(DEV))
    want, mag = rnorm.norm(flat.cpu(), scale, bias, act="silu")
    assert ((got.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2 ** -8) + 2.0 ** -17 * mag).all()
