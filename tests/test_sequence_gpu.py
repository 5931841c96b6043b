"""The sequence operators on the GPU against the double-precision reference
(oracle/seq.py): prompts, steps and gradients over the sizes where a tile, a
chunk or a segment ends, ragged and strided batches, captured graphs, other
streams, and the convolution and the scan run together.

Tolerances.  A result of type T is rounded once: half a step, 2^-8 (bf16) or
2^-24 (fp32) of its value.  Before that every sum of terms t_k carries an error
of at most c * sum |t_k|, where the reference evaluates sum |t_k| itself:
  convolution, fp32 arithmetic: F + 1 products and additions at 2^-24 and the
    sigmoid's two approximations (2^-22): c = 2^-20; its gradients sum up to
    N L further terms, in runs of 16 and then in a fixed tree: c = 2^-17.
  scan: operands computed on the way (M, states, dS) are sums of two or three
    bf16 numbers, off by 2^-16 at most; sums over 128 states, 64 tokens and the
    chunks add (128 + 64 + L / 32) 2^-24 < 2^-16; exponents |c_i| < 2^7 are
    rounded to 2^-24 of themselves, 2^-17 relative in each decay, of which a
    term meets two.  Together under 4 2^-16: c = 2^-14; the gradients chain two
    such products: c = 2^-13.  fp32 calls have the sums and the exponents only
    and meet the same bounds.
  ddt and dA: the sums over the pairs of tokens that a decay lies between are
    differences of sums over the chunk, so their errors go by the chunk's terms:
    sum |t_k| is taken over the 127 tokens around.
"""
import pytest
import torch

from oracle import seq

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


def _ops():
    from convolution_forward_implicit_amd import CausalConv, SelectiveScan
    return CausalConv, SelectiveScan


def _near(got, want, mag, half, c, what):
    got, want, mag = got.detach().cpu().double(), want.double(), mag.double().abs()
    assert torch.isfinite(got).all(), what
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


# ---- convolution -----------------------------------------------------------------
def _conv_case(N, L, C, F, dtype, state, lengths, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(TYPE[dtype])
    a = dict(x=r(N, L, C), w=r(C, F), bias=r(C), state=r(N, F - 1, C) if state else None)
    return a, r(N, L, C), r(N, F - 1, C), _lengths(lengths, N, L, g)


CONVS = [(1, 1, 1, 2, True, None), (2, 1, 8, 4, True, "zero"), (1, 7, 64, 4, False, None), (3, 8, 24, 3, True, "one"),
         (2, 9, 37, 5, True, "most"), (2, 130, 72, 4, True, "zero"), (1, 300, 265, 2, False, "most"),
         (2, 129, 520, 8, True, None), (1, 0, 16, 4, True, None), (0, 5, 16, 4, False, None), (2, 2, 40, 7, True, "one")]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CONVS, ids=str)
def test_convolution_and_gradient(case, dtype, silu):
    N, L, C, F, state, lengths = case
    CausalConv, _ = _ops()
    a, dy, dlast, n = _conv_case(N, L, C, F, dtype, state, lengths, 11 + L)
    p = CausalConv({"N": N, "L": L, "C": C, "F": F}, dtype, has_bias=True, silu=silu)
    y, last, v = seq.causal(**a, silu=silu, lengths=n)
    mag = seq.causal(a["x"].abs(), a["w"].abs(), a["bias"].abs(), False, a["state"].abs() if state else None, n)[0]
    out = torch.full((N, F - 1, C), 7.0, dtype=TYPE[dtype], device=DEV)
    G = _gpu(a)
    nd = None if n is None else n.to(DEV)
    got = p(**G, lengths=nd, state_out=out)
    _near(got, y, mag, HALF[dtype], 2.0 ** -20, "y")
    assert torch.equal(out.cpu(), last.to(TYPE[dtype]))
    want = seq.causal_grad(dy, **a, silu=silu, lengths=n, dstate_out=dlast)
    mags = seq.causal_grad(dy, **a, silu=silu, lengths=n, dstate_out=dlast, magnitude=True)
    # act' = s (1 + v (1 - s)) reaches v s (1 - s): its error goes by 1 + |v|, v's by the sum's terms
    far = 1 + (mag.max() if mag.numel() else 0)
    grads = p.backward(dy.to(DEV), **G, lengths=nd, dstate_out=dlast.to(DEV))
    assert (grads["dstate"] is not None) == state
    direct = seq.causal_grad(dy, **a, silu=False, lengths=n, dstate_out=dlast, magnitude=True)     # |act'| <= 1.1
    for k, t in grads.items():
        if t is not None:
            _near(t, want[k], mags[k] + (direct[k] * far if silu else 0), HALF[dtype], 2.0 ** -17, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_convolution_in_column_ranges(dtype):
    """x, y and dx as columns of wider tensors, aligned and not: the rest of the rows stays as it was."""
    CausalConv, _ = _ops()
    N, L, C, F = 2, 21, 24, 4
    a, dy, _, _ = _conv_case(N, L, C, F, dtype, True, None, 5)
    p = CausalConv({"N": N, "L": L, "C": C, "F": F}, dtype, has_bias=True, silu=True)
    G = _gpu(a)
    want = p(**G)
    grads = p.backward(dy.to(DEV), **G)
    for lo, wide in ((8, 64), (3, 33)):
        x = torch.full((N, L, wide), 5.0, dtype=TYPE[dtype], device=DEV)
        x[..., lo:lo + C] = G["x"]
        both = torch.full((N, L, 2 * wide), 9.0, dtype=TYPE[dtype], device=DEV)
        keep = both.clone()
        view = both[..., wide + lo:wide + lo + C]
        p(**dict(G, x=x[..., lo:lo + C]), out=view)
        assert torch.equal(view, want)
        view.fill_(9.0)
        assert torch.equal(both, keep)
        q = p.backward(dy.to(DEV), **dict(G, x=x[..., lo:lo + C]), out={"dx": view})
        assert torch.equal(view, grads["dx"]) and torch.equal(q["dw"], grads["dw"])
        view.fill_(9.0)
        assert torch.equal(both, keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_behind_a_sequence_is_read(dtype):
    """NaN and infinities in the rows behind the lengths reach nothing."""
    CausalConv, SelectiveScan = _ops()
    g = torch.Generator().manual_seed(2)
    N, L, H, P, G, S, F = 3, 70, 2, 24, 1, 20, 4
    n = torch.tensor([70, 0, 37], dtype=torch.int32)
    bad = lambda *s: torch.randn(*s, generator=g).to(TYPE[dtype])
    t = dict(x=bad(N, L, H, P), dt=bad(N, L, H), B=bad(N, L, G, S), C=bad(N, L, G, S))
    dy = bad(N, L, H, P)
    clean = {k: v.clone() for k, v in t.items()}
    for k, v in list(t.items()) + [("dy", dy)]:
        for i in range(N):
            v[i, n[i]:] = float("nan") if k in ("x", "dt", "dy") else float("inf")
    cdy = torch.where(torch.isnan(dy), torch.zeros((), dtype=dy.dtype), dy)
    A = -torch.rand(H, generator=g) - 0.5
    p = SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype)
    run = lambda v: p(**_gpu(v), A=A.to(DEV), lengths=n.to(DEV))
    assert torch.equal(run(t), run(clean))
    back = lambda v, d: p.backward(d.to(DEV), **_gpu(v), A=A.to(DEV), lengths=n.to(DEV))
    one, two = back(t, dy), back(clean, cdy)
    for k in ("dx", "ddt", "dA", "dB", "dC"):
        assert torch.equal(one[k], two[k]), k
        assert torch.isfinite(one[k]).all()
    c = CausalConv({"N": N, "L": L, "C": H * P, "F": F}, dtype, silu=True)
    w = bad(H * P, F).to(DEV)
    flat = lambda v: v.flatten(2).to(DEV)
    assert torch.equal(c(flat(t["x"]), w, lengths=n.to(DEV)), c(flat(clean["x"]), w, lengths=n.to(DEV)))
    one = c.backward(flat(dy), flat(t["x"]), w, lengths=n.to(DEV))
    two = c.backward(flat(cdy), flat(clean["x"]), w, lengths=n.to(DEV))
    assert torch.equal(one["dx"], two["dx"]) and torch.equal(one["dw"], two["dw"])


# ---- scan ------------------------------------------------------------------------
def _scan_case(N, L, H, P, G, S, dtype, state, lengths, seed, softplus=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = TYPE[dtype]
    a = dict(x=r(N, L, H, P).to(t), dt=(r(N, L, H) if softplus else r(N, L, H).abs() * 0.1).to(t),
             A=-torch.rand(H, generator=g) * 4 - 0.1, B=r(N, L, G, S).to(t), C=r(N, L, G, S).to(t), D=r(H),
             dt_bias=r(H) - 2 if softplus else None, state=r(N, H, P, S) if state else None)
    return a, r(N, L, H, P).to(t), r(N, H, P, S) if state else None, _lengths(lengths, N, L, g)


SCANS = [(1, 1, 1, 1, 1, 1, True, None), (2, 64, 2, 64, 1, 128, False, None), (2, 65, 4, 64, 2, 128, True, "most"),
         (1, 130, 3, 40, 3, 24, True, None), (3, 33, 2, 130, 1, 17, True, "zero"), (1, 200, 2, 16, 1, 64, False, None),
         (2, 63, 2, 128, 2, 100, True, "one"), (1, 500, 1, 64, 1, 32, True, None), (4, 70, 64, 8, 4, 16, True, "most"),
         (2, 0, 2, 16, 1, 16, True, None), (0, 9, 2, 16, 1, 16, False, None), (2, 192, 6, 24, 1, 33, True, "zero"),
         (2, 1030, 64, 8, 2, 16, True, "most"), (1, 900, 3, 72, 1, 40, False, None)]


def _around(v):
    """Sums over the 127 tokens around each, [N, L, H]."""
    if v.shape[1] == 0:
        return v
    c = torch.nn.functional.pad(v.cumsum(1), (0, 0, 1, 0))
    t = torch.arange(v.shape[1])
    return c[:, (t + 64).clamp(max=v.shape[1])] - c[:, (t - 63).clamp(min=0)]


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan(case, dtype, softplus):
    N, L, H, P, G, S, state, lengths = case
    _, SelectiveScan = _ops()
    a, _, _, n = _scan_case(N, L, H, P, G, S, dtype, state, lengths, 17 + L, softplus)
    p = SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype, softplus=softplus)
    y, last = seq.scan(**a, softplus=softplus, lengths=n)
    my, ml = seq.scan(**a, softplus=softplus, lengths=n, magnitude=True)
    out = torch.full((N, H, P, S), 7.0, device=DEV)
    got = p(**_gpu(a), lengths=None if n is None else n.to(DEV), state_out=out)
    _near(got, y, my, HALF[dtype], 2.0 ** -14, "y")
    _near(out, last, ml, HALF["f32"], 2.0 ** -15, "state_out")


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", SCANS, ids=str)
def test_scan_gradient(case, dtype, softplus):
    N, L, H, P, G, S, state, lengths = case
    _, SelectiveScan = _ops()
    a, dy, dlast, n = _scan_case(N, L, H, P, G, S, dtype, state, lengths, 23 + L, softplus)
    p = SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, dtype, softplus=softplus)
    kw = dict(a, softplus=softplus, lengths=n, dstate_out=dlast)
    want, mag = seq.scan_grad(dy, **kw), seq.scan_grad(dy, **kw, magnitude=True)
    my, _ = seq.scan(**a, softplus=softplus, lengths=n, magnitude=True)
    # of dl: what the chunk's sums are made of, and what crosses from chunk to chunk
    near = _around((dy.double().abs() * my).sum(-1) + mag["step"] * mag["e"]) + mag["dl"]
    mag["ddt"] = near * a["A"].double().abs() + mag["e"]
    mag["dA"] = (near * mag["step"]).sum((0, 1))
    mag["ddt_bias"] = mag["ddt"].sum((0, 1))
    got = p.backward(dy.to(DEV), **_gpu(a), lengths=None if n is None else n.to(DEV),
                     dstate_out=None if dlast is None else dlast.to(DEV))
    for k, t in got.items():
        if t is not None:
            _near(t, want[k], mag[k], HALF[dtype] if k in ("dx", "ddt", "dB", "dC") else HALF["f32"], 2.0 ** -13, k)
    assert (got["dstate"] is not None) == state


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (3, 4, 64, 2, 128), (2, 3, 40, 1, 24), (2, 2, 130, 2, 101),
                                  (5, 2, 33, 1, 8)], ids=str)
def test_scan_step(case, dtype):
    N, H, P, G, S = case
    _, SelectiveScan = _ops()
    a, _, _, _ = _scan_case(N, 1, H, P, G, S, dtype, True, None, 31)
    p = SelectiveScan({"N": N, "L": 1, "H": H, "P": P, "G": G, "S": S}, dtype)
    y, last = seq.scan(**a)
    my, ml = seq.scan(**a, magnitude=True)
    v = _gpu(a)
    got = p.step(*(v[k][:, 0] for k in ("x", "dt")), v["A"], v["B"][:, 0], v["C"][:, 0], v["state"], D=v["D"],
                 dt_bias=v["dt_bias"])
    # fp32 arithmetic: S + 3 terms, an exponent below 2^7
    _near(got, y[:, 0], my[:, 0], HALF[dtype], 2.0 ** -16, "y")
    _near(v["state"], last, ml, HALF["f32"], 2.0 ** -16, "state")


def test_scan_in_column_ranges():
    """The parts of one activation as inputs, their gradients into one buffer; y into columns of another.  Odd row
    lengths run on other kernels, which add the same terms in another order: both results are within half a step and
    c sum |t_k| of the exact one, so at most a step (of either, 2^-7 of the larger) and 2 c sum |t_k| apart."""
    _, SelectiveScan = _ops()
    N, L, H, P, G, S = 2, 70, 2, 32, 1, 40

    def same(got, want, mag, extra, c, what):
        if not extra:
            assert torch.equal(got, want), what
        else:
            _near(got, want.cpu(), mag, 2 * HALF["bf16"], 2 * c, what)

    for extra in (0, 3):        # whole 16-byte rows, and odd ones
        a, dy, _, _ = _scan_case(N, L, H, P, G, S, "bf16", False, None, 7)
        p = SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, "bf16")
        v = _gpu(a)
        want, grads = p(**v), p.backward(dy.to(DEV), **v)
        u = torch.cat([v["x"].flatten(2), v["B"].flatten(2), v["C"].flatten(2),
                       torch.zeros(N, L, extra, dtype=torch.bfloat16, device=DEV)], -1).contiguous()
        cut = lambda m: (m[..., :H * P].unflatten(-1, (H, P)), m[..., H * P:H * P + G * S].unflatten(-1, (G, S)),
                         m[..., H * P + G * S:H * P + 2 * G * S].unflatten(-1, (G, S)))
        x, B, C = cut(u)
        wide = torch.full((N, L, H * P + 8 + extra), 3.0, dtype=torch.bfloat16, device=DEV)
        out = wide[..., 8:8 + H * P].unflatten(-1, (H, P))
        w = dict(v, x=x, B=B, C=C)
        same(p(**w, out=out), want, seq.scan(**a, magnitude=True)[0], extra, 2.0 ** -14, "y")
        assert (wide[..., :8] == 3).all() and (wide[..., 8 + H * P:] == 3).all()
        du = torch.full_like(u, 5.0)
        dx, dB, dC = cut(du)
        p.backward(dy.to(DEV), **w, out={"dx": dx, "dB": dB, "dC": dC})
        mag = seq.scan_grad(dy, **a, magnitude=True)
        for k, t in (("dx", dx), ("dB", dB), ("dC", dC)):
            same(t, grads[k], mag[k], extra, 2.0 ** -13, k)
        assert (du[..., H * P + 2 * G * S:] == 5).all()


def test_long_decays_do_not_overflow():
    """Decays whose product over a chunk underflows, and steps of zero: exponents stay differences."""
    _, SelectiveScan = _ops()
    N, L, H, P, G, S = 1, 192, 3, 16, 1, 16
    a, dy, _, _ = _scan_case(N, L, H, P, G, S, "f32", True, None, 3, False)
    a["dt"][:, :, 0], a["dt"][:, :, 1] = 40.0, 0.0
    p = SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, "f32", softplus=False)
    y, _ = seq.scan(**a, softplus=False)
    my, _ = seq.scan(**a, softplus=False, magnitude=True)
    got = p(**_gpu(a))
    # head 0: |c_i| up to 2^14 is rounded to 2^-24 of itself, and a term that counts has a decay of 1 or e^-4 at most
    _near(got, y, my, 0, 2.0 ** -9, "y")
    g = p.backward(dy.to(DEV), **_gpu(a))
    assert all(torch.isfinite(t).all() for t in g.values() if t is not None)
    assert torch.equal(got, p(**_gpu(a)))


# ---- together ----------------------------------------------------------------------
MIXER = dict(N=2, H=4, P=16, G=2, S=24, F=4)


def _mixer(dtype, L, seed=1):
    N, H, P, G, S, F = (MIXER[k] for k in ("N", "H", "P", "G", "S", "F"))
    W = H * P + 2 * G * S
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = TYPE[dtype]
    v = dict(u=r(N, L, W).to(t), w=(0.5 * r(W, F)).to(t), bias=(0.1 * r(W)).to(t), dt=r(N, L, H).to(t),
             A=-torch.rand(H, generator=g) * 4 - 0.1, D=r(H), dt_bias=r(H) - 2)
    cut = lambda m: (m[..., :H * P].unflatten(-1, (H, P)), m[..., H * P:H * P + G * S].unflatten(-1, (G, S)),
                     m[..., H * P + G * S:].unflatten(-1, (G, S)))
    CausalConv, SelectiveScan = _ops()
    plans = lambda n: (CausalConv({"N": N, "L": n, "C": W, "F": F}, dtype, has_bias=True, silu=True),
                       SelectiveScan({"N": N, "L": n, "H": H, "P": P, "G": G, "S": S}, dtype))
    return v, cut, plans


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens_is_the_whole_sequence(dtype):
    """A prompt of 70 tokens, its states, then 5 single tokens: the outputs and states of 75 at once."""
    v, cut, plans = _mixer(dtype, 75)
    v = _gpu(v)
    N, H, P, S = (MIXER[k] for k in ("N", "H", "P", "S"))

    def run(lo, hi, cs, ss):
        conv, scan = plans(hi - lo)
        cs2 = torch.empty_like(cs)
        ss2 = torch.empty_like(ss)
        x, B, C = cut(conv(v["u"][:, lo:hi].contiguous(), v["w"], v["bias"], state=cs, state_out=cs2))
        y = scan(x, v["dt"][:, lo:hi].contiguous(), v["A"], B, C, v["D"], v["dt_bias"], state=ss, state_out=ss2)
        return y, cs2, ss2

    cs = torch.zeros(N, MIXER["F"] - 1, v["u"].shape[2], dtype=TYPE[dtype], device=DEV)
    ss = torch.zeros(N, H, P, S, device=DEV)
    whole, cw, sw = run(0, 75, cs, ss)
    first, cs, ss = run(0, 70, cs, ss)
    ys = [first]
    conv, scan = plans(1)
    for t in range(70, 75):
        x, B, C = cut(conv.step(v["u"][:, t], v["w"], cs, v["bias"]))
        ys.append(scan.step(x, v["dt"][:, t], v["A"], B, C, ss, v["D"], v["dt_bias"])[:, None])
    got = torch.cat(ys, 1)
    assert torch.equal(cs, cw)
    # the same terms in another grouping: twice the scan's bound
    x, B, C = (m.cpu() for m in cut(conv_out(v, plans)))
    rest = dict(dt=v["dt"].cpu(), A=v["A"].cpu(), D=v["D"].cpu(), dt_bias=v["dt_bias"].cpu())
    my, ms = seq.scan(x, B=B, C=C, **rest, magnitude=True)
    _near(got, whole.cpu(), my, 2 * HALF[dtype], 2.0 ** -13, "y")
    _near(ss, sw.cpu(), ms, HALF["f32"], 2.0 ** -14, "state")


def conv_out(v, plans):
    conv, _ = plans(v["u"].shape[1])
    return conv(v["u"], v["w"], v["bias"])


def test_gradient_through_both_against_differences():
    """The two gradients chained, in fp32: along random directions they are the slope of the loss, which the
    reference evaluates in double precision on both sides of the point."""
    v, cut, plans = _mixer("f32", 40)
    conv, scan = plans(40)
    d = _gpu(v)
    N, H, P = (MIXER[k] for k in ("N", "H", "P"))
    g = torch.Generator().manual_seed(8)
    dy = torch.randn(N, 40, H, P, generator=g)
    h = conv(d["u"], d["w"], d["bias"])
    x, B, C = cut(h)
    dh = torch.empty_like(h)
    dx, dB, dC = cut(dh)
    one = scan.backward(dy.to(DEV), x, d["dt"], d["A"], B, C, d["D"], d["dt_bias"], out={"dx": dx, "dB": dB, "dC": dC})
    two = conv.backward(dh, d["u"], d["w"], d["bias"])
    grad = {"u": two["dx"], "w": two["dw"], "bias": two["dbias"], "dt": one["ddt"], "A": one["dA"], "D": one["dD"],
            "dt_bias": one["ddt_bias"]}
    grad = {k: t.cpu().double() for k, t in grad.items()}
    v = {k: t.double() for k, t in v.items()}

    def loss(s, way):
        q = {k: t + s * way[k] for k, t in v.items()}
        x, B, C = cut(seq.causal(q["u"], q["w"], q["bias"], True)[0])
        return float((seq.scan(x, q["dt"], q["A"], B, C, q["D"], q["dt_bias"])[0] * dy.double()).sum())

    eps = 1e-5
    for k in v:
        way = {j: torch.randn(t.shape, generator=g, dtype=torch.float64) * (j == k) for j, t in v.items()}
        slope = (loss(eps, way) - loss(-eps, way)) / (2 * eps)
        got = float((grad[k] * way[k]).sum())
        # fp32 gradients: 2^-13 of sums of terms that in norm are about the gradient's own
        scale = float(grad[k].norm() * way[k].norm())
        assert abs(got - slope) <= 2.0 ** -13 * scale + 1e-6 * abs(slope), (k, got, slope)


# ---- streams, graphs, determinism -----------------------------------------------------
def _everything(dtype="bf16", L=130):
    v, cut, plans = _mixer(dtype, L)
    conv, scan = plans(L)
    d = _gpu(v)
    dy = torch.randn(MIXER["N"], L, MIXER["H"], MIXER["P"], generator=torch.Generator().manual_seed(4)).to(TYPE[dtype]).to(DEV)

    def run(stream=None):
        h = conv(d["u"], d["w"], d["bias"], stream=stream)
        x, B, C = cut(h)
        y = scan(x, d["dt"], d["A"], B, C, d["D"], d["dt_bias"], stream=stream)
        dh = torch.empty_like(h)
        dx, dB, dC = cut(dh)
        one = scan.backward(dy, x, d["dt"], d["A"], B, C, d["D"], d["dt_bias"], out={"dx": dx, "dB": dB, "dC": dC},
                            stream=stream)
        two = conv.backward(dh, d["u"], d["w"], d["bias"], stream=stream)
        return [y, dh] + [one[k] for k in ("ddt", "dA", "dD", "ddt_bias")] + [two[k] for k in ("dx", "dw", "dbias")]
    return d, run


def test_same_bits_every_time_and_on_another_stream():
    _, run = _everything()
    want = run()
    again = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = run(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        inside = run()
    torch.cuda.synchronize()
    for a, b, c, e in zip(want, again, there, inside):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, e)


def test_two_streams_at_once():
    """Calls of the same plans on two streams, on other inputs: each has a workspace of its own."""
    _, one = _everything(L=200)
    _, two = _everything(L=130)
    want = [[t.clone() for t in f()] for f in (one, two)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for f, side in zip((one, two), sides):
            with torch.cuda.stream(side):
                got.append(f())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_outputs_belong_to_the_stream_that_writes_them():
    """Memory that the current stream has still to write to is not what a call on another stream returns."""
    _, run = _everything(L=200)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = torch.ones(1 << 26, device=DEV)
    late = [torch.empty_like(t) for t in want]
    for _ in range(40):
        junk.mul_(1.0)                  # some milliseconds on the current stream
    for t in late:
        t.fill_(-7.0)
    del late, t
    got = run(side)[:1]                 # y: allocated by the call
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])


def test_one_row_wider_than_32_bit_offsets_of_a_tile():
    """One token of 2^26 channels: the rows that its tile has none of lie 2^27 bytes apart.  With one token and
    one state y = (dt B C + D) x; the factor is a sum of two terms of one sign here."""
    _, SelectiveScan = _ops()
    H, P = 1024, 65536
    g = torch.Generator(device=DEV).manual_seed(3)
    u = lambda *s: (torch.rand(*s, generator=g, device=DEV) + 0.5)
    x = torch.randn(1, 1, H, P, generator=g, device=DEV, dtype=torch.bfloat16)
    dt, B, C = (u(*s).to(torch.bfloat16) for s in ((1, 1, H), (1, 1, 1, 1), (1, 1, 1, 1)))
    A, D = -u(H), u(H)
    y = SelectiveScan({"N": 1, "L": 1, "H": H, "P": P, "G": 1, "S": 1}, "bf16", softplus=False)(x, dt, A, B, C, D)
    factor = (dt.double() * B.double()[..., 0] * C.double()[..., 0] + D.double()).float()
    want = x[0, 0].float() * factor[0, 0, :, None]
    assert ((y[0, 0].float() - want).abs() <= (HALF["bf16"] * (1 + 2 ** -8) + 2.0 ** -14) * want.abs() + 1e-37).all()


def test_offsets_past_32_bits():
    """Rows a megabyte and more apart: 4.4e9 bytes of x, addressed as the packed rows are."""
    CausalConv, SelectiveScan = _ops()
    N, L, H, P, G, S, wide = 2, 1100, 1, 64, 1, 16, 1 << 20
    g = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    x, dt, B, C, w = r(N, L, H, P), r(N, L, H), r(N, L, G, S), r(N, L, G, S), r(P, 4)
    A = torch.full((H,), -1.0, device=DEV)
    far = torch.empty(N, L, wide, dtype=torch.bfloat16, device=DEV)
    fx, fB = far[..., 64:64 + P], far[..., 256:256 + S].unflatten(-1, (G, S))
    fx.copy_(x[:, :, 0]), fB.copy_(B)
    p = SelectiveScan({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, "bf16")
    y = far[..., 512:512 + P].unflatten(-1, (H, P))
    p(fx.unflatten(-1, (H, P)), dt, A, fB, C, out=y)
    want = p(x, dt, A, B, C)
    assert torch.equal(y, want)
    c = CausalConv({"N": N, "L": L, "C": P, "F": 4}, "bf16", silu=True)
    out = far[..., 1024:1024 + P]
    c(fx, w, out=out)
    assert torch.equal(out, c(x[:, :, 0].contiguous(), w))
    dx = far[..., 2048:2048 + P]
    c.backward(out, fx, w, out={"dx": dx})
    assert torch.equal(dx, c.backward(out.contiguous(), x[:, :, 0].contiguous(), w)["dx"])


def test_captured_graphs_replay():
    """Two graphs of the whole chain, captured one after the other, replayed in turns with eager work between:
    each gives its own inputs' results every time."""
    sets = [_everything(L=130), _everything(L=75)]
    eager = [[t.clone() for t in run()] for _, run in sets]
    torch.cuda.synchronize()
    graphs = []
    for _, run in sets:
        side = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = run()
        graphs.append((g, out))
    torch.cuda.synchronize()
    for turn in range(3):
        for (g, out), want, (d, run) in zip(graphs, eager, sets):
            for t in out:
                t.fill_(1.0)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), turn
            run()
            torch.cuda.synchronize()


def test_steps_in_a_graph():
    v, cut, plans = _mixer("bf16", 1)
    conv, scan = plans(1)
    d = _gpu(v)
    N, H, P, S, F = (MIXER[k] for k in ("N", "H", "P", "S", "F"))
    cs = torch.zeros(N, F - 1, d["u"].shape[2], dtype=torch.bfloat16, device=DEV)
    ss = torch.zeros(N, H, P, S, device=DEV)
    u, dt = d["u"][:, 0].contiguous(), d["dt"][:, 0].contiguous()

    def token():
        x, B, C = cut(conv.step(u, d["w"], cs, d["bias"]))
        return scan.step(x, dt, d["A"], B, C, ss, d["D"], d["dt_bias"])

    want = [token().clone() for _ in range(4)]
    cs.zero_(), ss.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        y = token()
    for t in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[t]), t


def test_refusals_on_the_gpu():
    CausalConv, SelectiveScan = _ops()
    c = CausalConv({"N": 1, "L": 4, "C": 16, "F": 4}, "bf16")
    x, w = torch.zeros(1, 4, 16, dtype=torch.bfloat16, device=DEV), torch.zeros(16, 4, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(x=x.float()), dict(x=x[:, :3]), dict(w=w.t()), dict(w=w.cpu()), dict(bias=w[:, 0].contiguous()),
                dict(lengths=torch.zeros(1, dtype=torch.int64, device=DEV)), dict(state=x), dict(out=x.float())):
        with pytest.raises(ValueError):
            c(**dict(dict(x=x, w=w), **bad))
    with pytest.raises(ValueError):
        c.backward(x, x, w, out={"dbias": w})
    from convolution_forward_implicit_amd import ConvError
    with pytest.raises(ConvError):
        c(x, w, out=x)
