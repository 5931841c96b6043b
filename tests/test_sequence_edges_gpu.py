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


# ---- plans of large problems, at small cost -------------------------------------
# Heads are repeated: the reference computes `heads` of them, the kernels `times` as many in the same groups, whose
# copies must come out with the same bits.  Bounds as in test_sequence_gpu.py, whose helpers these are.
def _repeated(N, L, heads, times, P, G, S, dtype, seed):
    from test_sequence_gpu import _scan_case as case
    a, dy, dlast, _ = case(N, L, heads, P, G, S, dtype, True, None, seed)
    # group by group: the heads of a group are its own and their copies
    more = lambda v, d: v.unflatten(d, (G, heads // G)).repeat_interleave(times, d).flatten(d, d + 1) if v is not None else v
    wide = dict(a, **{k: more(a[k], {"x": 2, "dt": 2, "state": 1}.get(k, 0)) for k in ("x", "dt", "A", "D", "dt_bias", "state")})
    return a, wide, dy, more(dy, 2), dlast, more(dlast, 1)


def _check_forward(dims, times, dtype, lengths, what):
    from test_sequence_gpu import _near as near
    N, L, heads, P, G, S = dims
    a, wide, *_ = _repeated(N, L, heads, times, P, G, S, dtype, 41)
    p = _scan(N, L, heads * times, P, G, S, dtype)
    assert what(p.describe()), p.describe()
    n = torch.tensor(lengths, dtype=torch.int32)
    out = torch.full((N, heads * times, P, S), 7.0, device=DEV)
    y = p(**_gpu(wide), lengths=n.to(DEV), state_out=out)
    pick = torch.arange(G)[:, None] * (heads // G * times) + torch.arange(heads // G)[None]
    first = pick.flatten().to(DEV)
    for k in range(times):
        at = first + k * (heads // G)
        assert torch.equal(y[:, :, at], y[:, :, first]) and torch.equal(out[:, at], out[:, first]), k
    want, last = seq.scan(**a, lengths=n)
    my, ml = seq.scan(**a, lengths=n, magnitude=True)
    near(y[:, :, first], want, my, HALF[dtype], 2.0 ** -14, "y")
    near(out[:, first], last, ml, HALF["f32"], 2.0 ** -15, "state_out")


def test_two_state_segments_a_forward_workgroup():
    """The plan of long sequences of few heads: a workgroup's chunks are two segments of the pass over the states.
    One sequence ends within the first of the two."""
    _check_forward((2, 4100, 8, 8, 2, 16), 8, "bf16", [4100, 2500], lambda t: "(2 x 2 of whole bf16 vectors)" in t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [128, 64])
def test_many_chunks_of_whole_heads(S, dtype):
    """Heads of 64 channels over all chunks of the sequence in one workgroup, full and ragged."""
    one = "in 1 segments (1 x 1" if dtype == "bf16" else "in "
    _check_forward((2, 330, 5, 64, 1, S), 26, dtype, [330, 170], lambda t: one in t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims,times,lengths", [((2, 330, 5, 64, 1, 128), 13, [330, 170]), ((4, 70, 8, 72, 4, 16), 8, [70, 0, 33, 65]),
                                                ((2, 140, 2, 130, 1, 40), 24, [140, 77])], ids=str)
def test_gradient_of_several_heads_a_workgroup(dims, times, lengths, dtype):
    """... of more than 64 states, and of more than one block of 64 channels each."""
    from test_sequence_gpu import _around, _near as near
    N, L, heads, P, G, S = dims
    a, wide, dy, wdy, dlast, wlast = _repeated(N, L, heads, times, P, G, S, dtype, 43)
    p = _scan(N, L, heads * times, P, G, S, dtype)
    assert int(p.describe().split("slices of ")[1].split()[0]) > 1, p.describe()
    n = torch.tensor(lengths, dtype=torch.int32)
    got = p.backward(wdy.to(DEV), **_gpu(wide), lengths=n.to(DEV), dstate_out=wlast.to(DEV))
    kw = dict(a, lengths=n, dstate_out=dlast)
    want, mag = seq.scan_grad(dy, **kw), seq.scan_grad(dy, **kw, magnitude=True)
    my, _ = seq.scan(**a, lengths=n, magnitude=True)
    around = _around((dy.double().abs() * my).sum(-1) + mag["step"] * mag["e"]) + mag["dl"]
    mag["ddt"] = around * a["A"].double().abs() + mag["e"]
    mag["dA"] = (around * mag["step"]).sum((0, 1))
    mag["ddt_bias"] = mag["ddt"].sum((0, 1))
    first = (torch.arange(G)[:, None] * (heads // G * times) + torch.arange(heads // G)[None]).flatten().to(DEV)
    for k, v in got.items():
        if k in ("dB", "dC"):       # over the heads: every copy's
            near(v, want[k] * times, mag[k] * times, HALF[dtype], 2.0 ** -13, k)
            continue
        d = {"dx": 2, "ddt": 2, "dstate": 1}.get(k, 0)
        for i in range(1, times):
            assert torch.equal(v.index_select(d, first + i * (heads // G)), v.index_select(d, first)), (k, i)
        near(v.index_select(d, first), want[k], mag[k], HALF[dtype] if k in ("dx", "ddt") else HALF["f32"], 2.0 ** -13, k)


# ---- the convolution's forms ------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,C,F,bias,silu,apart", [
    (1, 1, 2, False, False, False), (3, 64, 4, True, True, True), (5, 37, 4, True, False, False), (2, 520, 8, False, True, True),
    (4, 24, 3, True, True, False), (7, 130, 5, False, False, True), (1, 2304, 4, True, True, False), (2, 9, 7, True, True, True),
    (3, 48, 6, False, True, False)])
def test_convolution_step(N, C, F, bias, silu, apart, dtype):
    """Every tap count, vectors and single channels, in place and apart, x and y as columns of wider rows.  Bound: F
    products and sums in fp32 and the sigmoid, 2^-20 of the terms."""
    import ctypes
    from convolution_forward_implicit_amd import capi
    from test_sequence_gpu import _near as near
    g = torch.Generator().manual_seed(50 + F)
    t = TYPE[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(t)
    x, w, b, state = r(N, C), r(C, F), r(C) if bias else None, r(N, F - 1, C)
    p = _conv(N, 1, C, F, dtype, has_bias=bias, silu=silu)
    want, last, _ = seq.causal(x[:, None], w, b, silu, state)
    mag = seq.causal(x[:, None].abs(), w.abs(), None if b is None else b.abs(), False, state.abs())[0]
    for wide, lo in ((C, 0), (2 * C + 16, 8), (2 * C + 5, 3)):
        rows = torch.full((N, wide), 5.0, dtype=t, device=DEV)
        rows[:, lo:lo + C] = x.to(DEV)
        into = torch.full((N, wide), 9.0, dtype=t, device=DEV)
        v = _gpu(dict(w=w, b=b, state=state))
        if apart:
            out = torch.full_like(v["state"], 7.0)
            e = rows.element_size()
            args = capi.conv_causal_args_t(rows.data_ptr() + lo * e, v["w"].data_ptr(), v["b"].data_ptr() if bias else None,
                                           v["state"].data_ptr(), None, into.data_ptr() + lo * e, out.data_ptr(), wide, wide)
            capi.conv_causal_step(p._plan, ctypes.byref(args), torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(v["state"].cpu(), state)
        else:
            out = v["state"]
            p.step(rows[:, lo:lo + C], v["w"], out, v["b"], out=into[:, lo:lo + C])
        near(into[:, lo:lo + C], want[:, 0], mag[:, 0], HALF[dtype], 2.0 ** -20, "y")
        assert torch.equal(out.cpu(), last.to(t))
        assert (into[:, :lo] == 9).all() and (into[:, lo + C:] == 9).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [40, 19])
def test_convolution_without_a_bias_and_lengths_out_of_range(C, dtype):
    """Lengths outside 0..L are the nearer end."""
    from test_sequence_gpu import _near as near
    g = torch.Generator().manual_seed(60)
    N, L, F, t = 3, 30, 4, TYPE[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(t)
    a, dy = dict(x=r(N, L, C), w=r(C, F), bias=None, state=r(N, F - 1, C)), r(N, L, C)
    n = torch.tensor([-3, L + 5, 11], dtype=torch.int32)
    p = _conv(N, L, C, F, dtype)
    out = torch.full((N, F - 1, C), 7.0, dtype=t, device=DEV)
    y = p(**_gpu(a), lengths=n.to(DEV), state_out=out)
    want, last, _ = seq.causal(**a, silu=False, lengths=n)
    near(y, want, seq.causal(a["x"].abs(), a["w"].abs(), None, False, a["state"].abs(), n)[0], HALF[dtype], 2.0 ** -20, "y")
    assert torch.equal(out.cpu(), last.to(t))
    got = p.backward(dy.to(DEV), **_gpu(a), lengths=n.to(DEV))
    assert got["dbias"] is None
    want, mag = (seq.causal_grad(dy, **a, silu=False, lengths=n, magnitude=m) for m in (False, True))
    for k in ("dx", "dw", "dstate"):
        near(got[k], want[k], mag[k], HALF[dtype], 2.0 ** -17, k)
