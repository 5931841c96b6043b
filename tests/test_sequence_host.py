"""Host-side tests of the sequence operators (conv_causal_*, conv_scan_*): the
header, the binding and the library agree, descriptors and calls outside the
documented ranges are refused before anything is launched, and the
double-precision reference agrees with torch's automatic differentiation and
with differences.  No GPU needed."""
import ctypes
import os
import re

import pytest
import torch

from convolution_forward_implicit_amd import CausalConv, ConvError, SelectiveScan, capi
from oracle import seq

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "convfwd.h")
INVALID, UNSUPPORTED = capi.CONV_ERR_INVALID_ARG, capi.CONV_ERR_UNSUPPORTED


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_binding_and_library_agree():
    declared = sorted(set(re.findall(r"\b(conv_(?:causal|scan)_\w+)\s*\(", _header())))
    assert declared == sorted(capi.SEQUENCE_EXPORTED)
    for name in declared:
        assert hasattr(capi.lib(), name), name


@pytest.mark.parametrize("name", ["conv_causal_desc_t", "conv_causal_args_t", "conv_causal_bwd_args_t",
                                  "conv_scan_desc_t", "conv_scan_args_t", "conv_scan_bwd_args_t"])
def test_structs_match_the_header(name):
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, _header()).group(1)
    want = []
    for decl in body.split(";"):
        decl = decl.strip()
        if decl:
            typ, names = re.match(r"((?:const )?\w+)\s+(.*)", decl, re.S).groups()
            for v in names.split(","):
                want.append((v.strip().lstrip("*"), 8 if "*" in v or "64" in typ else 4))
    got = getattr(capi, name)
    assert [(f, ctypes.sizeof(t)) for f, t in got._fields_] == want
    assert ctypes.sizeof(got) == sum(s for _, s in want)


CONV = {"N": 2, "L": 10, "C": 16, "F": 4}
SCAN = {"N": 2, "L": 10, "H": 4, "P": 16, "G": 2, "S": 16}


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(L=-1), INVALID), (dict(C=0), INVALID), (dict(F=1), INVALID), (dict(F=9), UNSUPPORTED),
    (dict(N=1 << 31), UNSUPPORTED), (dict(N=1 << 20, L=1 << 20, C=1 << 20), UNSUPPORTED)])
def test_causal_descriptors_refused(kw, status):
    with pytest.raises(ConvError) as e:
        CausalConv(dict(CONV, **kw), "bf16")
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(L=-1), INVALID), (dict(H=0), INVALID), (dict(P=0), INVALID), (dict(G=0), INVALID),
    (dict(S=0), INVALID), (dict(G=3), INVALID), (dict(S=129), UNSUPPORTED), (dict(P=65537), UNSUPPORTED),
    (dict(L=1 << 31), UNSUPPORTED), (dict(N=1 << 12, L=1 << 22, H=1 << 20, G=1), UNSUPPORTED)])
def test_scan_descriptors_refused(kw, status):
    with pytest.raises(ConvError) as e:
        SelectiveScan(dict(SCAN, **kw), "bf16")
    assert e.value.status == status


def test_flags_and_dtypes_refused():
    for desc, create in ((capi.conv_causal_desc_t(7, 0, 0, 0, 1, 1, 1, 2), capi.conv_causal_create),
                         (capi.conv_causal_desc_t(0, 2, 0, 0, 1, 1, 1, 2), capi.conv_causal_create),
                         (capi.conv_causal_desc_t(0, 0, 3, 0, 1, 1, 1, 2), capi.conv_causal_create),
                         (capi.conv_causal_desc_t(0, 0, 0, 1, 1, 1, 1, 2), capi.conv_causal_create),
                         (capi.conv_scan_desc_t(5, 0, 1, 1, 1, 1, 1, 1), capi.conv_scan_create),
                         (capi.conv_scan_desc_t(0, 2, 1, 1, 1, 1, 1, 1), capi.conv_scan_create)):
        with pytest.raises(ConvError) as e:
            create(desc)
        assert e.value.status == INVALID
    assert capi.lib().conv_scan_create(None, None) == INVALID
    assert capi.lib().conv_causal_run(None, None, None) == INVALID
    assert capi.lib().conv_scan_bwd_run(None, None, None, 0, None) == INVALID


def _refused(call, words, status=INVALID):
    with pytest.raises(ConvError) as e:
        call()
    assert e.value.status == status and words in e.value.message, e.value.message


def test_causal_calls_refused_before_a_launch():
    """Addresses are never followed: the checks come first."""
    p = CausalConv(CONV, "bf16", has_bias=True)
    M = 1 << 20
    good = dict(x=M, w=2 * M, bias=3 * M, y=4 * M, state=5 * M, state_out=6 * M)
    run = lambda **kw: capi.conv_causal_run(p._plan, ctypes.byref(capi.conv_causal_args_t(**dict(good, **kw))))
    step = lambda **kw: capi.conv_causal_step(p._plan, ctypes.byref(capi.conv_causal_args_t(**dict(good, **kw))))
    _refused(lambda: run(x=None), "NULL")
    _refused(lambda: run(w=None), "NULL")
    _refused(lambda: run(bias=None), "bias")
    _refused(lambda: run(x=M + 1), "aligned")
    _refused(lambda: run(x_ld=15), "x:")
    _refused(lambda: run(y_ld=-16), "y:")
    _refused(lambda: run(y=M + 32), "y overlaps x")
    _refused(lambda: run(state_out=5 * M), "state_out overlaps state")
    _refused(lambda: run(x_ld=40, y=M + 16, y_ld=40), "y overlaps x")
    _refused(lambda: run(x_ld=1 << 62), "token to token", UNSUPPORTED)
    _refused(lambda: step(state=None), "state")
    _refused(lambda: step(lengths=7 * M), "lengths")
    _refused(lambda: step(state_out=5 * M + 2), "state_out overlaps state")
    bgood = dict(dy=M, x=2 * M, w=3 * M, bias=4 * M, dx=5 * M, dw=6 * M, dbias=7 * M)
    need = p.bwd_workspace_bytes
    bwd = lambda ws=8 * M, n=need, **kw: capi.conv_causal_bwd_run(
        p._plan, ctypes.byref(capi.conv_causal_bwd_args_t(**dict(bgood, **kw))), ws, n)
    _refused(lambda: bwd(n=need - 1), "workspace has")
    _refused(lambda: bwd(ws=None), "workspace is NULL")
    _refused(lambda: bwd(ws=8 * M + 4), "16-byte")
    _refused(lambda: bwd(ws=5 * M), "workspace overlaps")
    _refused(lambda: bwd(dw=None), "dw")
    _refused(lambda: bwd(dbias=None), "dbias")
    _refused(lambda: bwd(dstate=9 * M), "dstate")
    _refused(lambda: bwd(dx=2 * M), "dx overlaps x")


def test_scan_calls_refused_before_a_launch():
    p = SelectiveScan(SCAN, "bf16")
    M = 1 << 20
    good = dict(x=M, dt=2 * M, a=3 * M, b=4 * M, c=5 * M, y=6 * M, state=7 * M, state_out=8 * M)
    call = lambda f, kw: f(p._plan, ctypes.byref(capi.conv_scan_args_t(**dict(good, **kw))))
    run = lambda ws=32 * M, n=p.workspace_bytes, **kw: call(lambda q, a: capi.conv_scan_run(q, a, ws, n), kw)
    step = lambda **kw: call(capi.conv_scan_step, kw)
    _refused(lambda: run(a=None), "a is NULL")
    for k in ("x", "dt", "b", "c", "y"):
        _refused(lambda: run(**{k: None}), "NULL")
        _refused(lambda: run(**{k: M * 16 + 1}), "aligned")
    _refused(lambda: run(dt_bias=9 * M + 2), "aligned")
    _refused(lambda: run(b_ld=31), "b:")
    _refused(lambda: run(y=M), "y overlaps x")
    _refused(lambda: run(state_out=7 * M + 64), "state_out overlaps state")
    # y as a column range of x's rows: refused where they meet
    _refused(lambda: run(x_ld=256, y=M + 2 * 40, y_ld=256), "y overlaps x")
    _refused(lambda: step(state_out=None), "state")
    _refused(lambda: step(lengths=9 * M), "lengths")
    _refused(lambda: step(state_out=7 * M + 64), "state_out overlaps state")
    bgood = dict(good, dy=9 * M, dx=10 * M, ddt=11 * M, da=12 * M, db=13 * M, dc=14 * M)
    for k in ("y", "state_out"):
        del bgood[k]
    need = p.bwd_workspace_bytes
    bwd = lambda ws=32 * M, n=need, **kw: capi.conv_scan_bwd_run(
        p._plan, ctypes.byref(capi.conv_scan_bwd_args_t(**dict(bgood, **kw))), ws, n)
    _refused(lambda: bwd(n=need - 1), "workspace has")
    _refused(lambda: bwd(d=15 * M), "dd must be")
    _refused(lambda: bwd(ddt_bias=15 * M), "ddt_bias")
    _refused(lambda: bwd(da=None), "da")
    _refused(lambda: bwd(dx=9 * M), "dx overlaps dy")
    _refused(lambda: bwd(db=10 * M), "db overlaps dx")
    _refused(lambda: bwd(ws=13 * M), "workspace overlaps")


def test_python_calls_refuse_tensors():
    """What the classes check before the library does, on CPU tensors."""
    c = CausalConv(CONV, "bf16")
    with pytest.raises(ValueError, match="cuda"):
        c(torch.zeros(2, 10, 16, dtype=torch.bfloat16), torch.zeros(16, 4, dtype=torch.bfloat16))
    s = SelectiveScan(SCAN, "bf16")
    rows = lambda t, inner: s._rows(t, (2, 10), inner, torch.bfloat16, torch.device("cpu"), "x")
    with pytest.raises(ValueError, match="cuda"):
        rows(torch.zeros(2, 10, 4, 16, dtype=torch.bfloat16), (4, 16))


def test_python_rows_accepts_column_ranges_only():
    """Strides, with a stand-in for a cuda tensor's device."""
    class Device(str):
        type, index = "cuda", 0

    class View:
        def __init__(self, t):
            self.t, self.dtype, self.shape, self.device = t, t.dtype, t.shape, Device("cuda:0")
            self.is_contiguous, self.stride, self.data_ptr = t.is_contiguous, t.stride, t.data_ptr
            self.is_cuda, self.get_device = True, lambda: 0

    s = SelectiveScan(SCAN, "f32")
    rows = lambda t, lead, inner: s._rows(View(t), lead, inner, torch.float32, Device("cuda:0"), "x")[1]
    wide = torch.zeros(2, 10, 100)
    assert rows(torch.zeros(2, 10, 4, 16), (2, 10), (4, 16)) == 0
    assert rows(wide[..., 20:84].unflatten(-1, (4, 16)), (2, 10), (4, 16)) == 100
    assert rows(wide[:, :1, 20:84].unflatten(-1, (4, 16)), (2, 1), (4, 16)) == 1000
    assert rows(wide[:1, :, 20:84].unflatten(-1, (4, 16)), (1, 10), (4, 16)) == 100
    for bad, lead in ((wide[:, ::2, :64].unflatten(-1, (4, 16))[:, :5], None), (wide[:, :9, :64].unflatten(-1, (4, 16)), (2, 9)),
                      (torch.zeros(2, 10, 1, 16).expand(2, 10, 4, 16), (2, 10)),
                      (torch.zeros(2, 10, 16, 4).transpose(2, 3), (2, 10)),
                      (torch.zeros(1, 1, 64).expand(2, 10, 64).unflatten(-1, (4, 16)), (2, 10)),
                      (torch.zeros(10, 2, 4, 16).transpose(0, 1), (2, 10))):
        if lead is None:
            assert rows(bad, (2, 5), (4, 16)) == 200          # every second token: evenly spaced all the same
            continue
        with pytest.raises(ValueError):
            rows(bad, lead, (4, 16))


# ---- the reference ---------------------------------------------------------------
def _scan_case(seed, N=2, L=7, H=4, P=3, G=2, S=5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    return dict(x=r(N, L, H, P), dt=r(N, L, H), A=-torch.rand(H, generator=g, dtype=torch.float64) * 3, B=r(N, L, G, S),
                C=r(N, L, G, S), D=r(H), dt_bias=r(H), state=r(N, H, P, S)), dict(dy=r(N, L, H, P), dstate_out=r(N, H, P, S))


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [7, 3], [0, 1]])
def test_reference_scan_gradient_is_autograds(softplus, lengths):
    a, o = _scan_case(3)
    leaves = {k: v.clone().requires_grad_() for k, v in a.items()}
    y, st = seq.scan(**leaves, softplus=softplus, lengths=lengths)
    ((y * o["dy"]).sum() + (st * o["dstate_out"]).sum()).backward()
    got = seq.scan_grad(o["dy"], **a, softplus=softplus, lengths=lengths, dstate_out=o["dstate_out"])
    for k, v in leaves.items():
        want = v.grad if v.grad is not None else torch.zeros_like(v)
        torch.testing.assert_close(got["d" + k], want, rtol=1e-11, atol=1e-11)


def test_reference_scan_gradient_is_the_difference_quotient():
    a, o = _scan_case(5)
    g = torch.Generator().manual_seed(9)
    way = {k: torch.randn(v.shape, generator=g, dtype=torch.float64) for k, v in a.items()}
    loss = lambda s: sum((p * q).sum() for p, q in zip(seq.scan(**{k: v + s * way[k] for k, v in a.items()}),
                                                       (o["dy"], o["dstate_out"])))
    grad = seq.scan_grad(o["dy"], **a, dstate_out=o["dstate_out"])
    slope = sum((grad["d" + k] * way[k]).sum() for k in a)
    eps = 1e-5     # central differences: error eps^2 times a third derivative, and 1e-16 / eps
    torch.testing.assert_close((loss(eps) - loss(-eps)) / (2 * eps), slope, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lengths", [None, [6, 2], [0, 1]])
def test_reference_convolution_gradient_is_autograds(silu, lengths):
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    a = dict(x=r(2, 6, 5), w=r(5, 4), bias=r(5), state=r(2, 3, 5))
    dy, last = r(2, 6, 5), r(2, 3, 5)
    leaves = {k: v.clone().requires_grad_() for k, v in a.items()}
    y, st, _ = seq.causal(**leaves, silu=silu, lengths=lengths)
    ((y * dy).sum() + (st * last).sum()).backward()
    got = seq.causal_grad(dy, **a, silu=silu, lengths=lengths, dstate_out=last)
    for k, v in leaves.items():
        want = v.grad if v.grad is not None else torch.zeros_like(v)
        torch.testing.assert_close(got["d" + k], want, rtol=1e-11, atol=1e-11)


def test_reference_convolution_is_torchs():
    g = torch.Generator().manual_seed(6)
    x, w, b = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((2, 9, 5), (5, 3), (5,)))
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (2, 0)), w[:, None], b, groups=5)
    torch.testing.assert_close(seq.causal(x, w, b, False)[0], want.transpose(1, 2))
