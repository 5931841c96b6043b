"""Host-side tests of the group norm (conv_gnorm_*): the header, the binding and the
library agree, descriptors and calls outside the documented ranges are refused
before anything is launched, and the double-precision reference agrees with torch's
automatic differentiation.  No GPU needed."""
import ctypes
import os
import re

import pytest
import torch

from convolution_forward_implicit_amd import ConvError, GroupNorm, capi
from oracle import norm as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "convfwd.h")
INVALID, UNSUPPORTED = capi.CONV_ERR_INVALID_ARG, capi.CONV_ERR_UNSUPPORTED
DIMS = {"N": 2, "L": 10, "G": 4, "C": 16}


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_binding_and_library_agree():
    declared = sorted(set(re.findall(r"\b(conv_gnorm_\w+)\s*\(", _header())))
    assert declared == sorted(capi.GNORM_EXPORTED)
    for name in declared:
        assert hasattr(capi.lib(), name), name
    for name, value in capi.NORM_ACTS.items():
        assert re.search(r"CONV_NORM_ACT_%s = %d\b" % (name.upper(), value), _header())


@pytest.mark.parametrize("name", ["conv_gnorm_desc_t", "conv_gnorm_args_t", "conv_gnorm_bwd_args_t"])
def test_structs_match_the_header(name):
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, _header()).group(1)
    want = []
    for decl in body.split(";"):
        decl = decl.strip()
        if decl:
            typ, names = re.match(r"((?:const )?\w+)\s+(.*)", decl, re.S).groups()
            for v in names.split(","):
                want.append((v.strip().lstrip("*"), 8 if "*" in v or "64" in typ or typ == "double" else 4))
    got = getattr(capi, name)
    assert [(f, ctypes.sizeof(t)) for f, t in got._fields_] == want
    assert ctypes.sizeof(got) == sum(s for _, s in want)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(L=-1), INVALID), (dict(G=0), INVALID), (dict(C=0), INVALID), (dict(L=1 << 31), UNSUPPORTED),
    (dict(G=1 << 16, C=1 << 16), UNSUPPORTED), (dict(N=1 << 30, L=1 << 30), UNSUPPORTED)])
@pytest.mark.parametrize("per_token", [False, True])
def test_descriptors_refused(kw, status, per_token):
    with pytest.raises(ConvError) as e:
        GroupNorm(dict(DIMS, **kw), "bf16", per_token=per_token)
    assert e.value.status == status


def test_flags_types_and_eps_refused():
    d = capi.conv_gnorm_desc_t
    good = [0, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1e-5]
    for at, bad in ((0, 5), (1, 3), (1, -1), (2, 2), (3, -1), (4, 2), (5, 7), (10, -1e-9), (10, float("nan")), (10, 1e39)):
        with pytest.raises(ConvError) as e:
            capi.conv_gnorm_create(d(*(good[:at] + [bad] + good[at + 1:])))
        assert e.value.status == INVALID
    with pytest.raises(ValueError, match="act"):
        GroupNorm(DIMS, "bf16", act="relu")
    assert capi.lib().conv_gnorm_create(None, None) == INVALID
    assert capi.lib().conv_gnorm_run(None, None, None, 0, None) == INVALID
    assert capi.lib().conv_gnorm_bwd_run(None, None, None, 0, None) == INVALID


def _refused(call, words, status=INVALID):
    with pytest.raises(ConvError) as e:
        call()
    assert e.value.status == status and words in e.value.message, e.value.message


def test_calls_refused_before_a_launch():
    """Addresses are never followed: the checks come first."""
    p = GroupNorm(DIMS, "bf16", act="silu", has_bias=True, gated=True)
    M = 1 << 20
    good = dict(x=M, w=2 * M, bias=3 * M, gate=4 * M, y=5 * M)
    run = lambda q=p, ws=64 * M, n=p.workspace_bytes, **kw: capi.conv_gnorm_run(
        q._plan, ctypes.byref(capi.conv_gnorm_args_t(**dict(good, **kw))), ws, n)
    assert p.workspace_bytes > 0
    for k in good:
        _refused(lambda: run(**{k: None}), k)
        _refused(lambda: run(**{k: 16 * M + 1}), "aligned")
    _refused(lambda: run(lengths=16 * M + 2), "aligned")
    _refused(lambda: run(x_ld=63), "x:")
    _refused(lambda: run(gate_ld=-64), "gate:")
    _refused(lambda: run(y_ld=1 << 24), "token to token", UNSUPPORTED)
    _refused(lambda: run(y=M), "y overlaps x")
    _refused(lambda: run(y=M + 2 * 40, x_ld=128, y_ld=128), "y overlaps x")
    _refused(lambda: run(ws=None), "workspace is NULL")
    _refused(lambda: run(n=p.workspace_bytes - 1), "workspace has")
    _refused(lambda: run(ws=64 * M + 8), "16-byte")
    _refused(lambda: run(ws=5 * M), "workspace overlaps")
    bare = GroupNorm(DIMS, "bf16")
    _refused(lambda: run(bare, bias=None), "no gate")
    _refused(lambda: run(bare, gate=None), "no bias")
    bgood = dict(good, dy=6 * M, dx=7 * M, dw=8 * M, dbias=9 * M, dgate=10 * M)
    del bgood["y"]
    need = p.bwd_workspace_bytes
    bwd = lambda ws=64 * M, n=need, **kw: capi.conv_gnorm_bwd_run(
        p._plan, ctypes.byref(capi.conv_gnorm_bwd_args_t(**dict(bgood, **kw))), ws, n)
    for k in bgood:
        _refused(lambda: bwd(**{k: None}), k)
    _refused(lambda: bwd(n=need - 1), "workspace has")
    _refused(lambda: bwd(dgate=7 * M), "dgate overlaps dx")
    _refused(lambda: bwd(dx=6 * M), "dx overlaps dy")
    _refused(lambda: bwd(ws=8 * M), "workspace overlaps")


def test_python_calls_refuse_tensors():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda"):
        GroupNorm(DIMS, "bf16")(z(2, 10, 4, 16), z(4, 16))


def test_nothing_to_do_is_no_error():
    p = GroupNorm(dict(DIMS, N=0), "f32")
    assert p.workspace_bytes == 0
    capi.conv_gnorm_run(p._plan, ctypes.byref(capi.conv_gnorm_args_t(w=16)), None, 0)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("per_token,lengths", [(False, None), (False, [5, 2]), (True, [0, 4]), (True, None)])
def test_reference_gradient_is_autograds(act, gated, center, per_token, lengths):
    g = torch.Generator().manual_seed(0)
    N, L, G, C = 2, 5, 2, 6
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, w, b, z, dy = r(N, L, G, C) + 1, r(G, C), r(G, C), r(N, L, G, C), r(N, L, G, C)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    kw = dict(lengths=n, act=act, center=center, per_token=per_token)
    got, _ = ref.norm_grad(dy, x, w, b, z if gated else None, **kw)
    f = {"none": lambda v: v, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    ins = [t.requires_grad_() for t in (x, w, b, z)]
    rows = []
    for i in range(N):
        m = L if n is None else int(n[i])
        xi = x[i, :m]
        dims = (-1,) if per_token else (0, 2)
        if m:
            xi = xi - xi.mean(dims, keepdim=True) if center else xi
            xi = xi / (xi.square().mean(dims, keepdim=True) + 1e-5).sqrt()
        v = xi * w + b
        y = v * f(z[i, :m]) if gated else f(v)
        rows.append(torch.cat([y, torch.zeros(L - m, G, C, dtype=torch.float64)]))
    y = torch.stack(rows)
    assert (ref.norm(x.detach(), w.detach(), b.detach(), z.detach() if gated else None, **kw)[0] - y).abs().max() <= 1e-13
    y.backward(dy)
    for t, k in zip(ins, ("dx", "dw", "dbias", "dgate")):
        want = torch.zeros_like(t) if t.grad is None else t.grad
        assert (want - got[k]).abs().max() <= 1e-12, k
