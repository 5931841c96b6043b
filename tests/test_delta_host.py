"""Host-side tests of the gated delta rule (conv_delta_*): the header, the binding
and the library agree, descriptors and calls outside the documented ranges are
refused before anything is launched, and the double-precision reference agrees with
torch's automatic differentiation.  No GPU needed."""
import ctypes
import os
import re

import pytest
import torch

from convolution_forward_implicit_amd import ConvError, DeltaRule, capi
from oracle import delta as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "convfwd.h")
INVALID, UNSUPPORTED = capi.CONV_ERR_INVALID_ARG, capi.CONV_ERR_UNSUPPORTED
DIMS = {"N": 2, "L": 10, "H": 4, "P": 16, "G": 2, "S": 16}


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_binding_and_library_agree():
    declared = sorted(set(re.findall(r"\b(conv_delta_\w+)\s*\(", _header())))
    assert declared == sorted(capi.DELTA_EXPORTED)
    for name in declared:
        assert hasattr(capi.lib(), name), name


@pytest.mark.parametrize("name", ["conv_delta_desc_t", "conv_delta_args_t", "conv_delta_bwd_args_t"])
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
    (dict(N=-1), INVALID), (dict(L=-1), INVALID), (dict(H=0), INVALID), (dict(P=0), INVALID), (dict(G=0), INVALID),
    (dict(S=0), INVALID), (dict(G=3), INVALID), (dict(S=257), UNSUPPORTED), (dict(P=65537), UNSUPPORTED),
    (dict(L=1 << 31), UNSUPPORTED), (dict(N=1 << 12, L=1 << 22, H=1 << 20, G=1), UNSUPPORTED)])
def test_descriptors_refused(kw, status):
    with pytest.raises(ConvError) as e:
        DeltaRule(dict(DIMS, **kw), "bf16")
    assert e.value.status == status


def test_flags_dtypes_and_scales_refused():
    d = capi.conv_delta_desc_t
    for desc in (d(5, 0, 1, 1, 1, 1, 1, 1, 1.0), d(0, 1, 1, 1, 1, 1, 1, 1, 1.0), d(0, 0, 1, 1, 1, 1, 1, 1, float("nan")),
                 d(0, 0, 1, 1, 1, 1, 1, 1, 1e39), d(0, 0, 1, 1, 1, 1, 1, 1, -float("inf"))):
        with pytest.raises(ConvError) as e:
            capi.conv_delta_create(desc)
        assert e.value.status == INVALID
    assert capi.lib().conv_delta_create(None, None) == INVALID
    assert capi.lib().conv_delta_run(None, None, None, 0, None) == INVALID
    assert capi.lib().conv_delta_step(None, None, None) == INVALID
    assert capi.lib().conv_delta_bwd_run(None, None, None, 0, None) == INVALID


def _refused(call, words, status=INVALID):
    with pytest.raises(ConvError) as e:
        call()
    assert e.value.status == status and words in e.value.message, e.value.message


def test_calls_refused_before_a_launch():
    """Addresses are never followed: the checks come first."""
    p = DeltaRule(DIMS, "bf16")
    M = 1 << 24
    good = dict(q=M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, y=6 * M, state=7 * M, state_out=8 * M)
    call = lambda f, kw: f(p._plan, ctypes.byref(capi.conv_delta_args_t(**dict(good, **kw))))
    run = lambda ws=64 * M, n=p.workspace_bytes, **kw: call(lambda q, a: capi.conv_delta_run(q, a, ws, n), kw)
    step = lambda **kw: call(capi.conv_delta_step, kw)
    for k in ("q", "k", "v", "g", "beta", "y"):
        _refused(lambda: run(**{k: None}), "NULL")
        _refused(lambda: run(**{k: 16 * M + 1}), "aligned")
    _refused(lambda: run(state=16 * M + 2), "aligned")
    _refused(lambda: run(k_ld=31), "k:")
    _refused(lambda: run(q_ld=1 << 24), "token to token", UNSUPPORTED)
    _refused(lambda: run(y=3 * M), "y overlaps v")
    _refused(lambda: run(y=3 * M + 2 * 40, v_ld=256, y_ld=256), "y overlaps v")
    _refused(lambda: run(state_out=7 * M + 64), "state_out overlaps state")
    _refused(lambda: run(n=p.workspace_bytes - 1), "workspace has")
    _refused(lambda: run(ws=None), "workspace is NULL")
    _refused(lambda: run(ws=64 * M + 8), "16-byte")
    _refused(lambda: run(ws=6 * M), "workspace overlaps")
    _refused(lambda: step(state_out=None), "state")
    _refused(lambda: step(lengths=9 * M), "lengths")
    _refused(lambda: step(state_out=7 * M + 64), "state_out overlaps state")
    bgood = dict(good, dy=9 * M, dq=10 * M, dk=11 * M, dv=12 * M, dg=13 * M, dbeta=14 * M)
    for k in ("y", "state_out"):
        del bgood[k]
    need = p.bwd_workspace_bytes
    bwd = lambda ws=64 * M, n=need, **kw: capi.conv_delta_bwd_run(
        p._plan, ctypes.byref(capi.conv_delta_bwd_args_t(**dict(bgood, **kw))), ws, n)
    for k in ("dy", "q", "k", "v", "g", "beta", "dq", "dk", "dv", "dg", "dbeta"):
        _refused(lambda: bwd(**{k: None}), "NULL")
    _refused(lambda: bwd(n=need - 1), "workspace has")
    _refused(lambda: bwd(state=None, dstate=15 * M), "dstate without")
    _refused(lambda: bwd(dv=9 * M), "dv overlaps dy")
    _refused(lambda: bwd(dk=10 * M), "dk overlaps dq")
    _refused(lambda: bwd(ws=13 * M), "workspace overlaps")


def test_nothing_to_do_is_no_error():
    p = DeltaRule(dict(DIMS, N=0), "f32")
    capi.conv_delta_run(p._plan, ctypes.byref(capi.conv_delta_args_t()), None, 0)
    capi.conv_delta_step(p._plan, ctypes.byref(capi.conv_delta_args_t()))
    capi.conv_delta_bwd_run(p._plan, ctypes.byref(capi.conv_delta_bwd_args_t()), None, 0)
    p = DeltaRule(dict(DIMS, L=0), "f32")
    assert p.workspace_bytes == 0 and p.bwd_workspace_bytes == 0
    capi.conv_delta_run(p._plan, ctypes.byref(capi.conv_delta_args_t()), None, 0)


def test_python_calls_refuse_tensors():
    p = DeltaRule(DIMS, "bf16")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda"):
        p(z(2, 10, 2, 16), z(2, 10, 2, 16), z(2, 10, 4, 16), torch.zeros(2, 10, 4), z(2, 10, 4))
    assert p.scale == 0.25 and DeltaRule(DIMS, "f32", scale=3).scale == 3.0


@pytest.mark.parametrize("lengths", [None, [9, 4], [0, 9]])
def test_reference_gradient_is_autograds(lengths):
    g = torch.Generator().manual_seed(0)
    N, L, H, P, G, S = 2, 9, 4, 3, 2, 5
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()
    q, k, v, s = unit(r(N, L, G, S)), unit(r(N, L, G, S)), r(N, L, H, P), r(N, H, P, S)
    gg, b = -r(N, L, H).abs(), r(N, L, H).abs().clamp(max=1.5)
    dy, dl = r(N, L, H, P), r(N, H, P, S)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    ins = [x.requires_grad_() for x in (q, k, v, gg, b, s)]
    y, last, loss = torch.zeros(N, L, H, P, dtype=torch.float64), [], 0
    for i in range(N):
        St = s[i]
        for t in range(L if n is None else int(n[i])):
            kk, qq = k[i, t].repeat_interleave(H // G, 0), q[i, t].repeat_interleave(H // G, 0)
            St = St * gg[i, t].exp()[:, None, None]
            e = v[i, t] - (St * kk[:, None]).sum(-1)
            St = St + (b[i, t][:, None] * e)[..., None] * kk[:, None]
            y[i, t] = 0.3 * (St * qq[:, None]).sum(-1).detach()
            loss = loss + 0.3 * ((St * qq[:, None]).sum(-1) * dy[i, t]).sum()
        loss = loss + (St * dl[i]).sum()
        last.append(St.detach())
    want = torch.autograd.grad(loss, ins)
    data = [x.detach() for x in (q, k, v, gg, b)]
    got, _ = ref.delta_grad(dy, *data, 0.3, state=s.detach(), lengths=n, dstate_out=dl)
    for w, name in zip(want, ("dq", "dk", "dv", "dg", "dbeta", "dstate")):
        assert (w - got[name]).abs().max() <= 1e-13, name
    ry, rs, _, _ = ref.delta(*data, 0.3, state=s.detach(), lengths=n)
    assert (ry - y).abs().max() <= 1e-13 and (rs - torch.stack(last)).abs().max() <= 1e-13
