"""The gradients of a mixer's operators run together, element by element against the chain of the
double-precision references' gradients: of a whole tensor, and of each part of it that a kernel could
lose by itself (a chunk's rows, the last ones, a sequence, a head, a group's queries or keys).

Tolerance: four operators forward and four back, each within a rounding and 2^-13 of its terms, and
each value used by two of them: 16 x 2^-8 in 2-norm of a part in bf16, 16 x 2^-13 in fp32.
"""
import pytest
import torch

from oracle import delta as rdelta, norm as rnorm, seq
from test_mixer_gpu import DEV, G, H, N, P, S, TYPE, Mixer, _cut, _gpu, _inputs

pytestmark = pytest.mark.gpu

FAR = {"bf16": 2.0 ** -4, "f32": 2.0 ** -9}
L = 135         # two chunks and the first rows of a third


def reference(v, dout, lengths):
    """The gradients that Mixer.backward names."""
    c, _, _ = seq.causal(v["u"], v["w"], v["bias"], True, lengths=lengths)
    q0, k0, x = _cut(c)
    unit = dict(lengths=lengths, center=False, per_token=True, eps=1e-6)
    q, k = (rnorm.norm(t, v["unit"], **unit)[0] for t in (q0, k0))
    y = rdelta.delta(q, k, x, v["g"], v["beta"], S ** -0.5, lengths=lengths)[0]
    a, _ = rnorm.norm_grad(dout, y, v["scale"], None, v["z"], lengths, "silu", False, True)
    b, _ = rdelta.delta_grad(a["dx"], q, k, x, v["g"], v["beta"], S ** -0.5, lengths=lengths)
    d, e = rnorm.norm_grad(b["dq"], q0, v["unit"], **unit)[0], rnorm.norm_grad(b["dk"], k0, v["unit"], **unit)[0]
    dc = torch.cat([t.flatten(2) for t in (d["dx"], e["dx"], b["dv"])], -1)
    f = seq.causal_grad(dc, v["u"], v["w"], v["bias"], True, lengths=lengths)
    return {"u": f["dx"], "w": f["dw"], "bias": f["dbias"], "g": b["dg"], "beta": b["dbeta"], "z": a["dgate"],
            "scale": a["dw"], "unit": d["dw"] + e["dw"]}


def parts(name, t):
    """(what, part) of a gradient."""
    yield "all", t
    if name in ("u", "g", "beta", "z"):
        for what, rows in (("first chunk", t[:, :64]), ("second chunk", t[:, 64:128]), ("last rows", t[:, 128:])):
            yield what, rows
        if name != "g":         # a first token's decay has no state to fade: zero
            yield "first row", t[:, :1]
        for n in range(N):
            yield "sequence %d" % n, t[n]
    if name == "u":
        q, k, x = _cut(t)
        for i in range(G):
            yield "queries %d" % i, q[:, :, i]
            yield "keys %d" % i, k[:, :, i]
        for h in range(H):
            yield "values %d" % h, x[:, :, h]
    if name in ("g", "beta", "z"):
        for h in range(H):
            for what, rows in (("all", slice(None)), ("first chunk", slice(0, 64)), ("last rows", slice(128, None))):
                yield "head %d, %s" % (h, what), t[:, rows, h]
    if name == "scale":
        for h in range(H):
            yield "head %d" % h, t[h]


def check(got, want, far):
    for name, t in want.items():
        for (what, a), (_, b) in zip(parts(name, got[name].detach().cpu().double()), parts(name, t)):
            assert float((a - b).norm()) <= far * float(b.norm()), (name, what, float((a - b).norm()), float(b.norm()))


@pytest.mark.parametrize("lengths", [None, [135, 77]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_part_of_the_gradients(dtype, lengths):
    v = _inputs(dtype, L, 3)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    nd = None if n is None else n.to(DEV)
    dout = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(6)).to(TYPE[dtype])
    m, d = Mixer(dtype, L), _gpu(v)
    _, kept = m.forward(d, nd)
    check(m.backward(dout.to(DEV), d, kept, nd), reference(v, dout, n), FAR[dtype])
