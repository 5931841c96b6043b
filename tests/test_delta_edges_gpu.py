"""The gated delta rule on the GPU: gradients whose offsets pass 32 bits, in the tensors and in the
workspace, and how far what is no number reaches."""
import pytest
import torch

from test_delta_gpu import DEV, TYPE, _case, _gpu, _plan

pytestmark = pytest.mark.gpu


def test_gradient_offsets_past_32_bits():
    """Rows 16 MB apart, all in one tensor: those of the last sequence lie past the 2^32nd element, of inputs and
    gradients."""
    N, L, H, P, G, S = 3, 192, 2, 32, 1, 32
    far = 1 << 23
    a, _, _ = _case(N, L, H, P, G, S, "bf16", False, None, 2)
    v = _gpu(a)
    dy = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    p = _plan(N, L, H, P, G, S, "bf16")
    want = p.backward(dy, **v)
    wide = torch.zeros(N * L * far, dtype=torch.bfloat16, device=DEV).view(N, L, far)       # 9.7 GB
    at = iter(range(0, 10 ** 6, 1024))
    put = lambda t: wide[..., (i := next(at)):i + t[0, 0].numel()].unflatten(-1, t.shape[2:])
    ins = {k: put(t).copy_(t) for k, t in dict(v, dy=dy).items() if k != "g"}
    out = {"d" + k: put(v[k]) for k in ("q", "k", "v", "beta")}
    got = p.backward(ins.pop("dy"), **ins, g=v["g"], out=out)
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[k], want[k]), k


def test_gradient_workspace_past_32_bits():
    """65536 tokens of 64 heads leave more than 2^32 bytes of states and of rows each: the last heads' gradients, and
    their prompt's y, are those of a call of their own, to the bit."""
    N, L, H, P, S = 1, 1 << 16, 64, 128, 128
    g = torch.Generator(DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    unit = lambda *s: torch.nn.functional.normalize(r(*s), dim=-1).bfloat16()
    a = dict(q=unit(N, L, H, S), k=unit(N, L, H, S), v=r(N, L, H, P).bfloat16(), g=-0.2 * r(N, L, H).abs(),
             beta=torch.sigmoid(r(N, L, H)).bfloat16())
    dy = r(N, L, H, P).bfloat16()
    p, one = _plan(N, L, H, P, H, S, "bf16"), _plan(N, L, H // 2, P, H // 2, S, "bf16")
    assert p.bwd_workspace_bytes > 2 * (1 << 32)
    last = {k: t[:, :, H // 2:].contiguous() for k, t in a.items()}
    assert torch.equal(p(**a)[:, :, H // 2:], one(**last))
    got, want = p.backward(dy, **a), one.backward(dy[:, :, H // 2:].contiguous(), **last)
    for k in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.isfinite(got[k]).all() and torch.equal(got[k][:, :, H // 2:], want[k]), k


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v", "beta", "state"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_how_far_what_is_no_number_reaches(dtype, what, bad):
    """Sequence 1, token 70, group (head) 1: the chunks in front, the other sequences and the other groups (heads) are
    what they are without it, to the bit; of the gradients, which go back to the first token, the others' are."""
    N, L, H, P, G, S = 3, 150, 4, 24, 2, 32
    a, s0, _ = _case(N, L, H, P, G, S, dtype, True, None, 5)
    dy = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(1)).to(TYPE[dtype]).to(DEV)
    p = _plan(N, L, H, P, G, S, dtype)
    heads = [2, 3] if what in "qk" else [1]
    results = []
    for value in (None, bad):
        if value is not None:
            t = s0 if what == "state" else a[what]
            t[(1, 1, 3, 3) if what == "state" else (1, 70, 1) + (3,) * (t.dim() - 3)] = value
        last = torch.empty(N, H, P, S, device=DEV)
        y = p(**_gpu(a), state=s0.to(DEV), state_out=last)
        results.append((y, last, p.backward(dy, **_gpu(a), state=s0.to(DEV))))
    (y, last, d), (yb, lastb, db) = results
    other = [h for h in range(H) if h not in heads]
    assert not torch.isfinite(yb[1, 70:, heads]).all() or what == "q"
    if what != "state":
        assert torch.equal(yb[1, :64], y[1, :64])
    for n in (0, 2):
        assert torch.equal(yb[n], y[n]) and torch.equal(lastb[n], last[n])
        for k in d:
            assert torch.equal(db[k][n], d[k][n]), k
    assert torch.equal(yb[:, :, other], y[:, :, other]) and torch.equal(lastb[:, other], last[:, other])
    for k in ("dv", "dg", "dbeta"):
        assert torch.equal(db[k][:, :, other], d[k][:, :, other]), k
    assert torch.equal(db["dstate"][:, other], d["dstate"][:, other])
    free = [i for i in range(G) if not any(h // (H // G) == i for h in heads)]
    for k in ("dq", "dk"):
        assert torch.equal(db[k][:, :, free], d[k][:, :, free]), k
