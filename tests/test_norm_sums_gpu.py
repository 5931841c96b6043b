"""The group norm on the GPU where a thread takes many rows: one slab a workgroup for thousands of
rows, all of them equal, so that every rounding of a long fp32 sum would go the same way.

Tolerances.  act none: d is dy itself, rounded nowhere, and every row is the same, so the sums are L
times a term.  A thread adds at most 64 terms in fp32 (64 x 2^-24 = 2^-18 of them), the rest is fp64,
one rounding to fp32 a slab and one of the result (2^-23): under 2^-17.  The statistics join at most 16
batches in fp32, of at most 16 values each (two roundings of the squares a join, 2^-19 with those inside
a batch, half of that for r; the mean one, 2^-20 of the mean of |x|: partial sums of terms that cancel are as
large as that, not as the mean): y is within 2^-18 of (|x| + |mean|) r w and 2^-20 of mean(|x|) r w.
"""
import pytest
import torch

from test_norm_gpu import DEV

pytestmark = pytest.mark.gpu

STEP = 1 + 2.0 ** -13       # added to a sum from 2^11 on, a tie goes to the even sum: 1


# G, C: as many workgroups of groups as two a compute unit, so that one slab holds all rows
@pytest.mark.parametrize("per_token,G,Ch,L", [(False, 512, 129, 4096), (False, 512, 260, 4096), (False, 513, 300, 4096),
                                              (True, 2048, 33, 4096), (True, 2048, 65, 4096), (True, 1024, 260, 8192)])
def test_long_sums_of_equal_terms(per_token, G, Ch, L):
    g = torch.Generator().manual_seed(Ch)
    row, dy = torch.randn(G, Ch, generator=g), torch.full((G, Ch), STEP)
    w = 1 + 0.3 * torch.randn(G, Ch, generator=g)
    from convolution_forward_implicit_amd import GroupNorm
    p = GroupNorm({"N": 1, "L": L, "G": G, "C": Ch}, "f32", has_bias=True, per_token=per_token)
    x = row.to(DEV).expand(1, L, G, Ch).contiguous()
    got = p.backward(dy.to(DEV).expand(1, L, G, Ch).contiguous(), x, w.to(DEV), torch.zeros(G, Ch, device=DEV))
    db, dw = got["dbias"].cpu().double(), got["dw"].cpu().double()
    y = p(x, w.to(DEV), torch.zeros(G, Ch, device=DEV))
    assert (y == y[:, :1]).all()
    y = y[0, 0].cpu().double()
    row = row.double()
    mean = row.mean(-1, keepdim=True)
    r = 1 / ((row - mean).square().mean(-1, keepdim=True) + 1e-5).sqrt()
    assert ((db - L * STEP).abs() <= 2.0 ** -17 * L * STEP).all(), float((db / (L * STEP) - 1).abs().max())
    rough = (row.abs() + mean.abs() + row.abs().mean(-1, keepdim=True) / 4) * r
    over = (dw - L * STEP * (row - mean) * r).abs() - 2.0 ** -17 * L * STEP * rough
    assert (over <= 0).all(), float(over.max())
    over = (y - (row - mean) * r * w.double()).abs() - 2.0 ** -18 * rough * w.double().abs()
    assert (over <= 0).all(), float(over.max())


@pytest.mark.parametrize("per_token", [False, True], ids=["sample", "token"])
def test_statistics_of_a_row_of_equal_parts(per_token):
    """4096 columns a thread, all of the same values, joined in fp64.  A batch is two rows of four values: eight roundings
    of its squares, 2^-21, and half of that for r; its mean 2^-21 of the mean of |x|; (x - mean) r three more, 2^-22 with
    the final one: under 2^-20 together."""
    from convolution_forward_implicit_amd import GroupNorm
    Ch, L = 1 << 22, 2
    part = torch.randn(1024, generator=torch.Generator().manual_seed(1))
    x = part.to(DEV).repeat(L, Ch // 1024).view(1, L, 1, Ch)
    y = GroupNorm({"N": 1, "L": L, "G": 1, "C": Ch}, "f32", per_token=per_token)(x, torch.ones(1, Ch, device=DEV))
    part = part.double()
    mean, r = part.mean(), 1 / (part.var(unbiased=False) + 1e-5).sqrt()
    want, rough = (part - mean) * r, (part.abs() + mean.abs() + part.abs().mean() / 4) * r
    over = (y.cpu().double().view(-1, 1024) - want).abs() - 2.0 ** -20 * rough
    assert (over <= 0).all(), float(over.max())
