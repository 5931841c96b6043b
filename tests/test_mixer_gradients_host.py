"""The check of a mixer's gradients rejects gradients that are right but for a part: rows, a sequence or
a head that is lost.  No GPU needed."""
import pytest
import torch

from test_mixer_gradients_gpu import FAR, L, check, parts, reference
from test_mixer_gpu import H, N, P, TYPE, _inputs


def test_lost_parts_are_rejected():
    v = _inputs("bf16", L, 3)
    dout = torch.randn(N, L, H, P, generator=torch.Generator().manual_seed(6)).to(TYPE["bf16"])
    want = reference(v, dout, None)
    check(want, want, FAR["bf16"])
    lost = 0
    for name in want:
        for i, _ in enumerate(parts(name, want[name])):
            got = {k: t.clone() for k, t in want.items()}
            list(parts(name, got[name]))[i][1].zero_()
            with pytest.raises(AssertionError):
                check(got, want, FAR["bf16"])
            lost += 1
    assert lost > 60
