"""The tests of the states' digits tell two bf16 terms from three: the chunks of the gated delta rule,
computed in double precision but for the operands of the matrix products, which are held in so many
terms.  No GPU needed."""
import pytest
import torch

from test_delta_digits_gpu import STATES, exact, inputs, near

F64 = torch.float64


def _terms(v, n):
    out, v = torch.zeros_like(v), v.float()
    for _ in range(n):
        t = v.bfloat16().float()
        out, v = out + t.double(), v - t
    return out


def _chunks(a, s0, n):
    """The last state with g = 0, operands in n terms."""
    k, v, b = a["k"][0, :, 0].double(), a["v"][0].double(), a["beta"][0].double()
    out = torch.empty(s0.shape, dtype=F64)
    for h in range(v.shape[1]):
        S = s0[0, h].double()
        for t in range(0, v.shape[0], 64):
            K, V, B = k[t:t + 64], v[t:t + 64, h], b[t:t + 64, h]
            T = (K @ K.T).tril(-1)
            N = torch.linalg.solve(torch.eye(len(K), dtype=F64) + T * B, T)
            Z = V - K @ _terms(S, n).T
            Y = Z - _terms(N * B, n) @ _terms(Z, n)
            S = S + _terms(B[:, None] * Y, n).T @ K
        out[0, h] = S
    return out


@pytest.mark.parametrize("case", STATES, ids=str)
def test_two_terms_are_told_from_three(case):
    S, L, _, tol = case
    a, s0 = inputs(S, L, "bf16")
    want, most = exact(a, s0)
    near(_chunks(a, s0, 3), want, most, tol)
    with pytest.raises(AssertionError):
        near(_chunks(a, s0, 2), want, most, tol)
