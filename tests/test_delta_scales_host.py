"""The scales that the reference of the gated delta rule gives for its errors are small enough to
tell a gradient that is wrong: mistakes planted in the reference's own gradients are rejected by the
check of the GPU tests, for every case of theirs and each gradient.  No GPU needed."""
import pytest
import torch

from oracle import delta as ref
from test_delta_gradient_gpu import ALL, check, inputs


def _wrong(got, want, mag, dtype, names, what):
    for k in names:
        if want[k] is None or torch.equal(got[k], want[k]):
            continue        # nothing was there to lose
        try:
            check(got, want, mag, dtype, k)
        except AssertionError:
            continue
        pytest.fail("%s passes in %s" % (what, k))


ROWS = ("dq", "dk", "dv", "dg", "dbeta")


# bf16's roundings hide the most; a large case's keys are random only, to save time
def _cases():
    for case in ALL:
        N, L, H, P, G, S = case[:6]
        for keys in ("random", "same", "few") if N * L * H * P * S < 1 << 22 else ("random",):
            yield case, keys


@pytest.mark.parametrize("case,keys", list(_cases()), ids=str)
def test_planted_mistakes_are_rejected(case, keys):
    N, L, H, P, G, S, _, _ = case
    dtype = "bf16"
    dy, a = inputs(case, dtype, keys)
    want, mag = ref.delta_grad(dy, **a)
    check(want, want, mag, dtype)
    if N * L == 0:
        return
    _wrong({k: torch.zeros_like(t) for k, t in want.items()}, want, mag, dtype, ROWS + ("dstate",), "nothing at all")
    for lo, hi in ((0, L - 32), (0, min(L, 64)), (64, min(L, 128)), (L - 1, L)):
        if 0 <= lo < hi:
            cut = {k: want[k].clone() for k in ROWS}
            for t in cut.values():
                t[:, lo:hi] = 0
            _wrong(cut, want, mag, dtype, ROWS, "zeros in rows %d to %d" % (lo, hi))
    for h in {0, H - 1}:        # a head's gradients lost, also in its group's sums
        cut = {k: want[k].clone() for k in ("dv", "dg", "dbeta")}
        for t in cut.values():
            t[:, :, h] = 0
        _wrong(cut, want, mag, dtype, cut, "no head %d" % h)
    cut = {"dstate": want["dstate"].clone()}
    cut["dstate"][:, :, P - 1] = 0
    _wrong(cut, want, mag, dtype, cut, "no last channel")
    if keys == "same":          # one key replaces all that a state holds under it: little of one reaches the tokens behind
        return
    if L > 64:                  # what a chunk hands to the next, either way, lost: sequences of 64 and of the rest
        parts = [dict(a, **{k: a[k][:, i:j] for k in ("q", "k", "v", "g", "beta")}) for i, j in ((0, 64), (64, L))]
        for p, (i, j) in zip(parts, ((0, 64), (64, L))):
            if a["lengths"] is not None:
                p["lengths"] = (a["lengths"] - i).clamp(0, j - i)
        parts[0]["dstate_out"], parts[1]["state"] = None, None
        (one, _), (two, _) = ref.delta_grad(dy[:, :64], **parts[0]), ref.delta_grad(dy[:, 64:], **parts[1])
        _wrong({k: torch.cat([one[k], two[k]], 1) for k in ROWS}, want, mag, dtype,
               ("dk", "dv", "dbeta") + (("dg",) if keys == "random" else ()), "a state that a chunk does not hand on")
    for lost in ("state", "dstate_out"):
        if a[lost] is not None:
            less, _ = ref.delta_grad(dy, **dict(a, **{lost: None}))
            _wrong({k: less[k] for k in ROWS}, want, mag, dtype, ("dk", "dg", "dbeta") if lost == "state" else ("dk", "dv", "dg", "dbeta"),
                   "without %s" % lost)
