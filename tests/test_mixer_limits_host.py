"""The gated delta rule and the group norm at the limits of a launch (fewer than 2^32
threads), on the host: what cannot run is refused before anything is launched, what
can is planned.  No GPU needed; addresses are never followed."""
import ctypes

import pytest

from convolution_forward_implicit_amd import ConvError, DeltaRule, GroupNorm, capi

UNSUPPORTED = capi.CONV_ERR_UNSUPPORTED
TB = 1 << 40


def _refused(call, words="too large"):
    with pytest.raises(ConvError) as e:
        call()
    assert e.value.status == UNSUPPORTED and words in e.value.message, e.value.message


# A prompt takes 512 threads to 16 channels of a head, a step 256 to 32 of 128 keys or 1024 of 4
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims,more", [
    (dict(N=(1 << 19) - 1, L=1, H=16, P=16, G=1, S=128), dict(N=1 << 20, P=32)),
    (dict(N=(1 << 23) - 1, L=64, H=1, P=16, G=1, S=128), dict(N=1 << 23, P=1024)),
    (dict(N=1, L=4, H=(1 << 23) - 1, P=1, G=1, S=1), dict(H=1 << 24)),
    (dict(N=1 << 23, L=1, H=1, P=512, G=1, S=4), dict(S=128))])               # too large for a prompt only
def test_delta_plans(dtype, dims, more):
    DeltaRule(dims, dtype).close()
    _refused(lambda: DeltaRule(dict(dims, **more), dtype))


def test_delta_calls_whose_form_needs_more_than_the_plans():
    """A gradient's two passes over the states share a launch."""
    run = dict(q=TB, k=2 * TB, v=3 * TB, g=4 * TB, beta=5 * TB)
    p = DeltaRule(dict(N=1 << 19, L=1, H=8, P=16, G=8, S=16), "bf16")
    bwd = capi.conv_delta_bwd_args_t(dy=6 * TB, dq=7 * TB, dk=8 * TB, dv=9 * TB, dg=10 * TB, dbeta=11 * TB, **run)
    _refused(lambda: capi.conv_delta_bwd_run(p._plan, ctypes.byref(bwd), 20 * TB, p.bwd_workspace_bytes))
    p.close()
    p = DeltaRule(dict(N=1 << 23, L=1, H=1, P=512, G=1, S=4), "bf16")         # planned for its steps
    args = capi.conv_delta_args_t(y=6 * TB, **run)
    _refused(lambda: capi.conv_delta_run(p._plan, ctypes.byref(args), 20 * TB, p.workspace_bytes))
    p.close()


def test_norm_gradients_sums_share_a_launch():
    """63 x 2^16 workgroups of 1024 threads for the samples' groups, and 2^19 for dw: too many together."""
    p = GroupNorm(dict(N=63, L=1, G=1 << 20, C=8), "bf16")
    bwd = capi.conv_gnorm_bwd_args_t(dy=TB, x=2 * TB, w=3 * TB, dx=4 * TB, dw=5 * TB)
    _refused(lambda: capi.conv_gnorm_bwd_run(p._plan, ctypes.byref(bwd), 20 * TB, p.bwd_workspace_bytes))
    p.close()
