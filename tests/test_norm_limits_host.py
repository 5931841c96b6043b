"""The group norm at the limits of a launch (fewer than 2^32 threads), on the host: a plan is refused
for the launches that its calls make, not for others.  No GPU needed; addresses are never followed."""
import ctypes

import pytest

from convolution_forward_implicit_amd import ConvError, GroupNorm, capi

UNSUPPORTED = capi.CONV_ERR_UNSUPPORTED
TB = 1 << 40


def _refused(call, words="too large"):
    with pytest.raises(ConvError) as e:
        call()
    assert e.value.status == UNSUPPORTED and words in e.value.message, e.value.message


# a wave for each group of each sample in the join, a workgroup for each sample: more of both than a launch has
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [dict(N=1, L=1 << 21, G=32, C=128), dict(N=1 << 12, L=1 << 12, G=1, C=8),
                                  dict(N=1 << 20, L=1 << 8, G=4, C=3)])
def test_tokens_in_registers_need_no_slabs(dtype, dims):
    p = GroupNorm(dims, dtype, per_token=True)
    assert p.workspace_bytes == 0 and p.bwd_workspace_bytes > 0
    p.close()
    samples = dict(dims, N=dims["N"] * dims["L"], L=1)
    _refused(lambda: GroupNorm(samples, dtype))
    _refused(lambda: GroupNorm(dict(dims, C=4099), dtype, per_token=True))       # no register form


def test_a_call_that_needs_slabs_is_refused():
    """2048 channels are in registers in vectors of 8; tensors that allow none go over slabs, of 2^26 tokens too many."""
    p = GroupNorm(dict(N=1 << 16, L=1 << 10, G=1, C=2048), "bf16", per_token=True)
    args = capi.conv_gnorm_args_t(x=TB + 2, w=2 * TB, y=1 << 48)
    _refused(lambda: capi.conv_gnorm_run(p._plan, ctypes.byref(args), None, 0))
    bwd = capi.conv_gnorm_bwd_args_t(dy=TB + 2, x=1 << 48, w=2 * TB, dx=1 << 49, dw=3 * TB)
    _refused(lambda: capi.conv_gnorm_bwd_run(p._plan, ctypes.byref(bwd), 4 * TB, p.bwd_workspace_bytes))
    p.close()
