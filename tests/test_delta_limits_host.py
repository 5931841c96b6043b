"""The gated delta rule at the limits of a launch (fewer than 2^32 threads), on the host: a call is
held to the launches that it makes, not to others.  Only where there is no GPU: there a call that
passes its checks ends with the runtime's error; addresses are never followed."""
import ctypes

import pytest
import torch

from convolution_forward_implicit_amd import ConvError, DeltaRule, capi

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on made-up addresses")

TB = 1 << 40
RUN = dict(q=TB, k=2 * TB, v=3 * TB, g=4 * TB, beta=5 * TB)


def _run(dims, dtype):
    p = DeltaRule(dims, dtype)
    try:
        capi.conv_delta_run(p._plan, ctypes.byref(capi.conv_delta_args_t(y=6 * TB, **RUN)), 20 * TB, p.workspace_bytes)
    finally:
        p.close()


def _bwd(dims, dtype):
    p = DeltaRule(dims, dtype)
    args = capi.conv_delta_bwd_args_t(dy=6 * TB, dq=7 * TB, dk=8 * TB, dv=9 * TB, dg=10 * TB, dbeta=11 * TB, **RUN)
    try:
        capi.conv_delta_bwd_run(p._plan, ctypes.byref(args), 20 * TB, p.bwd_workspace_bytes)
    finally:
        p.close()


def _ends(call, dims, dtype, status):
    with pytest.raises(ConvError) as e:
        call(dims, dtype)
    assert e.value.status == status, e.value.message


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [dict(N=1, L=1 << 20, H=32, G=32, P=16, S=128), dict(N=1, L=1 << 22, H=8, G=8, P=16, S=256)])
def test_a_gradient_without_slices_sums_none(dtype, dims):
    """The sums of dq and dk over slices of a group's heads take no launch where there is one slice."""
    _ends(_bwd, dims, dtype, capi.CONV_ERR_HIP)
