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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("call,N", [(_run, (1 << 19) - 1), (_bwd, (1 << 18) - 1)], ids=["prompt", "gradient"])
def test_two_blocks_a_workgroup_are_one(call, N, dtype):
    """Up to 128 keys a workgroup takes 32 channels where there are many, and only half as many are launched."""
    dims = dict(N=N, L=1, H=16, P=32, G=1, S=32)
    _ends(call, dims, dtype, capi.CONV_ERR_HIP)
    _ends(call, dict(dims, N=N + 1), dtype, capi.CONV_ERR_UNSUPPORTED)
    _ends(call, dict(dims, S=129), dtype, capi.CONV_ERR_UNSUPPORTED)
