"""Sequence operators at the limits of a launch (fewer than 2^32 threads) and of
their types, on the host: what cannot run is refused before anything is
launched, what can is planned.  No GPU needed; addresses are never followed."""
import ctypes

import pytest

from convolution_forward_implicit_amd import CausalConv, ConvError, SelectiveScan, capi

UNSUPPORTED = capi.CONV_ERR_UNSUPPORTED
TB = 1 << 40


def _refused(call, words="too large"):
    with pytest.raises(ConvError) as e:
        call()
    assert e.value.status == UNSUPPORTED and words in e.value.message, e.value.message


# A prompt takes 256 threads to 64 vectors of 32 tokens, a step to 256 vectors: 2^24 of those are one too many
@pytest.mark.parametrize("dtype,dims,more", [
    ("bf16", dict(N=(1 << 24) - 1, L=1, C=2048, F=4), dict(N=1 << 24)),
    ("f32", dict(N=(1 << 22) - 1, L=32, C=4096, F=4), dict(N=1 << 22)),
    ("f32", dict(N=(1 << 22) - 1, L=64, C=1023, F=4), dict(N=1 << 30)),
    ("bf16", dict(N=1 << 24, L=1, C=16, F=4), dict(N=1 << 30, C=2048))])      # too large for a prompt only
def test_convolution_plans(dtype, dims, more):
    CausalConv(dims, dtype).close()
    _refused(lambda: CausalConv(dict(dims, **more), dtype))


# ... and the scan to 64 channels of a head, its step to 32 of 128 states or 1024 of 4
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims,more", [
    (dict(N=(1 << 20) - 1, L=1, H=16, P=64, G=1, S=128), dict(N=1 << 20)),
    (dict(N=(1 << 23) - 1, L=64, H=1, P=128, G=1, S=128), dict(P=129, N=1 << 23)),
    (dict(N=1, L=4, H=(1 << 24) - 1, P=1, G=1, S=1), dict(H=1 << 24)),
    (dict(N=1 << 23, L=1, H=1, P=512, G=1, S=4), dict(S=128))])               # too large for a prompt only
def test_scan_plans(dtype, dims, more):
    SelectiveScan(dims, dtype).close()
    _refused(lambda: SelectiveScan(dict(dims, **more), dtype))


def test_calls_whose_form_needs_more_than_the_plans():
    """Rows that are no whole vectors take eight times the workgroups, and a gradient's have twice the threads."""
    args = capi.conv_causal_args_t(x=TB, w=2 * TB, y=3 * TB + 2)
    for n in (1 << 22, 1 << 24):
        with CLOSE(CausalConv(dict(N=n, L=1, C=512, F=4), "bf16")) as p:
            _refused(lambda: capi.conv_causal_run(p._plan, ctypes.byref(args)))
            bwd = capi.conv_causal_bwd_args_t(dy=TB + 2, x=2 * TB, w=3 * TB, dx=4 * TB, dw=5 * TB)
            _refused(lambda: capi.conv_causal_bwd_run(p._plan, ctypes.byref(bwd), 8 * TB, p.bwd_workspace_bytes))
    step = capi.conv_causal_args_t(x=TB, w=2 * TB, y=3 * TB + 2, state=4 * TB, state_out=4 * TB)
    with CLOSE(CausalConv(dict(N=1 << 23, L=1, C=512, F=4), "bf16")) as p:
        _refused(lambda: capi.conv_causal_step(p._plan, ctypes.byref(step)))
    run = dict(x=TB, dt=2 * TB, a=3 * TB, b=4 * TB, c=5 * TB)
    with CLOSE(SelectiveScan(dict(N=1 << 19, L=1, H=16, P=64, G=1, S=16), "bf16")) as p:
        args = capi.conv_scan_args_t(y=6 * TB, **run)
        _refused(lambda: capi.conv_scan_run(p._plan, ctypes.byref(args), 9 * TB, p.workspace_bytes))
        bwd = capi.conv_scan_bwd_args_t(dy=7 * TB, dx=8 * TB, ddt=9 * TB, da=10 * TB, db=11 * TB, dc=12 * TB, **run)
        _refused(lambda: capi.conv_scan_bwd_run(p._plan, ctypes.byref(bwd), 20 * TB, p.bwd_workspace_bytes))
    with CLOSE(SelectiveScan(dict(N=1 << 19, L=1, H=16, P=64, G=1, S=128), "f32")) as p:
        step = capi.conv_scan_args_t(y=6 * TB, state=20 * TB, state_out=20 * TB, **run)
        _refused(lambda: capi.conv_scan_step(p._plan, ctypes.byref(step)))


class CLOSE:
    def __init__(self, plan):
        self.plan = plan

    def __enter__(self):
        return self.plan

    def __exit__(self, *e):
        self.plan.close()
