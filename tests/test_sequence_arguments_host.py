"""What the sequence classes make of their arguments before the library sees
them.  No GPU needed."""
import pytest
import torch

from convolution_forward_implicit_amd import CausalConv, ConvError, SelectiveScan, capi

PLANS = [lambda t: CausalConv({"N": 2, "L": 10, "C": 16, "F": 4}, t),
         lambda t: SelectiveScan({"N": 2, "L": 10, "H": 4, "P": 16, "G": 2, "S": 16}, t)]


@pytest.mark.parametrize("plan", PLANS)
def test_a_type_by_its_number_is_the_type_by_its_name(plan):
    """The tensors' type is the plan's however it was named: fp32 kernels on bf16 tensors would read past their end."""
    for name, number, t in (("f32", capi.CONV_DT_F32, torch.float32), ("bf16", capi.CONV_DT_BF16, torch.bfloat16)):
        for p in (plan(name), plan(number)):
            assert p.dtype == name and p._type(torch) is t and (" %s " % name) in p.describe()
    with pytest.raises(ConvError):
        plan(7)
    with pytest.raises((KeyError, ValueError, TypeError)):
        plan("f16")


@pytest.mark.parametrize("plan", PLANS)
def test_a_stream_of_another_device_is_refused(plan):
    """... with stand-ins: the kernels would run there on tensors that are here."""
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0

    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        plan("bf16")._on(torch, torch.device("cuda", 0), Stream())
