"""CPU build checks of the sequence kernels (no GPU): the largest instance of
each is compiled for gfx950 and must keep its registers out of scratch memory,
all but the bf16 gradient of 128 states, whose addresses taken before the loop
over the heads take 32 bytes a lane; and the workgroups that are meant to share
a compute unit must fit its 160 KB of LDS together."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_implicit_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# kernel, its parameters, bytes of scratch, workgroups a compute unit
KERNELS = [
    ("causal_conv_kernel<bf16_t, 4, 8, true>", "CausalParams", 0, 1),
    ("causal_bwd_kernel<bf16_t, 4, 4, true>", "CausalParams", 0, 1),
    ("causal_bwd_kernel<float, 8, 1, true>", "CausalParams", 0, 1),
    ("scan_fwd_dma_kernel<128>", "ScanParams", 0, 1),
    ("scan_state_dma_kernel<128, true>", "ScanParams", 0, 2),
    ("scan_fwd_kernel<bf16_t, 128>", "ScanParams", 0, 2),
    ("scan_fwd_kernel<float, 128>", "ScanParams", 0, 2),
    ("scan_state_kernel<bf16_t, 128, true>", "ScanParams", 0, 2),
    ("scan_bwd_kernel<bf16_t, 64>", "ScanParams", 0, 1),
    ("scan_bwd_kernel<float, 128>", "ScanParams", 0, 1),
    ("scan_bwd_kernel<bf16_t, 128>", "ScanParams", 32, 1),
]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_registers_and_shared_memory():
    lines = ['#include "causal_conv.h"', '#include "scan_dma.h"', "namespace convfwd {"]
    lines += ["template __global__ void %s(%s);" % (k, p) for k, p, _, _ in KERNELS] + ["}"]
    d = tempfile.mkdtemp()
    try:
        src = os.path.join(d, "inst.hip")
        with open(src, "w") as f:
            f.write("\n".join(lines) + "\n")
        cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-c", "--cuda-device-only",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
               "-Rpass-analysis=kernel-resource-usage", src, "-o", os.path.join(d, "inst.o")]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
        assert r.returncode == 0, r.stdout[-3000:]
    finally:
        shutil.rmtree(d, ignore_errors=True)
    field = lambda what: [int(v) for v in re.findall(re.escape(what) + r": (\d+)", r.stdout)]
    scratch, lds = field("ScratchSize [bytes/lane]"), field("LDS Size [bytes/block]")
    assert len(scratch) == len(lds) == len(KERNELS), r.stdout[-2000:]
    for (name, _, most, together), s, m in zip(KERNELS, scratch, lds):
        assert s <= most and m * together <= 160 * 1024, (name, s, m)
