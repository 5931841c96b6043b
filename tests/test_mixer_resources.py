"""CPU build checks of the gated delta rule's and the group norm's kernels (no GPU): the
largest instances are compiled for gfx950 and must keep their registers out of
scratch memory, all but the gradient of 128 keys (addresses and factors of the next
head, spilled once a chunk) and of 256 (sums of three products); and the workgroups
that are meant to share a compute unit must fit its 160 KB of LDS together."""
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
    ("delta_prepare_kernel<bf16_t, 128, true>", "DeltaParams", 0, 2),
    ("delta_prepare_kernel<float, 128, true>", "DeltaParams", 0, 2),
    ("delta_prepare_kernel<float, 256, true>", "DeltaParams", 0, 1),
    ("delta_y_kernel<bf16_t, 128, 1>", "DeltaParams", 0, 1),
    ("delta_y_kernel<bf16_t, 128, 2>", "DeltaParams", 0, 1),
    ("delta_y_kernel<float, 256, 1>", "DeltaParams", 0, 1),
    ("delta_states_kernel<bf16_t, 128, 2>", "DeltaParams", 0, 1),
    ("delta_states_kernel<float, 128, 1>", "DeltaParams", 0, 1),
    ("delta_grad_kernel<bf16_t, 64>", "DeltaParams", 0, 1),
    ("delta_grad_kernel<bf16_t, 128>", "DeltaParams", 64, 1),
    ("delta_grad_kernel<float, 128>", "DeltaParams", 96, 1),
    ("delta_grad_kernel<bf16_t, 256>", "DeltaParams", 672, 1),
    ("delta_step_kernel<bf16_t, true>", "DeltaParams, int, int", 0, 1),
    ("gnorm_sums_kernel<bf16_t, 8>", "NormParams", 0, 2),
    ("gnorm_grad_kernel<bf16_t, 8>", "NormParams", 0, 2),
    ("gnorm_token_kernel<bf16_t, 8, 4>", "NormParams", 0, 1),
    ("gnorm_token_grad_kernel<bf16_t, 8, 4>", "NormParams", 0, 2),
]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_registers_and_shared_memory():
    lines = ['#include "delta_chain.h"', '#include "group_norm.h"', "namespace convfwd {"]
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
    kernels = re.split(r"Function Name: ", r.stdout)[1:]
    field = lambda text, what: int(re.search(re.escape(what) + r": (\d+)", text).group(1))
    assert len(kernels) >= len(KERNELS), r.stdout[-2000:]
    plain = lambda name: re.sub(r"\W", "", name.split("<")[0])
    for name, _, most, together in KERNELS:
        sizes = re.findall(r"\d+", name.split(",", 1)[1])
        kind = "f" if "float" in name else "DF16b"
        flag = "true" in name
        mine = [k for k in kernels if plain(name) + "I" + kind in k.split()[0]
                and re.findall(r"Li(\d+)E", k.split()[0]) == sizes and ("Lb1E" in k.split()[0]) == flag]
        assert len(mine) == 1, (name, [k.split()[0] for k in mine])
        scratch, lds = field(mine[0], "ScratchSize [bytes/lane]"), field(mine[0], "LDS Size [bytes/block]")
        assert scratch <= most and lds * together <= 160 * 1024, (name, scratch, lds)
