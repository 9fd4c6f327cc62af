"""Loads of the kernels between a step's linears and its attention.  A kernel
launched ahead of its predecessor's end may be on the GPU while what it will
read is still being written; ld.global.nc (__ldg) promises that nothing writes
it while the kernel lives, so these kernels use ordinary loads behind
griddepcontrol.wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_02_gb300", "csrc")


@pytest.mark.parametrize("name", ["kvrope.cu", "route.cu", "sample.cu", "serving.cuh", "twofloat.cuh"])
def test_no_load_promises_that_its_source_is_constant(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"ld_nc_\w+|__ldg\b|ld\.global(\.\w+)*\.nc|prefetch\.global", code)


@pytest.mark.parametrize("name", ["kvrope.cu", "route.cu", "sample.cu"])
def test_every_kernel_waits_for_its_predecessor(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    kernels = [k.split("\n}\n")[0] for k in code.split("__global__")[1:]]
    assert kernels and all("pdl_wait()" in k for k in kernels)
