"""The error bound of two_exp2 (csrc/twofloat.cuh) over its whole range, compiled for the host.  No GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_exponential_over_its_range(tmp_path):
    exe = tmp_path / "twofloat_range"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-ffp-contract=off", "-I",
                    os.path.join(ROOT, "fp8_block_scaled_02_gb300", "csrc"), "-o", str(exe),
                    os.path.join(ROOT, "tests", "csrc", "twofloat_range.cpp"), "-lm"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout
