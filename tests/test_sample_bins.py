"""The sampling kernel's histogram of exponents has a bin for every token that
counts (csrc/samplebins.cuh), compiled for the host.  No GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_block_scaled_02_gb300", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_every_token_that_counts_has_a_bin(tmp_path):
    exe = tmp_path / "sample_bins"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-ffp-contract=off", "-I", CSRC, "-o", str(exe),
                    os.path.join(ROOT, "tests", "csrc", "sample_bins.cpp"), "-lm"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout


def test_the_kernel_takes_its_window_from_there():
    with open(os.path.join(CSRC, "sample.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert re.findall(r"job\.lowest = ([^;]*);", code) == ["max(max(K::from(window_end(job.m, job.c.h)), K::kNegInf + 1), bound)"]
