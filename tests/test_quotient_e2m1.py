"""The 4-bit cache's append forms x / d with Markstein's correction instead of
an IEEE division (csrc/kv4.cu).  The same binary32 steps on the host, for
every divisor mantissa and the bf16 values next to every border between e2m1
codes, give the code of the IEEE quotient.  (The GPU tests then compare the
kernel's codes with a reference that divides.)"""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_markstein_quotient_encodes_like_ieee_division(tmp_path):
    exe = tmp_path / "quotient_e2m1"
    subprocess.run(["gcc", "-std=c11", "-O2", "-ffp-contract=off", "-fno-fast-math", "-fopenmp",
                    "-o", str(exe), os.path.join(HERE, "csrc", "quotient_e2m1.c"), "-lm"], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600).stdout.split()
    assert int(out[1]) == 3 * 7 * 2 ** 23 and int(out[3]) == 0
