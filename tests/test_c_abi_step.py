"""The entry points between linears and attention from a plain C11 program
(tests/csrc/abi_check_step.c): header, exports and argument validation, as
tests/test_c_abi.py has it for the others.  No GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("gcc") is None or
                                (shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc")),
                                reason="gcc or nvcc not available")


def test_c_client_of_the_step(tmp_path):
    from fp8_block_scaled_02_gb300 import build
    lib = build.build()
    exe = tmp_path / "abi_check_step"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic",
                    "-I", os.path.join(ROOT, "include"), "-o", str(exe),
                    os.path.join(ROOT, "tests", "csrc", "abi_check_step.c"),
                    lib, "-Wl,--no-undefined", "-Wl,-rpath," + os.path.dirname(lib)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    words = out.stdout.split()
    assert words[-4] == "checks" and int(words[-3]) >= 63 and words[-2] == "failures" and words[-1] == "0", out.stdout
