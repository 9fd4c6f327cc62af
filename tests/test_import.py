"""The package without torch: importing it, building, and the calls that only
ask the library need none (a build host may have no torch at all)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.split()


def test_importing_does_not_load_torch():
    assert run("import sys, fp8_block_scaled_02_gb300\n"
               "from fp8_block_scaled_02_gb300 import build\n"
               "print('torch' in sys.modules)") == ["False"]


def test_host_only_calls_work_without_torch():
    assert run("import os, sys\n"
               "sys.modules['torch'] = None\n"
               "import fp8_block_scaled_02_gb300 as p\n"
               "from fp8_block_scaled_02_gb300 import build\n"
               "print(p.kv4_cache_shape(4, 32, 2, 128) == (4, 2, 2, 1152))\n"
               "print(p.select_path(1, 256, 256) if os.path.exists(p.LIB_PATH) else 1)\n"
               "try:\n"
               "    p.gemv(None, None, None)\n"
               "except (ImportError, AttributeError):\n"
               "    print('refused')") == ["True", "1", "refused"]
