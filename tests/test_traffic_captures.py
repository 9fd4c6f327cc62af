"""profiles/traffic.json holds captures of the kernels as they are: bench.py
reports a DRAM traffic figure only while the kernel's sources hash to the
captured ones, so a helper for another kernel must not go into a header that
they include."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
    CAPTURES = {k: v for k, v in json.load(f).items() if not k.startswith("_")}


@pytest.mark.parametrize("name", CAPTURES)
def test_the_capture_is_of_the_present_source(name):
    spec = importlib.util.spec_from_file_location("bench_under_test", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    kernel, workload = name.rsplit(" ", 1)
    assert bench.measured_traffic(kernel, workload) == CAPTURES[name]["dram_bytes_per_launch"]
