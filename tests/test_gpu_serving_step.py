"""GPU test of the serving step that runs the plan, the 4-bit cache and the
log probabilities together (examples/serving_step.py): decode steps replayed
from a graph against the same tokens given as one prompt, and the bookkeeping.

The two runs attend over the same cache bytes for the same tokens; they
differ in the order of fp32 sums and in which GEMV kernel runs (m rows), each
rounding to bf16 (2^-9 relative) a few times per layer.  The logits are normal
with a standard deviation of about 1; 0.15 is about 40 such roundings of a
value of 2, and a wrong key, slot or block moves them by their own size.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import serving_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    lib_or_skip()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


PROMPTS = [[3, 14, 15], [9], [2, 6, 5, 35, 8, 97, 93], list(range(40))]


def test_decode_is_the_prompt_token_by_token(example):
    m = example.Decoder()
    first = m.prompt(PROMPTS)
    steps = [(t, lp, e) for t, lp, e in m.decode(first, 20)]
    assert m.lens.tolist() == [len(p) + 20 for p in PROMPTS]
    full = [p + [int(first[b])] + [int(t[b]) for t, _, _ in steps[:-1]] for b, p in enumerate(PROMPTS)]
    again = example.Decoder()
    new = torch.tensor([len(p) for p in full], dtype=torch.int32, device="cuda")
    tokens = torch.tensor([t for p in full for t in p], dtype=torch.int32, device="cuda")
    plan, logits, _, _ = again.step(tokens, new, max(len(p) for p in full))
    # the same slots in use, and the same bytes of the first layer's cache in them
    assert again.lens.tolist() == m.lens.tolist()
    assert int(again.free_head) == int(m.free_head) == sum(-(-len(p) // 16) for p in full)
    x = logits.double().cpu().numpy()
    cu = plan.cu_new.cpu().numpy()
    for b, p in enumerate(PROMPTS):
        for i, (t, lp, e) in enumerate(steps):
            row = x[cu[b] + len(p) + i]
            want, _ = ref.logprobs(row[None], [int(t[b])], 1)
            assert row[int(t[b])] >= row.max() - 0.15            # the same choice, or one as good
            assert abs(float(lp[b]) - want["logprobs"][0]) < 0.3
            assert abs(float(e[b]) - want["entropy"][0]) < 0.15
    import fp8_block_scaled_02_gb300 as fp8bs
    assert fp8bs.check_device_error() == 0


def test_a_full_pool_refuses_and_reports(example):
    import fp8_block_scaled_02_gb300 as fp8bs
    m = example.Decoder(batch=2, max_len=32)
    m.free = m.free[:3].contiguous()
    m.prompt([list(range(30)), list(range(20))])
    assert m.lens.tolist() == [30, 0] and int(m.free_head) == 2
    assert fp8bs.check_device_error() == 32


def test_the_example_runs(example, capsys):
    example.main()
    out = capsys.readouterr().out
    assert "lengths [11, 9, 15, 48]" in out and np.all(["step %d" % i in out for i in range(8)])
