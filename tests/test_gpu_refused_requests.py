"""A serving step whose free list runs out (examples/serving_step.py): what a
refused request gives, that it goes on when blocks come back, and that the
others do not notice.

Log probabilities of two runs are compared within 0.3, as in
test_gpu_serving_step.py: the runs' attention cuts its work differently once
their lengths differ, which moves roundings to bf16.
"""
import pytest
import torch

from test_gpu_serving_step import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

PROMPTS = [list(range(30)), list(range(100, 120))]


def keys(m, b, n):
    """The first layer's cached keys and values of request b."""
    import fp8_block_scaled_02_gb300 as fp8bs
    pos = torch.arange(n, device="cuda")
    slots = (m.table[b].long()[pos // m.page] * m.page + pos % m.page).to(torch.int32)
    return fp8bs.kv4_gather(*m.caches[0], slots, m.scale, m.scale)


def test_a_request_of_some_length_is_refused_and_goes_on(example):  # noqa: F811
    import fp8_block_scaled_02_gb300 as fp8bs
    ample = example.Decoder(batch=2, max_len=64)
    first = ample.prompt(PROMPTS)
    want = list(ample.decode(first, 20))
    assert fp8bs.check_device_error() == 0

    m = example.Decoder(batch=2, max_len=64)
    spare = m.free[5:6].clone()
    m.free = m.free[:5].clone()                                   # both prompts, and one block for request 0 at 32
    assert torch.equal(m.prompt(PROMPTS), first)
    got = list(m.decode(first, 20))                               # request 1 has 20 cached: 12 steps fit
    assert m.lens.tolist() == [50 - 2, 32]                        # and request 0 stops at 48
    assert int(m.free_head) == 5 and fp8bs.check_device_error() == 32
    for i in range(12):
        assert all(torch.equal(a, w) for a, w in zip(got[i], want[i])), i
    kept = keys(m, 1, 32)
    for i in range(12, 20):
        tokens, logprobs, entropy = got[i]
        assert int(tokens[1]) == -1 and float(logprobs[1]) == 0 and float(entropy[1]) == 0
        assert (int(tokens[0]) == -1) == (i >= 18)
        if i < 18:
            assert abs(float(logprobs[0]) - float(want[i][1][0])) < 0.3
    # a block comes back: request 0, first in line and refused too, is left out; request 1 offers its token again
    last = torch.tensor([-1, int(got[11][0][1])], dtype=torch.int32, device="cuda")
    m.free[4:5] = spare
    m.free_head -= 1
    tokens, logprobs, entropy = next(m.decode(last, 1))
    assert m.lens.tolist() == [48, 33] and int(m.free_head) == 5 and fp8bs.check_device_error() == 0
    assert int(tokens[0]) == -1 and float(logprobs[0]) == 0 and int(tokens[1]) >= 0
    assert abs(float(logprobs[1]) - float(want[12][1][1])) < 0.3
    assert abs(float(entropy[1]) - float(want[12][2][1])) < 0.3
    for a, b in zip(keys(m, 1, 33), kept):
        assert torch.equal(a[:32].view(torch.int16), b.view(torch.int16))


def test_a_refused_prompt_is_left_out(example):  # noqa: F811
    import fp8_block_scaled_02_gb300 as fp8bs
    m = example.Decoder(batch=3, max_len=32)
    m.free = m.free[:4].clone()
    first = m.prompt([list(range(14)), list(range(40, 71)), list(range(7))])
    assert (first >= 0).tolist() == [True, True, True] and m.lens.tolist() == [14, 31, 7]
    assert fp8bs.check_device_error() == 0

    m = example.Decoder(batch=3, max_len=32)
    m.free = m.free[:2].clone()                                   # the second prompt needs two
    first = m.prompt([list(range(14)), list(range(40, 71)), list(range(7))])
    assert (first >= 0).tolist() == [True, False, False]          # handed out in order: the third waits too
    assert m.lens.tolist() == [14, 0, 0] and fp8bs.check_device_error() == 32
    for tokens, logprobs, entropy in m.decode(first, 3):
        assert (tokens >= 0).tolist() == [True, False, False]
        assert logprobs[1:].tolist() == entropy[1:].tolist() == [0, 0] and float(logprobs[0]) < 0
    assert m.lens.tolist() == [17, 0, 0] and fp8bs.check_device_error() == 0
