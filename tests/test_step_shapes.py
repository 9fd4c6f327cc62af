"""Tensors of the step's entry points have the shape that is documented, not
only as many elements: one of the transposed shape would be read in the wrong
order without a word.  The checks before a launch, on the CPU and, marked gpu, on
the quick path that CUDA tensors take."""
import pytest
import torch

import fp8_block_scaled_02_gb300 as fp8bs

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


def calls(device):
    def t(shape, dtype=F32):
        return torch.zeros(shape, dtype=dtype, device=device)

    def route(**kw):
        return fp8bs.moe_route(t((6, 16)), 2, **kw)

    def combine(weights=(6, 2), **kw):
        return fp8bs.moe_combine(t((6, 2, 64), BF), t(weights), **kw)

    def sample(u):
        return fp8bs.sample_tokens(t((6, 50), BF), t(u))

    def rope(cache, out):
        q, kv = t((4, 8, 128), BF), t((4, 2, 128), BF)
        at, c = torch.arange(4, dtype=I32, device=device), (t(cache, U8), t(cache, U8))
        fn = fp8bs.kv_rope_append if len(cache) == 4 and cache[1] == 16 else fp8bs.kv4_rope_append
        return fn(q, kv, kv, at, at, t((9, 64)), t(1) + 1, t(1) + 1, *c, out=t(out, BF))

    c8, c4 = (2, 16, 2, 128), (2, 2, 1, 1152)
    wrong = [lambda: route(ids=t((2, 6), I32)), lambda: route(ids=t(12, I32)), lambda: route(weights=t((2, 6))),
             lambda: route(weights=t((3, 4))), lambda: combine((2, 6)), lambda: combine((12,)),
             lambda: combine(ids=t((2, 6), I32), num_experts=4), lambda: combine(ids=t((4, 3), I32), num_experts=4),
             lambda: combine(residual=t((64, 6), BF)), lambda: combine(residual=t((3, 128), BF)),
             lambda: combine(out=t((64, 6), BF)), lambda: combine(out=t(384, BF)), lambda: sample((3, 2, 2)),
             lambda: sample((1, 6, 2)), lambda: rope(c8, (8, 4, 128)), lambda: rope(c8, (4, 1024)),
             lambda: rope(c4, (128, 8, 4)), lambda: rope(c4, (2, 16, 128))]
    right = [lambda: route(ids=t((6, 2), I32), weights=t((6, 2))),
             lambda: combine(ids=t((6, 2), I32), num_experts=4, residual=t((6, 64), BF), out=t((6, 64), BF)),
             lambda: sample((6, 2)), lambda: rope(c8, (4, 8, 128)), lambda: rope(c4, (4, 8, 128))]
    return wrong, right


@pytest.mark.parametrize("i", range(18))
def test_other_shapes_of_as_many_elements_raise(i):
    with pytest.raises(ValueError, match="has shape"):
        calls("cpu")[0][i]()


@pytest.mark.parametrize("i", range(5))
def test_the_documented_shapes_get_past_the_check(i):
    with pytest.raises(TypeError, match="CUDA"):
        calls("cpu")[1][i]()


@pytest.mark.gpu
def test_other_shapes_raise_on_the_gpu():
    from gpu_helpers import lib_or_skip
    pkg = lib_or_skip()
    wrong, right = calls("cuda")
    assert len(wrong) == 18 and len(right) == 5
    for call in wrong:
        with pytest.raises(ValueError, match="has shape"):
            call()
    for call in right:
        call()
    assert pkg.check_device_error() == 0
