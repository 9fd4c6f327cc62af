"""GPU tests of fp8bs_moe_route where large biases leave the choice to scores
far apart from each other in multiples of 2^-44, but not in what a number near
the bias can hold."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib_or_skip
from route_reference import choose

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("large", [0.03125, 1.0, 300.5, 65536.0, -65536.0, -7.25])
@pytest.mark.parametrize("e,topk,groups,topk_groups", [(2, 1, 1, 1), (31, 8, 1, 1), (64, 32, 1, 1), (64, 4, 8, 3), (256, 8, 8, 4)])
def test_scores_decide_beside_any_bias(e, topk, groups, topk_groups, large, scoring):
    """Logits in steps of 2^-32: sigmoid scores differ by 2^-34, softmax ones by 2^-32 / e: 64 units and more."""
    pkg = lib_or_skip()
    rng = np.random.default_rng(e)
    x = np.stack([rng.permutation(e) for _ in range(32)]).astype(np.float32) * np.float32(2.0 ** -32)
    bias = np.full(e, large, dtype=np.float32)
    bias[rng.random(e) < 0.5] = np.float32(large - 1.0)        # the scores decide among equal ones
    if groups > 1:
        bias[:] = np.float32(large)
    ids, _ = pkg.moe_route(torch.from_numpy(x).to(DEV), topk, scoring=scoring, bias=torch.from_numpy(bias).to(DEV),
                           groups=groups, topk_groups=topk_groups, group_top=min(groups, 2))
    counted = 0
    for t, got in enumerate(ids.cpu().tolist()):
        want, _, clear = choose(x[t], topk, scoring, bias, groups, topk_groups, min(groups, 2))
        if clear:
            counted += 1
            assert got == want, t
    assert 4 * counted >= 3 * len(x)                        # sums of two can be equal
    assert pkg.check_device_error() == 0
