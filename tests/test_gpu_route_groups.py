"""GPU tests of fp8bs_moe_route where a group's two best experts cancel: a
large positive bias and a large negative one, so that the group's score is small
and what its parts lost in fp32 is not.  Ids have to be those of whole numbers."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib_or_skip
from route_reference import choose

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check(x, bias, topk, scoring, groups, topk_groups, group_top=2):
    pkg = lib_or_skip()
    ids, _ = pkg.moe_route(torch.from_numpy(x).to(DEV), topk, scoring=scoring, bias=torch.from_numpy(bias).to(DEV),
                           groups=groups, topk_groups=topk_groups, group_top=group_top)
    ids = ids.cpu().numpy()
    counted = 0
    for t in range(len(x)):
        want, _, clear = choose(x[t], topk, scoring, bias, groups, topk_groups, group_top)
        if clear:
            counted += 1
            assert ids[t].tolist() == want, t
    assert 10 * counted >= 9 * len(x)
    assert pkg.check_device_error() == 0


def test_the_smallest_case():
    """Scores 0.9999466 and 0.9999886; with each c rounded to fp32 1.0 and 0.9999390."""
    x = (np.array([[-40, 26, -56, 53]]) / 65536).astype(np.float32)
    check(x, np.array([1000, -1000, 1000, -1000], dtype=np.float32), 2, "sigmoid", 2, 1)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("large", [1.0, 16.0, 64.0, 333.25, 1000.0, 32768.0, 65536.0])
@pytest.mark.parametrize("groups,per,topk_groups", [(2, 2, 1), (16, 2, 5), (8, 32, 4), (5, 12, 2), (32, 4, 8), (3, 40, 1)])
def test_biases_that_cancel(groups, per, topk_groups, large, scoring):
    rng = np.random.default_rng(int(large) + groups)
    m, e = 64, groups * per
    # near scores, at several distances
    x = (rng.integers(-64, 65, (m, e)) / 65536 * 2.0 ** rng.integers(-3, 8, (m, 1))).astype(np.float32)
    bias = np.full((groups, per), -65536.0)                 # the others of a group come after its two
    two = np.stack([np.full(groups, large), np.full(groups, -large)], 1)
    for g in range(groups):
        bias[g, rng.permutation(per)[:2]] = two[g]
    check(x, bias.reshape(-1).astype(np.float32), 2, scoring, groups, topk_groups)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("groups,per,topk_groups", [(2, 2, 1), (8, 32, 4), (6, 20, 2), (32, 32, 8)])
def test_biases_of_both_signs(groups, per, topk_groups, group_top, scoring):
    """Random ones from 1 to 65536, each in steps of its own."""
    rng = np.random.default_rng(groups + per + group_top)
    m, e = 64, groups * per
    x = (rng.standard_normal((m, e)) * 1.5).astype(np.float32)
    for top in (1.0, 64.0, 4096.0, 65536.0):
        bias = (rng.choice([-1.0, 1.0], e) * np.exp(rng.uniform(0, np.log(top) + 1e-9, e))).astype(np.float32)
        check(x, bias, min(4, topk_groups * per), scoring, groups, topk_groups, group_top)
        # a few values only, so that groups and experts differ by their scores alone
        check(x, np.round(bias / top * 2).astype(np.float32) * np.float32(top / 2), min(4, topk_groups * per), scoring,
              groups, topk_groups, group_top)
