"""GPU tests of fp8bs_moe_route with NaN in the biases: such an expert's c is
NaN, and it comes after every other, those shut out by a bias of -inf or of the
largest size included; a group with one among its best comes after the others."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib_or_skip
from route_reference import choose

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("e,topk,groups,topk_groups,group_top", [
    (6, 6, 1, 1, 1), (64, 32, 1, 1, 1), (40, 31, 1, 1, 1), (64, 8, 8, 3, 2), (64, 8, 8, 3, 1), (12, 6, 3, 2, 2),
    (256, 8, 8, 4, 2), (1000, 32, 8, 2, 2)])
@pytest.mark.parametrize("share", [0.1, 0.5, 0.9, 1.0])
def test_nan_bias_comes_last(e, topk, groups, topk_groups, group_top, share, scoring):
    pkg = lib_or_skip()
    rng = np.random.default_rng(e + topk + int(10 * share))
    x = (rng.standard_normal((40, e)) * 1.5).astype(np.float32)
    bias = (rng.standard_normal(e) * 0.1).astype(np.float32)
    bias[rng.random(e) < 0.3] = -np.inf
    bias[rng.random(e) < 0.2] = -65536.0
    bias[rng.random(e) < share] = np.nan
    ids, w = pkg.moe_route(torch.from_numpy(x).to(DEV), topk, scoring=scoring, bias=torch.from_numpy(bias).to(DEV),
                           groups=groups, topk_groups=topk_groups, group_top=group_top, renormalize=False)
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    counted = 0
    for t in range(len(x)):
        want, s, clear = choose(x[t], topk, scoring, bias, groups, topk_groups, group_top)
        if clear:
            counted += 1
            assert ids[t].tolist() == want, t
            assert np.all(np.abs(w[t] - s[want]) <= 2.0 ** -18 * s[want])      # the bias only chooses
    assert 10 * counted >= 9 * len(x)
    assert pkg.check_device_error() == 0
