"""GPU tests of fp8bs_sample_tokens by top-p alone on rows of fewer blocks than
a CTA has warps, many times over: a warp without a block reaches the next step
while others are still in the one before, and results may not depend on that.

Each row's top_p lies halfway into the mass of one token of at least 2^-12 of all,
and its random numbers are at least 2^-16 from a border: far more than what masses
are off by (16 + 1 + 1 + 5 fp32 additions and ex2's 2^-22: below 2^-19 of the mass).
"""
import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = 2.0 ** -16


def a_row(x, rng, temperature):
    """top_p, u, token and log probability of a row, clear of every border."""
    order = np.lexsort((np.arange(len(x)), -x))
    w = np.exp((x[order] - x[order[0]]) / temperature)
    upto = np.cumsum(w)
    large = int((w >= 2.0 ** -12 * upto[-1]).sum())
    n = int(rng.integers(0, max(large, 1)))
    top_p = float(np.float32((upto[n] - 0.5 * w[n]) / upto[-1]))
    while True:
        u = rng.random(2).astype(np.float32)
        token, lp, near = ref.sample(x, float(u[0]), float(u[1]), temperature, top_p=top_p)
        if near >= FAR:
            return top_p, u, token, lp


# 1, 3, 5 and 15 blocks on 16 warps, a CTA a row; 69 and 30 blocks on a cluster, 8 or 9 and 7 or 8 a CTA
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v", [(320, 700), (320, 2500), (330, 5000), (310, 15001), (4, 70001), (40, 30003)])
def test_top_p_alone_again_and_again(m, v, dtype):
    pkg = lib_or_skip()
    rng = np.random.default_rng(m + v)
    x = torch.from_numpy(rng.standard_normal((m, v)) * 2.0).to(dtype)
    temperature = rng.uniform(0.4, 1.2, m).astype(np.float32)
    rows = [a_row(x[r].double().numpy(), rng, float(temperature[r])) for r in range(m)]
    want = torch.tensor([r[2] for r in rows], dtype=torch.int32)
    want_lp = torch.tensor([r[3] for r in rows], dtype=torch.float64)
    args = (x.to(DEV), torch.tensor(np.stack([r[1] for r in rows]), device=DEV), torch.tensor(temperature, device=DEV))
    top_p = torch.tensor([r[0] for r in rows], dtype=torch.float32, device=DEV)
    first = pkg.sample_tokens(*args, top_p=top_p)
    assert torch.equal(first.tokens.cpu(), want)
    # log p: two fp32 rounded once and logf, 2^-22 of |log p| + log W <= 14 each way; W within 2^-19
    assert bool(((first.logprobs.cpu().double() - want_lp).abs() <= 2.0 ** -19 + 2.0 ** -22 * (want_lp.abs() + 28)).all())
    other = torch.full((m,), 0.5, device=DEV)
    for i in range(200):
        if i % 3 == 2:
            pkg.sample_tokens(*args, top_p=other)               # other sums before the next call's
        again = pkg.sample_tokens(*args, top_p=top_p)
        assert torch.equal(again.tokens, first.tokens) and torch.equal(again.logprobs, first.logprobs), i
    assert pkg.check_device_error() == 0
