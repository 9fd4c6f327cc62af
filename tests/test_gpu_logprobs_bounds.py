"""fp8bs_token_logprobs against float64 where a thread adds the most terms:
rows that are a CTA of 128 threads each, with a bound for what the kernel
does there.

l = sum 2^d over the row, d = x log2 e - r with a reference r of the thread
that lies at most 5 (in log2) below its maximum.  A thread of the smallest CTA
adds V / 128 terms one after the other, the merges of the warp, the CTA and the
cluster fewer than 64 (half a step, 2^-24, each).  A term is off by an exp2
(2^-22) and by the roundings of d and of log2 e, 2^-24 and 2^-25 of |d|, whose
mean under the weights is the row's dist = |t / l| in log2, and the lag of 5.
Moving the reference, bringing it to the maximum and the three merges multiply
by an exp2 each (five, and the sums before a move weigh 2^-5 of those after):
    r = (V / 128 + 64) 2^-24 + 7 2^-22 + (dist log2 e + 5) 2^-23
and log l moves by r.  t = sum d 2^d moves by r of sum |d| 2^d, so the entropy
log l - t / l by r (1 + 2 (dist + 5 ln 2)).  The differences and the logarithm
round by 2^-22 of what they hold, |log p| or dist and log l < 12.
"""
import math

import numpy as np
import pytest
import torch

import serving_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


@pytest.mark.parametrize("dtype,v", [(torch.bfloat16, 66003), (torch.float32, 33003), (torch.float32, 9001)])
@pytest.mark.parametrize("m,top", [(613, 5), (1230, 0)])
def test_the_longest_sums(pkg, m, top, dtype, v):
    g = torch.Generator().manual_seed(v + m)
    x = torch.randn((m, v), generator=g) * 2.0
    x[0::7] = 0.25                                                # equals: every rounding on the same side
    x[1::7] = torch.linspace(-3, 3, v)                            # rising: the reference is always behind
    x[2::7] = torch.linspace(0, 40, v)                            # and has to move
    x[3::7] = torch.linspace(5, -5, v)
    x[4::7, v // 3:] = -math.inf
    x = x.to(dtype)
    t = np.random.default_rng(m).integers(0, v // 3, m)
    got = pkg.token_logprobs(x.to(DEV), torch.tensor(t, dtype=torch.int32, device=DEV), top)
    with np.errstate(invalid="ignore"):
        want, dist = ref.logprobs(x.double().numpy(), t, top)
    r = (v / 128 + 64) * 2.0 ** -24 + 7 * 2.0 ** -22 + (dist * math.log2(math.e) + 5) * 2.0 ** -23
    e = np.abs(got.logprobs.cpu().numpy() - want["logprobs"])
    assert np.all(e <= r + 2.0 ** -22 * (np.abs(want["logprobs"]) + 12)), e.max()
    e = np.abs(got.entropy.cpu().numpy() - want["entropy"])
    assert np.all(e <= r * (1 + 2 * (dist + 5 * math.log(2))) + 2.0 ** -22 * (12 + dist)), e.max()
    assert np.array_equal(got.top_ids.cpu().numpy(), want["top_ids"])
    if top:
        e = np.abs(got.top_logprobs.cpu().numpy() - want["top_logprobs"])
        assert np.all(e <= r[:, None] + 2.0 ** -22 * (np.abs(want["top_logprobs"]) + 12)), e.max()
    assert pkg.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v", [(4, 6000), (3, 152064), (700, 3001)])
def test_a_row_of_nothing_but_nan(pkg, m, v, dtype):
    """No token of it is among its top; the other rows keep every bit."""
    x = (torch.randn((m, v), generator=torch.Generator().manual_seed(v)) * 2).to(dtype).to(DEV)
    t = torch.zeros(m, dtype=torch.int32, device=DEV)
    clean = pkg.token_logprobs(x, t, 20)
    x[1] = float("nan")
    r = pkg.token_logprobs(x, t, 20)
    assert bool((r.top_ids[1] == -1).all())
    others = torch.arange(m, device=DEV) != 1
    for a, b in zip(r, clean):
        assert torch.equal(a[others], b[others])
    assert pkg.check_device_error() == 0
