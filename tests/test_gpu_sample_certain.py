"""GPU tests of fp8bs_sample_tokens where one token has nearly all the mass: its
log probability, -log(1 + rest), keeps its relative precision however small it is.

The drawn block's mass is summed from pairs of fp32 in steps of 2^-45, the other blocks'
are within 2^-19.2 of themselves, as the rest is in sum, and in steps of 2^-41 of the largest
weight: 2^-19 of the log probability, and 2^-42 for each of up to 150 blocks and of
as many tokens at a cut: 2^-34.
"""
import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p", "min_p"])
@pytest.mark.parametrize("m,v", [(6, 40), (8, 1000), (320, 3001), (4, 32003), (1, 152064), (40, 20011)])
def test_log_probability_of_a_certain_token(m, v, kind, dtype):
    pkg = lib_or_skip()
    rng = np.random.default_rng(m + v)
    x = rng.standard_normal((m, v))
    best = rng.integers(0, v, m)
    above = np.linspace(12.0, 28.0, m) if m > 1 else np.array([16.0])
    x[np.arange(m), best] = above
    x = torch.from_numpy(x).to(dtype)
    kw, one = {}, [{} for _ in range(m)]
    if kind == "top_k":
        kw = dict(top_k=torch.full((m,), 20, dtype=torch.int32, device=DEV))
        one = [dict(top_k=20)] * m
    if kind == "min_p":
        p = np.exp(2.0 - above).astype(np.float32)              # tokens above 2 are kept, none of them near it
        x = torch.where((x.double() - 2.0).abs() < 0.01, torch.zeros_like(x), x)
        kw, one = dict(min_p=torch.from_numpy(p).to(DEV)), [dict(min_p=float(a)) for a in p]
    if kind == "top_p":
        tops = []
        for r in range(m):                                      # halfway into the mass of the second token
            order, w = ref.kept_tokens(x[r].double().numpy())
            p = np.float32((w[order[0]] + 0.5 * w[order[1]]) / w.sum())
            # 1 where fp32 cannot say it: all are kept
            tops.append(p if p < 1 and 2.0 ** -17 < 0.5 * w[order[1]] / w.sum() else np.float32(1.0))
        kw, one = dict(top_p=torch.tensor(np.array(tops), device=DEV)), [dict(top_p=float(a)) for a in tops]
    u = torch.full((m, 2), 0.5, device=DEV)
    got = pkg.sample_tokens(x.to(DEV), u, **kw)
    assert got.tokens.tolist() == best.tolist()
    for r in range(m):
        kept, w = ref.kept_tokens(x[r].double().numpy(), 1.0, **one[r])
        want = -np.log1p(np.sort(w[kept])[:-1].sum())           # the largest's weight is 1
        have = float(got.logprobs[r])
        assert abs(have - want) <= 2.0 ** -19 * abs(want) + 2.0 ** -34, (r, have, want)
    assert pkg.check_device_error() == 0
