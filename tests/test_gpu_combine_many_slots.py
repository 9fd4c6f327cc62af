"""GPU tests of fp8bs_moe_combine with more slots a token than a warp has lanes:
ids and weights are loaded 32 at a time.

topk fused multiply-adds round by half a step, 2^-24 of the running sum, below the
sum of the magnitudes; one bf16 rounding, 2^-8 of the result at most.
"""
import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import bits, guard_intact, guarded_empty, lib_or_skip
from oracle.tolerance import bf16_bits_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k,n", [(3, 33, 64), (2, 35, 7), (5, 64, 1032), (4, 100, 264), (1, 1024, 40), (2, 67, 1001)])
def test_more_slots_than_lanes(m, k, n, residual, dropped):
    pkg = lib_or_skip()
    g = torch.Generator().manual_seed(m + k + n)
    y = torch.randn((m, k, n), generator=g).to(torch.bfloat16)
    w = torch.randn((m, k), generator=g)
    res = (torch.randn((m, n), generator=g) * 3).to(torch.bfloat16) if residual else None
    ids, live = None, np.ones((m, k), dtype=bool)
    if dropped:
        ids = torch.randint(-2, 10, (m, k), generator=g).to(torch.int32)
        ids[0, :32] = -1                                        # none of the first 32
        ids[-1, 32:] = 9                                        # none of the others
        live = ((ids >= 0) & (ids < 7)).numpy()
        y[torch.from_numpy(~live)] = float("nan")               # is not read
    out, raw = guarded_empty((m, n), torch.bfloat16, DEV)
    dev = [None if t is None else t.to(DEV) for t in (y, w, ids, res)]
    pkg.moe_combine(dev[0], dev[1], ids=dev[2], num_experts=7 if dropped else 0, residual=dev[3], out=out)
    assert guard_intact(raw, m * n * 2)
    y64 = np.where(live[..., None], bf16_bits_to_f64(bits(y)), 0.0)
    r64 = None if res is None else bf16_bits_to_f64(bits(res))
    want = ref.combine(y64, w.double().numpy(), residual=r64)
    size = ref.combine(np.abs(y64), np.abs(w.double().numpy()), residual=None if res is None else np.abs(r64))
    tol = k * 2.0 ** -24 * size
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -133
    assert np.all(np.abs(bf16_bits_to_f64(bits(out.cpu())) - want) <= tol)
    assert pkg.check_device_error() == 0
