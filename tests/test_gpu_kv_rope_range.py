"""GPU tests of the norm at the ends of the range in which include/fp8bs.h
defines its roundings: |a| just below 2^50, and mean a^2 just above 2^-100 with eps = 0.
Caches bit for bit, q within its roundings."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib_or_skip
from test_gpu_kv_rope import inputs_of, run, table, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,d", [(4, 128), (4, 64), (8, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("log_scale", [-49, 0, 47])             # the largest of some 10^5 normal numbers is below 6
def test_ends_of_the_range(bits, d, interleaved, log_scale):
    pkg = lib_or_skip()
    t, hq, hkv, page = 300, 2, 2, 16
    x = inputs_of(t, hq, hkv, d, 50 + log_scale, 2.0 ** log_scale)
    heads = x.double().view(t, -1, d)
    assert float(heads.abs().max()) < 2.0 ** 50 and float(heads.square().mean(-1).min()) >= 2.0 ** -100
    run(pkg, bits, x, hq, hkv, d, np.arange(t), np.arange(t), table(300, d), page, t // page + 1, weights(d, 1), weights(d, 2),
        interleaved, eps=0.0, vs=np.float32(2.0 ** (log_scale - 7)))
