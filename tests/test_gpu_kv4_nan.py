"""NaN in the 4-bit cache and in the queries: a row is touched by what it
sees and by nothing else.

A NaN key or value is stored as a NaN scale of its group of 16.  Against the
same call without it: a row that does not see the key (it is behind the row's
own position, or before its window) keeps every bit; a row that sees it is NaN
in the 16 elements of a value's group, or as a whole where a key or the query
is NaN, as sum_l w_l V_l and the softmax are.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import bits, lib_or_skip
from test_gpu_kv4 import attend, layer, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def poisoned(cache, table, b, key, head, group):
    """The cache with a NaN scale (the e4m3 code 0x7F or, for odd keys, 0xFF) in one group of one key."""
    c = cache.copy()
    page, d = c.shape[2] * 16, c.shape[3] // 9
    blk, off = table[b, key // page], key % page
    c[blk, head, off // 16, 8 * d + off % 16 * (d // 16) + group] = 0xFF if key & 1 else 0x7F
    return c


def rows_that_see(cu, lens, b, key, window):
    n = cu[b + 1] - cu[b]
    at = [lens[b] - n + i for i in range(n)]
    return np.array([key <= p and (not window or key > p - window) for p in at], dtype=bool)


def run(pkg, q, kc, vc, table, lens, cu, window, sm):
    o, lse = attend(pkg, q, kc, vc, table, lens, sm, cu_q=cu, max_q=int(np.diff(cu).max()), window=window)
    assert pkg.check_device_error() == 0
    return bits(o.cpu()), lse.cpu().numpy()


def is_nan(o):
    return (o & 0x7FFF) > 0x7F80


# lengths, query tokens, window, poisoned (sequence, key)
CASES = [([20, 33], [4, 1], 0, [(0, 18), (0, 19), (0, 3), (1, 32)]),
         ([47], [7], 0, [(0, 40), (0, 44), (0, 46), (0, 10)]),
         ([130, 90], [3, 2], 17, [(0, 111), (0, 112), (0, 113), (0, 129), (1, 72), (1, 88), (1, 89)]),
         ([2500], [4], 0, [(0, 2497), (0, 2499), (0, 1000), (0, 0)]),
         ([1500, 16], [1, 1], 700, [(0, 799), (0, 800), (0, 1499), (1, 15)])]


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (8, 1, 128), (12, 2, 128), (16, 1, 64), (4, 2, 64)])
@pytest.mark.parametrize("lens,qls,window,keys", CASES)
@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_keys_and_values(pkg, where, lens, qls, window, keys, hq, hkv, d):
    cu = np.concatenate([[0], np.cumsum(qls)])
    kc, vc, table = layer(lens, hkv, d, 16, 71)
    q = normal((int(cu[-1]), hq, d), 72)
    sm = d ** -0.5
    o, lse = run(pkg, q, kc, vc, table, lens, cu, window, sm)
    assert not is_nan(o).any() and np.isfinite(lse).all()
    for b, key in keys:
        head, group, per = hkv - 1, d // 16 - 1 - key % 3, hq // hkv
        if where == "k":
            o2, lse2 = run(pkg, q, poisoned(kc, table, b, key, head, group), vc, table, lens, cu, window, sm)
        else:
            o2, lse2 = run(pkg, q, kc, poisoned(vc, table, b, key, head, group), table, lens, cu, window, sm)
        hit = np.zeros((int(cu[-1]), hq), dtype=bool)
        hit[cu[b]:cu[b + 1], head * per:(head + 1) * per] = rows_that_see(cu, lens, b, key, window)[:, None]
        want = np.zeros(o.shape, dtype=bool)
        if where == "k":
            want[hit] = True
        else:
            want[hit, 16 * group:16 * group + 16] = True
        assert np.array_equal(is_nan(o2), want), (b, key)
        assert np.array_equal(o2[~want], o[~want]), (b, key)
        assert np.array_equal(np.isnan(lse2), hit if where == "k" else np.zeros_like(hit)), (b, key)
        assert np.array_equal(lse2[~np.isnan(lse2)], lse[~np.isnan(lse2)]), (b, key)


@pytest.mark.parametrize("lens,qls", [([20], [1]), ([5, 300], [3, 2]), ([3000], [4])])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 1, 64)])
def test_nan_queries(pkg, lens, qls, hq, hkv, d):
    """A NaN query is not taken for a row that sees no key (o = 0, lse = -inf)."""
    cu = np.concatenate([[0], np.cumsum(qls)])
    kc, vc, table = layer(lens, hkv, d, 16, 73)
    q = normal((int(cu[-1]), hq, d), 74)
    o, lse = run(pkg, q, kc, vc, table, lens, cu, 0, 0.1)
    q2 = q.clone()
    q2[-1, 1, 5] = float("nan")
    q2[0, hq - 1] = float("nan")
    o2, lse2 = run(pkg, q2, kc, vc, table, lens, cu, 0, 0.1)
    hit = np.zeros((int(cu[-1]), hq), dtype=bool)
    hit[-1, 1] = hit[0, hq - 1] = True
    assert np.array_equal(is_nan(o2), np.broadcast_to(hit[..., None], o.shape))
    assert np.array_equal(np.isnan(lse2), hit)
    assert np.array_equal(o2[~hit], o[~hit]) and np.array_equal(lse2[~hit], lse[~hit])


def test_a_far_smaller_weight_still_counts(pkg):
    """The sequence's maximum is elsewhere, by more than fp32's range of weights: 0 times NaN is NaN."""
    lens, hq, d = [2000], 8, 128
    kc, vc, table = layer(lens, 1, d, 16, 75)
    q = normal((1, hq, d), 76, 30.0)
    cu = np.array([0, 1])
    o, _ = run(pkg, q, kc, vc, table, lens, cu, 0, 0.5)
    for key in (3, 500, 1999):
        o2, _ = run(pkg, q, kc, poisoned(vc, table, 0, key, 0, 2), table, lens, cu, 0, 0.5)
        want = np.zeros(o.shape, dtype=bool)
        want[:, :, 32:48] = True
        assert np.array_equal(is_nan(o2), want), key
        assert np.array_equal(o2[~want], o[~want]), key
