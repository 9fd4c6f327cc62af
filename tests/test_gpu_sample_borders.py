"""GPU tests of fp8bs_sample_tokens next to its borders: top_p on either side
of the mass of a few large tokens, and first random numbers on either side of a
block's, as near as include/fp8bs.h says that they are told apart.

A block's mass: a lane's two chains of 16 fp32 additions, their sum, the fma that
takes the exponents' losses back and 5 additions across the warp round by half a step
each, 23 2^-24, and ex2 is within 2^-22: 2^-19.2, and 2^-18 for the two masses that a first
number's border compares.  A cut compares the mass of all with that of the
histogram, whose weights are in steps of 2^-20, or of 2^-(5 + b) where tokens are counted too (with
top_k, or many equals), b = 18 to 2^14 tokens and one less for each doubling, at least 12: half a
step and 2^-22 of the series each, with top_k in both masses: 2^-17, above 2^18 tokens
2^-16.
"""
import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


def peaked(m, v, rng, large):
    """Rows of a few large tokens over a light bulk, fp32."""
    x = rng.standard_normal((m, v)) - 14.0
    for r in range(m):
        at = rng.permutation(v)[:large]
        x[r, at] = rng.uniform(0.0, 2.0, large)
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top_k", [0, 6, 50])
@pytest.mark.parametrize("m,v", [(320, 600), (64, 1000), (24, 32003), (8, 152064), (330, 20011), (2, 1 << 20)])
def test_top_p_on_either_side(m, v, top_k, dtype):
    pkg = lib_or_skip()
    rng = np.random.default_rng(m + v + top_k)
    far = 2.0 ** -16 if v > 1 << 18 and top_k else 2.0 ** -17
    x = torch.from_numpy(peaked(m, v, rng, 4)).to(dtype)
    t = rng.uniform(0.7, 1.3, m).astype(np.float32)
    p = {-1: [], 1: []}
    lps = {-1: [], 1: []}
    for r in range(m):
        row = x[r].double().numpy()
        kept, w = ref.kept_tokens(row, float(t[r]), top_k)
        upto = np.cumsum(w[kept])
        n = int(rng.integers(0, 3))
        for side in (-1, 1):
            at = upto[n] / upto[-1] * (1 + side * far)
            p[side].append(np.nextafter(np.float32(at), np.float32(2 * side)))      # its rounding does not come nearer
            count = n + 1 if side < 0 else n + 2
            first = min(kept[:count])                           # u = 0: the first kept token
            lps[side].append((first, np.log(w[first] / upto[count - 1])))
    k = None if top_k == 0 else torch.full((m,), top_k, dtype=torch.int32, device=DEV)
    for side in (-1, 1):
        got = pkg.sample_tokens(x.to(DEV), torch.zeros((m, 2), device=DEV), torch.from_numpy(t).to(DEV), top_k=k,
                                top_p=torch.tensor(np.array(p[side]), device=DEV))
        assert got.tokens.tolist() == [a for a, _ in lps[side]]
        # the kept tokens weigh some 2^-4 of the mass each: their number shows in the log probability
        want = np.array([b for _, b in lps[side]])
        assert np.all(np.abs(got.logprobs.cpu().double().numpy() - want) <= 2.0 ** -18 + 2.0 ** -22 * (np.abs(want) + 28))
    assert pkg.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p"])
@pytest.mark.parametrize("m,v", [(320, 2500), (64, 2048), (24, 32003), (8, 152064), (3, 1 << 20)])
def test_first_number_on_either_side(m, v, kind, dtype):
    pkg = lib_or_skip()
    rng = np.random.default_rng(m + v)
    far = 2.0 ** -18
    x = torch.from_numpy((rng.standard_normal((m, v)) * 1.5).astype(np.float32)).to(dtype)
    u = {-1: np.zeros((m, 2), dtype=np.float32), 1: np.zeros((m, 2), dtype=np.float32)}
    want = {-1: [], 1: []}
    p = np.full(m, 0.5, dtype=np.float32)
    for r in range(m):
        row = x[r].double().numpy()
        if kind == "top_p":                                     # halfway into a token's mass, of 500 kept ones
            order, w = ref.kept_tokens(row)
            upto = np.cumsum(w[order])
            p[r] = (upto[499] - 0.5 * w[order[499]]) / upto[-1]
        kept, w = ref.kept_tokens(row, 1.0, 500 if kind == "top_k" else 0, float(p[r]) if kind == "top_p" else 1.0)
        mass = np.zeros(-(-v // 1024) * 1024)
        mass[kept] = w[kept]
        blocks = np.cumsum(mass.reshape(-1, 1024).sum(1))
        while True:                                             # a border between blocks of some mass each
            b = int(rng.integers(0, len(blocks) - 1))
            if all(np.diff(np.concatenate([[0], blocks]))[b:b + 2] > 4 * far * blocks[-1]):
                break
        for side in (-1, 1):
            u[side][r, 0] = np.nextafter(np.float32(blocks[b] / blocks[-1] + side * far), np.float32(2 * side))
            u[side][r, 1] = 0.5
            want[side].append(ref.sample(row, float(u[side][r, 0]), 0.5, 1.0, 500 if kind == "top_k" else 0,
                                         float(p[r]) if kind == "top_p" else 1.0)[0])
            assert want[side][-1] // 1024 == b + (side > 0)
    kw = dict(top_k=torch.full((m,), 500, dtype=torch.int32, device=DEV)) if kind == "top_k" else \
        dict(top_p=torch.from_numpy(p).to(DEV)) if kind == "top_p" else {}
    for side in (-1, 1):
        got = pkg.sample_tokens(x.to(DEV), torch.from_numpy(u[side]).to(DEV), **kw).tokens.cpu().numpy()
        assert np.array_equal(got, want[side])
    assert pkg.check_device_error() == 0
