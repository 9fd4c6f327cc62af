"""Pins of the plain references in step_reference.py (CPU only): rotation
against complex numbers and its inverse, stores against torch's casts and the
appends' reference, routing against torch's topk and brute force, sampling
against closed forms and its shares, and that the bounds used on the GPU's
outputs reject planted mistakes."""
import itertools
import math

import numpy as np
import pytest
import torch

import serving_reference as serving
import step_reference as ref
from oracle.tolerance import bf16_bits_to_f64

F32 = np.float32


def bf16_bits(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def angles(t, rot):
    a = np.arange(t)[:, None] * 100.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(a).astype(F32), np.sin(a).astype(F32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64])
def test_rotation_is_a_product_of_complex_numbers(rot, interleaved):
    x = bf16_bits(np.random.default_rng(0).standard_normal((9, 3, 64)))
    cos, sin = angles(9, rot)
    v = bf16_bits_to_f64(x)
    a, b = (v[..., 0:rot:2], v[..., 1:rot:2]) if interleaved else (v[..., :rot // 2], v[..., rot // 2:rot])
    z = (a + 1j * b) * (cos.astype(np.float64) + 1j * sin)[:, None]
    want = v.copy()
    if interleaved:
        want[..., 0:rot:2], want[..., 1:rot:2] = z.real, z.imag
    else:
        want[..., :rot // 2], want[..., rot // 2:rot] = z.real, z.imag
    assert np.allclose(ref.turned(x, None, 0, cos, sin, interleaved, rounded=False), want, rtol=1e-14, atol=1e-14)
    got = ref.turned(x, None, 0, cos, sin, interleaved)
    assert np.all(got == got.astype(F32)) and np.all(np.abs(got - want) <= 3 * 2.0 ** -24 * 2 * np.abs(v).max())
    assert np.array_equal(got[0], v[0])                          # position 0 turns nothing


def test_norm_makes_heads_of_one_size():
    rng = np.random.default_rng(1)
    x = bf16_bits(rng.standard_normal((5, 4, 128)) * 10.0 ** rng.uniform(-3, 3, (5, 4, 1)))
    one, cs = bf16_bits(np.ones(128)), angles(5, 128)
    got = ref.turned(x, one, 0.0, *cs, False, rounded=False)
    assert np.allclose((got * got).mean(-1), 1.0, atol=1e-6)     # cos^2 + sin^2 in fp32
    v = torch.from_numpy(bf16_bits_to_f64(x))
    still = ref.turned(x, one, 1e-6, np.ones((5, 64), F32), np.zeros((5, 64), F32), False, rounded=False)
    assert np.allclose(still, torch.nn.functional.rms_norm(v, (128,), eps=float(F32(1e-6))).numpy(), rtol=1e-12)


def test_stores_are_those_of_the_appends():
    rng = np.random.default_rng(2)
    x = bf16_bits(rng.standard_normal((7, 2, 64)))
    slots = np.array([31, 0, 15, -1, 47, 48, 7])
    cache = rng.integers(0, 100, (3, 2, 1, 9 * 64), dtype=np.uint8)
    assert np.array_equal(ref.store4(bf16_bits_to_f64(x), slots, 0.01, cache), serving.append(x, slots, 0.01, cache))
    c8 = rng.integers(0, 100, (3, 16, 2, 64), dtype=np.uint8)
    got = ref.store8(bf16_bits_to_f64(x), slots, 0.01, c8)
    want = torch.from_numpy(c8.copy()).view(-1, 2, 64)
    v = (torch.from_numpy(bf16_bits_to_f64(x)).float() / 0.01).to(torch.float8_e4m3fn).view(torch.uint8)
    for t, s in enumerate(slots):
        if 0 <= s < 48:
            want[s] = v[t]
    assert np.array_equal(got.reshape(-1, 2, 64), want.numpy())
    assert ref.e4m3_codes(np.array([1e9, -1e9, np.nan, -0.0], F32)).tolist() == [126, 254, 127, 128]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_routing_is_torchs_topk(scoring):
    x = torch.randn((40, 24), generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    s = x.softmax(1) if scoring == "softmax" else x.sigmoid()
    want, ids = s.topk(5)
    got_ids, got = ref.route(x.numpy(), 5, scoring, renormalize=False, scale=2.5)
    assert np.array_equal(got_ids, ids.numpy()) and np.allclose(got, 2.5 * want.numpy(), rtol=1e-13)
    _, got = ref.route(x.numpy(), 5, scoring)
    assert np.allclose(got.sum(1), 1) and np.allclose(got, (want / want.sum(1, keepdim=True)).numpy())


def test_grouped_routing_by_brute_force():
    """All pairs of groups: the open ones have the largest sum of two; all sets of experts: the chosen ones the largest c."""
    rng = np.random.default_rng(4)
    x, bias = rng.standard_normal((30, 12)), rng.standard_normal(12).astype(F32) * 0.2
    ids, w = ref.route(x, 3, "sigmoid", bias, groups=4, topk_groups=2, group_top=2, renormalize=False)
    for t in range(30):
        s = 1 / (1 + np.exp(-x[t]))
        c = s + bias
        two = [np.sort(c[3 * g:3 * g + 3])[1:].sum() for g in range(4)]
        pair = max(itertools.combinations(range(4), 2), key=lambda p: two[p[0]] + two[p[1]])
        live = [e for e in range(12) if e // 3 in pair]
        best = max(itertools.combinations(live, 3), key=lambda p: sum(c[list(p)]))
        assert set(ids[t]) == set(best) and np.all(np.diff(c[ids[t]]) <= 0) and np.allclose(w[t], s[ids[t]])


def test_routing_without_anything():
    ids, w = ref.route(np.full((1, 6), -math.inf), 2, "softmax")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0, 0]]
    x = np.array([[1.0, math.nan, 3.0, 3.0]])
    assert ref.route(x, 4, "sigmoid")[0].tolist() == [[2, 3, 0, 1]]


def test_combination_is_einsum():
    rng = np.random.default_rng(5)
    y, w, r = rng.standard_normal((4, 3, 8)), rng.random((4, 3)), rng.standard_normal((4, 8))
    assert np.allclose(ref.combine(y, w, residual=r), np.einsum("tkn,tk->tn", y, w) + r)
    ids = np.array([[0, 1, -1], [2, 2, 2], [0, 5, 4], [7, 7, 7]])
    live = (ids >= 0) & (ids < 5)
    y[~live] = np.nan
    assert np.allclose(ref.combine(y, w, ids, 5), np.einsum("tkn,tk->tn", np.where(live[..., None], y, 0), w))


def test_kept_tokens_in_closed_form():
    x = np.log(np.array([0.1, 0.4, 0.05, 0.25, 0.2]))
    kept = lambda **kw: ref.kept_tokens(x, **kw)[0].tolist()     # noqa: E731
    assert kept() == [1, 3, 4, 0, 2]
    assert kept(top_k=2) == [1, 3] and kept(top_k=9) == [1, 3, 4, 0, 2] and kept(temperature=0) == [1]
    assert kept(top_p=0.39) == [1] and kept(top_p=0.41) == [1, 3] and kept(top_p=0.86) == [1, 3, 4, 0]
    assert kept(top_p=0) == [1] and kept(min_p=0.49) == [1, 3, 4] and kept(min_p=2) == [1]
    assert kept(top_k=3, top_p=0.75) == [1, 3]                   # 0.65 of 0.85 reaches 0.75
    assert ref.kept_tokens(np.zeros(4), top_k=3)[0].tolist() == [0, 1, 2]


def test_sampling_in_closed_form():
    x = np.log(np.array([0.1, 0.4, 0.05, 0.25, 0.2]))
    for u, want in ((0.0, 0), (0.09, 0), (0.11, 1), (0.49, 1), (0.51, 2), (0.56, 3), (0.81, 4), (0.999, 4)):
        token, lp, _ = ref.sample(x, 0.5, u)
        assert token == want and math.isclose(lp, x[want], abs_tol=1e-12)
    two = np.full(1500, -math.inf)
    two[[3, 1400]] = 0.0                                         # a token in each of two blocks
    assert [ref.sample(two, u, 0.3)[0] for u in (0.0, 0.49, 0.51, 0.99)] == [3, 3, 1400, 1400]
    for bad in (dict(temperature=-1.0), dict(top_p=math.nan), dict(temperature=math.inf)):
        assert ref.sample(x, 0.5, 0.5, **bad)[:2] == (-1, 0.0)
    assert ref.sample(np.array([1.0, math.nan]), 0.5, 0.5)[0] == ref.sample(np.full(3, -math.inf), 0.5, 0.5)[0] == -1


def test_draws_have_their_shares():
    """Over a grid of 64 x 64 of both numbers each token is drawn as often as its probability says, up to the grid: a
    block's border moves its share by one row of 64, a token's by one column."""
    rng = np.random.default_rng(6)
    x = np.concatenate([rng.standard_normal(6), np.full(1018, -math.inf), rng.standard_normal(4)])
    p = np.exp(x) / np.exp(x).sum()
    grid = (np.arange(64) + 0.5) / 64
    got = np.zeros(len(x))
    for u0 in grid:
        for u1 in grid:
            got[ref.sample(x, u0, u1)[0]] += 1 / 4096
    assert np.all(np.abs(got - p) <= 2 / 64) and got.sum() == pytest.approx(1)


def test_the_bounds_on_q_reject_mistakes():
    """The bound of the GPU tests, 14 half steps of fp32 and half a step of bf16, against planted mistakes: the sin
    of the next position, a mean over one element fewer, an eps left out, the pairs of the other layout."""
    rng = np.random.default_rng(7)
    x, w = bf16_bits(rng.standard_normal((8, 2, 128)) * 1e-2), bf16_bits(1 + 0.2 * rng.standard_normal(128))
    cos, sin = angles(9, 128)
    want = ref.turned(x, w, 1e-6, cos[:8], sin[:8], False, rounded=False)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max(-1, keepdims=True)
    assert np.all(np.abs(ref.turned(x, w, 1e-6, cos[:8], sin[:8], False) - want) <= tol)
    assert np.any(np.abs(ref.turned(x, w, 1e-6, cos[:8], sin[1:], False) - want) > tol)
    assert np.any(np.abs(want * math.sqrt(127 / 128) - want) > tol)
    assert np.any(np.abs(ref.turned(x, w, 0.0, cos[:8], sin[:8], False) - want) > tol)
    assert np.any(np.abs(ref.turned(x, w, 1e-6, cos[:8], sin[:8], True) - want) > tol)
