"""GPU tests of fp8bs_moe_route and fp8bs_moe_combine against float64.

Ids have to be equal.  Weights: the exponential is within 2^-22 (ex2) + 2^-23,
the sum over all experts by as much and the roundings of its 32 + 5 additions at
most (E = 1024), half a step each and each of a part of the sum only (8 + 5 of
them to E = 256); the quotient, the sum of the chosen by five additions, its quotient and the
product with the scale round by half a step: (4 + 2 + 37 + 8) 2^-24 < 2^-18 of the
weight, below 2^-19 to E = 256.
Combine: topk fused multiply-adds round by 2^-24 of the running sum, below
the sum of the magnitudes; one bf16 rounding, 2^-8 of the result at most.
"""
import math

import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import bits, guard_intact, guarded_empty, lib_or_skip
from oracle.tolerance import bf16_bits_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def check(pkg, x, topk, bias=None, **kw):
    """x: CPU tensor [M, E]."""
    m = len(x)
    ids, raw_i = guarded_empty((m, topk), torch.int32, DEV)
    w, raw_w = guarded_empty((m, topk), torch.float32, DEV)
    got = pkg.moe_route(x.to(DEV), topk, bias=None if bias is None else bias.to(DEV), ids=ids, weights=w, **kw)
    assert got[0] is ids and guard_intact(raw_i, m * topk * 4) and guard_intact(raw_w, m * topk * 4)
    kw.setdefault("scoring", "softmax")
    want_i, want_w = ref.route(x.double().numpy(), topk, bias=None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), want_i)
    w = w.cpu().double().numpy()
    nan = np.isnan(want_w)
    assert np.array_equal(np.isnan(w), nan)
    e = np.abs(w - want_w)[~nan]
    assert np.all(e <= 2.0 ** (-19 if x.shape[1] <= 256 else -18) * np.abs(want_w)[~nan] + 2.0 ** -126), e.max()
    assert pkg.check_device_error() == 0
    return ids


def logits(m, e, seed, dtype=torch.float32, scale=1.5):
    return (torch.randn((m, e), generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,e,topk", [(1, 1, 1), (3, 2, 2), (7, 31, 5), (5, 32, 32), (9, 33, 8), (4, 60, 4), (33, 64, 6),
                                      (2, 129, 32), (65, 256, 12), (11, 384, 8), (3, 1000, 17), (2, 1024, 32)])
def test_matches_float64(pkg, m, e, topk, scoring, dtype):
    x = logits(m, e, m + e, dtype)
    check(pkg, x, topk, scoring=scoring)
    bias = torch.randn(e, generator=torch.Generator().manual_seed(e)) * 0.1
    check(pkg, x, topk, bias, scoring=scoring, renormalize=False, scale=2.5)


@pytest.mark.parametrize("scoring,with_bias", [("sigmoid", True), ("softmax", False), ("softmax", True)])
@pytest.mark.parametrize("m,e,topk,groups,topk_groups,group_top", [
    (50, 256, 8, 8, 4, 2), (9, 160, 6, 8, 3, 1), (5, 60, 4, 4, 2, 2), (3, 1024, 32, 32, 7, 2), (7, 12, 2, 12, 3, 1),
    (4, 33, 11, 3, 1, 2), (6, 64, 16, 2, 2, 1), (3, 100, 3, 20, 1, 2), (70, 160, 6, 8, 3, 2), (5, 384, 8, 8, 4, 2),
    (7, 93, 5, 3, 2, 1), (3, 1023, 8, 31, 4, 2), (4, 70, 4, 7, 3, 2), (5, 333, 9, 9, 2, 2)])
def test_groups(pkg, m, e, topk, groups, topk_groups, group_top, scoring, with_bias):
    x = logits(m, e, e + topk)
    bias = torch.randn(e, generator=torch.Generator().manual_seed(1)) * 0.05 if with_bias else None
    check(pkg, x, topk, bias, scoring=scoring, groups=groups, topk_groups=topk_groups, group_top=group_top)


def test_many_tokens(pkg):
    x = logits(5000, 256, 3)
    check(pkg, x, 12)
    bias = torch.randn(256, generator=torch.Generator().manual_seed(1)) * 0.05
    check(pkg, x[:3001], 8, bias, scoring="sigmoid", groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_near_ties(pkg, scoring):
    """Scores a few of their own fp32 steps apart, or equal, ordered by what 24 bits do not hold."""
    g = torch.Generator().manual_seed(5)
    base = torch.rand((64, 1), generator=g) * 4 - 2
    x = base * (1 + torch.randint(-3, 4, (64, 128), generator=g) * 2.0 ** -24)
    bias = torch.randint(-2, 3, (128,), generator=g).float() * 2.0 ** -30
    check(pkg, x, 16, scoring=scoring)
    check(pkg, x, 16, bias, scoring=scoring)
    check(pkg, x, 16, bias, scoring=scoring, groups=16, topk_groups=5, group_top=2)
    # the bias makes up for the score's difference to some 2^-30
    y = logits(40, 128, 6).double()
    s = torch.softmax(y, 1) if scoring == "softmax" else torch.sigmoid(y)
    flat = (0.5 - s[0]).float()
    check(pkg, y.float()[:1].expand(40, 128).contiguous(), 16, flat, scoring=scoring)


def test_equals_go_to_the_lowest(pkg):
    x = torch.zeros((3, 200))
    x[1, 70:90] = 1
    ids = check(pkg, x, 24)
    assert ids[0].tolist() == list(range(24)) and ids[1].tolist() == list(range(70, 90)) + list(range(4))
    check(pkg, x, 24, torch.zeros(200), scoring="sigmoid", groups=10, topk_groups=3, group_top=2)
    x[2, 5], x[2, 6] = 0.0, -0.0                                # the same number
    check(pkg, x - 0.0, 24)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_shut_experts_and_empty_rows(pkg, scoring):
    x = logits(6, 64, 7)
    x[0, ::2] = -float("inf")
    x[1] = -float("inf")                                        # nothing left
    x[2] = -float("inf")
    x[2, 9] = 3.0                                               # fewer than topk left
    x[3] = torch.finfo(torch.float32).min                       # masked with the lowest value
    x[4, 10:] = torch.finfo(torch.float32).min
    x[5] *= 1e30
    check(pkg, x, 8, scoring=scoring)
    bias = torch.randn(64, generator=torch.Generator().manual_seed(2))
    check(pkg, x, 8, bias, scoring=scoring)
    check(pkg, x, 8, scoring=scoring, groups=4, topk_groups=2, group_top=2)
    bias[:20], bias[20:30] = -float("inf"), 1e9                 # experts shut and forced by the bias
    check(pkg, x, 8, bias, scoring=scoring)


@pytest.mark.parametrize("with_bias", [False, True])
def test_nan_comes_last_and_ids_stay_distinct(pkg, with_bias):
    x = logits(4, 96, 8)
    x[0, 3] = float("nan")
    x[1, :90] = float("nan")
    x[2] = float("nan")
    bias = torch.randn(96, generator=torch.Generator().manual_seed(2)) * 0.1 if with_bias else None
    check(pkg, x, 10, bias, scoring="sigmoid")
    check(pkg, x, 10, bias, scoring="softmax")
    check(pkg, x, 10, bias, scoring="sigmoid", groups=8, topk_groups=3, group_top=2)
    x[3, 5] = float("inf")
    ids, _ = pkg.moe_route(x.to(DEV), 10, bias=None if bias is None else bias.to(DEV))
    for row in ids.tolist():
        assert len(set(row)) == 10 and min(row) >= 0 and max(row) < 96


@pytest.mark.parametrize("scoring,with_bias", [("sigmoid", True), ("sigmoid", False), ("softmax", False), ("softmax", True)])
@pytest.mark.parametrize("e,topk,groups,topk_groups", [(256, 8, 8, 4), (256, 12, 1, 1), (40, 32, 1, 1), (7, 7, 1, 1),
                                                       (160, 20, 8, 1), (96, 5, 3, 2), (600, 31, 1, 1)])
def test_any_logits_give_distinct_ids(pkg, e, topk, groups, topk_groups, scoring, with_bias):
    """Rows of equals, of few values, of zeros of both signs, of infinities, the largest numbers and NaN: ids in range and
    distinct; and the definition's where nothing is NaN or +inf."""
    g = torch.Generator().manual_seed(e + topk)
    big = torch.finfo(torch.float32).max
    values = torch.tensor([0.0, -0.0, 1.0, 1.0 + 2.0 ** -23, -1.0, big, -big, 1e-40, -math.inf, 90.0, -90.0, math.inf, math.nan])
    x = torch.randn((60, e), generator=g)
    for r in range(60):
        pick = values[torch.randint(0, 9 + 4 * (r % 4 == 3), (e,), generator=g)]
        x[r] = torch.where(torch.rand(e, generator=g) < (r % 10) / 9, pick, x[r])
    x[0], x[1], x[2] = 0.25, -math.inf, math.nan
    bias = torch.randn(e, generator=g) * 0.05 if with_bias else None
    kw = dict(scoring=scoring, groups=groups, topk_groups=topk_groups, group_top=1)
    ids, w = pkg.moe_route(x.to(DEV), topk, bias=None if bias is None else bias.to(DEV), **kw)
    ids = ids.cpu().numpy()
    assert ids.min() >= 0 and ids.max() < e and all(len(set(row)) == topk for row in ids)
    fine = [r for r in range(60) if not bool((torch.isnan(x[r]) | (x[r] == math.inf)).any())]
    want, weights = ref.route(x[fine].double().numpy(), topk, bias=None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(ids[fine], want)
    # within 2^-18 of itself; of e^-|x| below 2^-126 nothing is left
    assert np.all(np.abs(w.cpu().double().numpy()[fine] - weights) <= 2.0 ** -18 * weights + 2.0 ** -120)
    assert pkg.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows(pkg, dtype):
    x = logits(9, 70, 9, dtype)
    d = x.to(DEV)[:, 3:68]
    want = pkg.moe_route(d.contiguous(), 5)
    got = pkg.moe_route(d, 5)
    one = pkg.moe_route(d[2:3].expand(4, 65), 5)                # one row for every token
    for a, b, c in zip(want, got, one):
        assert torch.equal(a, b) and torch.equal(c, b[2:3].expand(4, 5))
    with pytest.raises(ValueError, match="overlap"):
        pkg.moe_route(x.to(DEV).as_strided((5, 65), (30, 1)), 5)
    assert pkg.moe_route(d[:0], 5)[0].shape == (0, 5)


# --------------------------------------------------------------- combination
def check_combine(pkg, y, w, ids=None, num_experts=0, residual=None):
    m, k, n = y.shape
    out, raw = guarded_empty((m, n), torch.bfloat16, DEV)
    dev = [None if t is None else t.to(DEV) for t in (y, w, ids, residual)]
    assert pkg.moe_combine(dev[0], dev[1], ids=dev[2], num_experts=num_experts, residual=dev[3], out=out) is out
    assert guard_intact(raw, m * n * 2)
    y64 = bf16_bits_to_f64(bits(y))
    w64 = w.double().numpy()
    live = np.ones((m, k), dtype=bool) if ids is None else ((ids >= 0) & (ids < num_experts)).numpy()
    yz = np.where(live[..., None], y64, 0)
    res = None if residual is None else bf16_bits_to_f64(bits(residual))
    want = ref.combine(yz, w64, residual=res)
    size = ref.combine(np.abs(yz), np.abs(w64), residual=None if res is None else np.abs(res))
    got = bf16_bits_to_f64(bits(out.cpu()))
    tol = k * 2.0 ** -24 * size
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -133
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)
    if residual is not None:                                    # in place
        assert torch.equal(pkg.moe_combine(dev[0], dev[1], ids=dev[2], num_experts=num_experts, residual=dev[3],
                                           out=dev[3]), out)
    assert pkg.check_device_error() == 0


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k,n", [(1, 1, 1), (1, 12, 4096), (3, 2, 7), (5, 8, 2056), (33, 3, 1001), (257, 4, 64),
                                   (2, 32, 128), (700, 12, 512)])
def test_combine_matches_float64(pkg, m, k, n, residual):
    g = torch.Generator().manual_seed(m + n)
    y = torch.randn((m, k, n), generator=g).to(torch.bfloat16)
    w = torch.randn((m, k), generator=g)
    r = (torch.randn((m, n), generator=g) * 3).to(torch.bfloat16) if residual else None
    check_combine(pkg, y, w, residual=r)
    ids = torch.randint(-2, 10, (m, k), generator=g).to(torch.int32)
    ids[0] = -1                                                 # a token without any expert
    check_combine(pkg, y, w, ids, 7, r)


def test_combine_reads_nothing_of_dropped_slots(pkg):
    g = torch.Generator().manual_seed(1)
    y = torch.randn((4, 5, 96), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.rand((4, 5), generator=g).to(DEV)
    ids = torch.tensor([[0, 1, 2, 3, 4], [0, -1, 8, 3, 4], [-1] * 5, [7, 6, 5, 4, 8]], dtype=torch.int32, device=DEV)
    clean = torch.where(((ids >= 0) & (ids < 8))[..., None], y, torch.zeros_like(y))
    want = pkg.moe_combine(clean, w)
    y[(ids < 0) | (ids >= 8)] = float("nan")
    assert torch.equal(pkg.moe_combine(y, w, ids=ids, num_experts=8), want)


def test_combine_unaligned(pkg):
    g = torch.Generator().manual_seed(2)
    raw = torch.randn(3 * 4 * 64 + 1, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.rand((3, 4), generator=g).to(DEV)
    y = raw[1:].view(3, 4, 64)
    assert torch.equal(pkg.moe_combine(y, w), pkg.moe_combine(y.clone(), w))


# ------------------------------------------------------------------ together
def test_route_gemv_combine_is_the_layer(pkg):
    """The ids and weights as moe_gemv and moe_combine take them, in a graph."""
    from fp8_block_scaled_02_gb300 import inputs
    e, n, k, m, topk = 16, 256, 128, 9, 4
    pairs = [pkg.quantize(inputs.gaussian_bf16((n, k), 0.05, 10 + i).to(DEV)) for i in range(e)]
    codes, scales = (torch.stack([p[j] for p in pairs]) for j in (0, 1))
    x = inputs.activations(m, k, 3, device=DEV)
    logits_ = logits(m, e, 4).to(DEV)
    res = inputs.activations(m, n, 5, device=DEV)

    def layer():
        ids, w = pkg.moe_route(logits_, topk)
        y = pkg.moe_gemv(x, ids, codes, scales)
        return ids, w, y, pkg.moe_combine(y, w, ids=ids, num_experts=e, residual=res)
    eager = layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, got):
        assert torch.equal(a, b)
    ids, w, y, out = got
    want = ref.combine(y.double().cpu().numpy(), w.double().cpu().numpy(), residual=res.double().cpu().numpy())
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + 0.01) + 1e-5)
    assert pkg.check_device_error() == 0
