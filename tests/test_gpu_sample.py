"""GPU tests of fp8bs_sample_tokens against float64: the same tokens, and log
probabilities within their roundings.

log p = (x - m) / T - log W: the difference and its product are held in two
fp32 and rounded once (2^-24 of |log p| + log W <= |log p| + 14), W is within
2^-22 (ex2) + 2^-24 for each of the sums that a weight passes through (at most 4 + 8
+ 5 in fp32), below 2^-19, and logf within 2^-22 of log W <= 14.
"""
import math

import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import guard_intact, guarded_empty, lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def settings(m, kind, seed):
    rng = np.random.default_rng(seed)
    t = rng.uniform(0.3, 2.0, m)
    k = rng.choice([0, 1, 2, 5, 40, 200, 1000], m)
    p = rng.choice([1.0, 0.1, 0.5, 0.8, 0.9, 0.95, 0.99], m)
    mp = rng.choice([0.0, 0.0, 0.02, 0.1, 0.5], m)
    if kind == "temperature":
        return dict(temperature=t)
    if kind == "top_k":
        return dict(temperature=t, top_k=k)
    if kind == "top_p":
        return dict(temperature=t, top_p=p)
    if kind == "min_p":
        return dict(temperature=t, min_p=mp)
    if kind == "none":
        return {}
    t = np.where(rng.random(m) < 0.1, 0.0, t)
    return dict(temperature=t, top_k=k, top_p=p, min_p=mp)


def check(pkg, x, u, err=0, device_rows=None, **kw):
    """x: CPU tensor [M, V], a view with padded rows will do."""
    base = x._base if x._base is not None else x
    xd = base.to(DEV).as_strided(x.shape, x.stride(), x.storage_offset())
    m = len(x)
    tok, raw_t = guarded_empty((m,), torch.int32, DEV)
    lp, raw_l = guarded_empty((m,), torch.float32, DEV)
    dev = {n: torch.tensor(np.asarray(v), dtype=torch.int32 if n == "top_k" else torch.float32, device=DEV)
           for n, v in kw.items()}
    u = torch.as_tensor(u, dtype=torch.float32)
    got = pkg.sample_tokens(xd, u.to(DEV), tokens=tok, logprobs=lp, **dev)
    assert got.tokens is tok and guard_intact(raw_t, m * 4) and guard_intact(raw_l, m * 4)
    x64, u64 = x.double().numpy(), u.double().numpy()
    held = {n: v.double().cpu().numpy() for n, v in dev.items()}
    tokens, logprobs = tok.cpu().numpy(), lp.cpu().double().numpy()
    for r in range(m):
        one = {n: (int(v[r]) if n == "top_k" else float(v[r])) for n, v in held.items()}
        want, want_lp, near = ref.sample(x64[r], u64[r, 0], u64[r, 1], **one)
        assert tokens[r] == want, (r, tokens[r], want, near, one)
        assert abs(logprobs[r] - want_lp) <= 2.0 ** -19 + 2.0 ** -22 * (abs(want_lp) + 28), (r, logprobs[r], want_lp, one)
    assert pkg.check_device_error() == err
    return tokens, logprobs


def logits(m, v, seed, dtype, pad=0, offset=0, scale=2.0, tall=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, v + pad + offset), generator=g) * scale
    if tall:
        at = torch.randint(0, v, (m, 8), generator=g) + offset
        x.scatter_add_(1, at, torch.rand(at.shape, generator=g) * 10)
    return x.to(dtype)[:, offset:offset + v]


def uniform(m, seed):
    return torch.rand((m, 2), generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["none", "temperature", "top_k", "top_p", "min_p", "mixed"])
@pytest.mark.parametrize("m,v", [(1, 1), (2, 2), (7, 31), (9, 1023), (9, 1024), (9, 1025), (40, 5000), (16, 32003),
                                 (3, 152064), (170, 9001), (400, 2049)])
def test_matches_float64(pkg, m, v, kind, dtype):
    check(pkg, logits(m, v, m + v, dtype), uniform(m, v), **settings(m, kind, m))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (5, 3), (0, 1), (24, 7), (0, 2), (3, 4)])
def test_padded_and_unaligned_rows(pkg, pad, offset, dtype):
    x = logits(6, 3001, pad, dtype, pad, offset)
    x._base[:, :offset] = 1e4                                     # nothing of the padding may be read
    x._base[:, offset + 3001:] = 1e4
    check(pkg, x, uniform(6, 1), **settings(6, "mixed", 3))
    check(pkg, x, uniform(6, 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temperature", [0.05, 5.0, 100.0, 1e-6, 1e6])
def test_far_temperatures(pkg, temperature, dtype):
    """Nearly greedy and nearly uniform; the nucleus of a flat row is most of the vocabulary."""
    m, v = 12, 20011
    x = logits(m, v, 5, dtype, scale=1.5)
    t = np.full(m, temperature)
    check(pkg, x, uniform(m, 3), temperature=t)
    check(pkg, x, uniform(m, 4), temperature=t, top_p=np.linspace(0.05, 0.99, m))
    check(pkg, x, uniform(m, 5), temperature=t, top_k=np.array([1, 2, 3, 100, 1000, 1024, 1025, 5000, 19999, 20010, 20011,
                                                                20012]), top_p=np.linspace(0.3, 1.0, m))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [8, 320])
def test_ends_of_the_temperatures(pkg, m, dtype):
    """The smallest is greedy among equals, the largest uniform."""
    v = 3001
    x = logits(m, v, 37, dtype)
    x[:, 2990] = x.max(1).values                                # two largest ones
    for temperature in (float(np.float32(1.0001e-30)), float(np.float32(0.9999e30))):
        t = np.full(m, temperature)
        check(pkg, x, uniform(m, 38), temperature=t)
        check(pkg, x, uniform(m, 39), temperature=t, top_p=np.linspace(0.05, 0.99, m))
        check(pkg, x, uniform(m, 40), temperature=t, top_k=np.arange(m) + 1, min_p=np.full(m, 0.5))
        check(pkg, x, uniform(m, 41), temperature=t, top_k=np.full(m, 1500), top_p=np.full(m, 0.6))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale,temperature", [(1e31, 0.9e30), (5e37, 0.9e30), (5e37, 1.0), (1e-35, 1e-30), (1e-38, 1.0)])
def test_huge_and_tiny_logits(pkg, scale, temperature, dtype):
    """Logits near the type's largest, and subnormal ones."""
    m, v = 12, 5003
    x = (logits(m, v, 42, torch.float32, tall=False).clamp(-6, 6).double() * scale).to(dtype)
    t = np.full(m, np.float64(np.float32(temperature)))
    check(pkg, x, uniform(m, 43), temperature=t)
    check(pkg, x, uniform(m, 44), temperature=t, top_p=np.linspace(0.05, 0.99, m))
    check(pkg, x, uniform(m, 45), temperature=t, top_k=np.arange(m) * 9 + 1, min_p=np.full(m, 0.01))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [8, 320])
def test_equals(pkg, m, dtype):
    """Rows of few values: cuts through equals keep the lowest of them."""
    v = 10007
    g = torch.Generator().manual_seed(m)
    x = torch.randint(0, 3, (m, v), generator=g).to(dtype)
    x[1] = 0.5
    x[2] = -0.0
    x[2, ::2] = 0.0
    x[3] = torch.finfo(dtype).min
    x[4, 5000:] = -math.inf
    x[5] = torch.finfo(dtype).min
    x[5, 77] = 1.0
    u = uniform(m, 6)
    for k in (1, 2, 700, 3500, 7001, v - 1):
        check(pkg, x, u, top_k=np.full(m, k))
    for p in (0.0, 0.25, 0.5, 0.75, 0.9):
        check(pkg, x, u, top_p=np.full(m, p))
        check(pkg, x, u, top_p=np.full(m, p), top_k=np.full(m, 4100), temperature=np.full(m, 0.7))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_rows(pkg, dtype):
    """Constrained decoding: most of the vocabulary at -inf or at the type's lowest value."""
    m, v = 30, 12001
    x = logits(m, v, 8, dtype)
    g = torch.Generator().manual_seed(9)
    shut = torch.rand((m, v), generator=g) > 0.01
    for value in (-math.inf, torch.finfo(dtype).min):
        y = x.masked_fill(shut, value)
        y[0] = value
        y[0, 11999] = 3.0                                         # one token left
        check(pkg, y, uniform(m, 10), **settings(m, "mixed", 11))
        check(pkg, y, uniform(m, 12), **settings(m, "top_p", 13))
        check(pkg, y, uniform(m, 14), **settings(m, "temperature", 15))


@pytest.mark.parametrize("m", [6, 310])
def test_rows_without_a_token(pkg, m):
    x = logits(m, 3001, 16, torch.float32)
    x[1] = -math.inf
    tokens, _ = check(pkg, x, uniform(m, 17), **settings(m, "top_p", 18))
    assert tokens[1] == -1
    for bad in (math.nan, math.inf):
        y = x.clone()
        y[3, 2999] = bad
        tokens, lp = check(pkg, y, uniform(m, 19), err=16, **settings(m, "mixed", 20))
        assert tokens[3] == -1 and lp[3] == 0
    for name, bad in (("temperature", -1.0), ("temperature", math.nan), ("temperature", math.inf), ("temperature", 1e-40),
                      ("top_p", math.nan), ("min_p", math.nan)):
        s = settings(m, "mixed", 21)
        s["temperature"] = np.where(s["temperature"] == 0, 1.0, s["temperature"])
        s[name] = s[name].copy()
        s[name][4] = bad
        if bad == 1e-40:
            got = pkg.sample_tokens(x.to(DEV), uniform(m, 1).to(DEV), torch.tensor(s["temperature"], device=DEV).float())
            assert int(got.tokens[4]) == -1 and pkg.check_device_error() == 16
            continue
        tokens, _ = check(pkg, x, uniform(m, 22), err=16, **s)
        assert tokens[4] == -1


def test_ends_of_the_settings(pkg):
    m, v = 16, 4001
    x = logits(m, v, 23, torch.bfloat16)
    u = uniform(m, 24)
    best = x.float().argmax(1).numpy()
    for kw in (dict(temperature=np.zeros(m)), dict(top_k=np.ones(m)), dict(top_p=np.zeros(m)), dict(top_p=np.full(m, -1.0)),
               dict(min_p=np.ones(m)), dict(min_p=np.full(m, 7.0))):
        tokens, _ = check(pkg, x, u, **kw)
        assert np.array_equal(x[np.arange(m), tokens].float().numpy(), x[np.arange(m), best].float().numpy())
    free = check(pkg, x, u)
    for kw in (dict(top_k=np.zeros(m)), dict(top_k=np.full(m, -5)), dict(top_k=np.full(m, v)), dict(top_p=np.ones(m)),
               dict(top_p=np.full(m, 2.0)), dict(min_p=np.zeros(m)), dict(min_p=np.full(m, -1.0)),
               dict(temperature=np.ones(m))):
        got = check(pkg, x, u, **kw)
        assert np.array_equal(got[0], free[0]) and np.array_equal(got[1], free[1])


def test_ends_of_the_random_numbers(pkg):
    m, v = 8, 5000
    x = logits(m, v, 25, torch.float32, scale=0.5, tall=False)
    last = 1 - 2.0 ** -24
    u = np.array([[0, 0], [0, last], [last, 0], [last, last], [0.5, 0], [0.5, last], [0, 0.5], [last, 0.5]])
    tokens, _ = check(pkg, x, u)
    assert tokens[0] == 0 and tokens[3] == v - 1
    check(pkg, x, u, top_k=np.full(m, 50))
    out = torch.tensor([[1.0, 1.0], [2.0, 9.0], [-1.0, -3.0], [math.nan, math.nan]], device=DEV)
    got = pkg.sample_tokens(x[:4].to(DEV), out).tokens.tolist()
    assert got == [v - 1, v - 1, 0, 0] and pkg.check_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_row_for_many_draws_and_their_shares(pkg, dtype):
    """A row expanded: every draw that of the row on its own; and the tokens come as often as they should (five standard
    deviations of each count)."""
    v, m = 3000, 20000
    x = logits(1, v, 26, dtype)
    u = uniform(m, 27).to(DEV)
    one = torch.ones(m, device=DEV)
    got = pkg.sample_tokens(x.to(DEV).expand(m, v), u, one, top_k=torch.full((m,), 20, dtype=torch.int32, device=DEV))
    kept, w = ref.kept_tokens(x[0].double().numpy(), top_k=20)
    share = w[kept] / w[kept].sum()
    n = np.bincount(got.tokens.cpu().numpy(), minlength=v)
    assert n.sum() == n[kept].sum() == m
    assert np.all(np.abs(n[kept] - m * share) <= 5 * np.sqrt(m * share * (1 - share)) + 1)
    for r in (0, 777, m - 1):
        want, lp, _ = ref.sample(x[0].double().numpy(), float(u[r, 0]), float(u[r, 1]), top_k=20)
        assert int(got.tokens[r]) == want


def test_largest_vocabulary(pkg):
    v = 1 << 20
    for dtype, m in ((torch.bfloat16, 2), (torch.float32, 2), (torch.bfloat16, 310)):
        x = logits(2, v, 28, dtype, scale=1.0, tall=False)
        d = x.to(DEV)
        u = uniform(m, 29)
        p = torch.full((m,), 0.9, device=DEV)
        full = d if m == 2 else d[:1].expand(m, v)
        got = pkg.sample_tokens(full, u.to(DEV), top_p=p)
        free = pkg.sample_tokens(full, u.to(DEV))
        for r in (0, 1):
            row = x[r if m == 2 else 0].double().numpy()
            assert int(got.tokens[r]) == ref.sample(row, float(u[r, 0]), float(u[r, 1]), top_p=float(p[r]))[0]
            assert int(free.tokens[r]) == ref.sample(row, float(u[r, 0]), float(u[r, 1]))[0]
    with pytest.raises(pkg.Fp8bsError, match="SHAPE"):
        pkg.sample_tokens(torch.zeros((1, v + 1), dtype=torch.bfloat16, device=DEV), uniform(1, 1).to(DEV))
    assert pkg.check_device_error() == 0


def test_results_do_not_depend_on_the_batch_or_the_run(pkg):
    """The same row alone (a cluster) and among many (one CTA); twice the same call."""
    m, v = 400, 30011
    x = logits(m, v, 30, torch.bfloat16).to(DEV)
    u = uniform(m, 31).to(DEV)
    s = {n: torch.tensor(np.asarray(z), dtype=torch.int32 if n == "top_k" else torch.float32, device=DEV)
         for n, z in settings(m, "mixed", 32).items()}
    a, b = pkg.sample_tokens(x, u, **s), pkg.sample_tokens(x, u, **s)
    assert torch.equal(a.tokens, b.tokens) and torch.equal(a.logprobs, b.logprobs)
    for r in range(0, m, 23):
        c = pkg.sample_tokens(x[r:r + 1], u[r:r + 1], **{n: z[r:r + 1] for n, z in s.items()})
        assert int(c.tokens[0]) == int(a.tokens[r])


def test_graph_streams_and_empty(pkg):
    m, v = 20, 32000
    x = logits(m, v, 33, torch.bfloat16).to(DEV)
    u = uniform(m, 34).to(DEV)
    s = {n: torch.tensor(np.asarray(z), dtype=torch.int32 if n == "top_k" else torch.float32, device=DEV)
         for n, z in settings(m, "mixed", 35).items()}
    want = pkg.sample_tokens(x, u, **s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkg.sample_tokens(x, u, **s)
    graph.replay()
    assert torch.equal(got.tokens, want.tokens) and torch.equal(got.logprobs, want.logprobs)
    u.copy_(uniform(m, 36))
    graph.replay()
    again = pkg.sample_tokens(x, u, **s)
    assert torch.equal(got.tokens, again.tokens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = pkg.sample_tokens(x, u, stream=side, **s)
    side.synchronize()
    assert torch.equal(other.tokens, again.tokens)
    none = pkg.sample_tokens(x[:0], u[:0])
    assert none.tokens.shape == (0,) and pkg.check_device_error() == 0
