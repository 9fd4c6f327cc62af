"""GPU tests of fp8bs_token_logprobs against float64.

Tolerances: the sums l = sum e^(x - m) and t = sum (x - m) e^(x - m) run in
fp32, at most V / 256 + 64 terms one after the other (half a step, 2^-24,
each) and an exp2 within 2^-22: relative error r = (V / 256 + 64) 2^-24 +
2^-21.  log l moves by r; x - m and the last difference round once each
(2^-24 of their size); the entropy log l - t / l moves by r (1 + 2 |t / l|)
and its own rounding.  Ids have to be equal.
"""
import numpy as np
import pytest
import torch

import serving_reference as ref
from gpu_helpers import guard_intact, guarded_empty, lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def check(pkg, x, targets, top, err=0, **kw):
    """x: CPU tensor [M, V] (a view with padded rows will do)."""
    base = x._base if x._base is not None else x
    d = base.to(DEV)
    xd = d.as_strided(x.shape, x.stride(), x.storage_offset())
    r = pkg.token_logprobs(xd, torch.tensor(targets, dtype=torch.int32, device=DEV), top, **kw)
    x64 = x.double().numpy()
    with np.errstate(invalid="ignore"):
        want, dist = ref.logprobs(x64, targets, top)
    got = {n: v.cpu().numpy() for n, v in r._asdict().items()}
    assert np.array_equal(got["top_ids"], want["top_ids"])
    rel = (x.shape[1] / 256 + 64) * 2.0 ** -24 + 2.0 ** -21

    def close(g, w, tol):
        fin = np.isfinite(w)
        assert np.array_equal(g[~fin], w[~fin])
        e = np.abs(g[fin] - w[fin])
        assert np.all(e <= np.broadcast_to(tol, w.shape)[fin]), (e.max(), tol)

    for n in ("logprobs", "top_logprobs"):
        w = np.where(np.isfinite(want[n]), want[n], 0)
        close(got[n], want[n], rel + 2.0 ** -22 * (np.abs(w) + 12))
    close(got["entropy"], want["entropy"], rel * (1 + 2 * dist) + 2.0 ** -22 * (12 + dist))
    assert pkg.check_device_error() == err
    return r


def logits(m, v, seed, dtype, pad=0, offset=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((m, v + pad + offset), generator=g) * scale).to(dtype)
    return x[:, offset:offset + v]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v,top", [(1, 1, 1), (1, 2, 2), (3, 31, 5), (2, 33, 32), (1, 255, 0), (4, 1000, 20),
                                     (7, 4097, 32), (2, 32003, 20), (1, 152064, 20), (33, 8192, 1), (400, 2049, 3)])
def test_matches_float64(pkg, m, v, top, dtype):
    x = logits(m, v, m + v, dtype)
    t = np.random.default_rng(v).integers(0, v, m)
    check(pkg, x, t, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (5, 3), (0, 1), (24, 7)])
def test_padded_and_unaligned_rows(pkg, pad, offset, dtype):
    x = logits(5, 3001, pad, dtype, pad, offset)
    x._base[:, :offset] = 1e4                                     # nothing of the padding may be read
    x._base[:, offset + 3001:] = 1e4
    check(pkg, x, [0, 3000, 1500, 7, 8], 20)


@pytest.mark.parametrize("dtype,v", [(torch.bfloat16, 24576 + 8), (torch.bfloat16, 25003), (torch.float32, 12289),
                                     (torch.float32, 20000)])
@pytest.mark.parametrize("pad", [0, 3])
def test_more_rows_than_a_wave_of_long_ones(pkg, dtype, v, pad):
    """More CTAs than fit at once, rows of every alignment."""
    x = logits(330, v, v, dtype, pad)
    check(pkg, x, np.random.default_rng(v).integers(0, v, 330), 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v,top", [(609, 3001, 20), (700, 1, 1), (1301, 500, 0), (650, 9001, 32)])
def test_many_rows(pkg, m, v, top, dtype):
    """More rows than CTAs at once; among them masked ones, of equals, of large values a fixed distance apart, far
    from zero."""
    x = logits(m, v, m, dtype, pad=5).clone()
    if v > 100:
        x[3::50] = torch.finfo(dtype).min
        x[3::50, 7:13] = 1.0
        x[4::50] = -np.inf
        x[5::50] = 0.25
        x[6::50, ::512] += 100
        x[7::50] -= 1e6
        x[8::50, v // 2:] = -np.inf
    check(pkg, x, np.random.default_rng(m).integers(0, v, m), top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v,top", [(160, 50003, 20), (290, 49152, 0)])
def test_rows_of_one_block_each_in_one_wave(pkg, m, v, top, dtype):
    x = logits(m, v, m, dtype, pad=3).clone()
    x[3::50] = torch.finfo(dtype).min
    x[4::50] = -np.inf
    x[5::50] = 0.25
    x[8::50, v // 2:] = -np.inf
    check(pkg, x, np.random.default_rng(m).integers(0, v, m), top)


@pytest.mark.parametrize("dtype,v", [(torch.bfloat16, 66003), (torch.float32, 33003)])
@pytest.mark.parametrize("m,top", [(613, 20), (1230, 0), (1230, 20)])
def test_many_long_rows(pkg, dtype, v, m, top):
    x = logits(m, v, v, dtype, pad=1).clone()
    x[3::50] = torch.finfo(dtype).min
    x[3::50, 7:13] = 1.0
    x[4::50] = -np.inf
    x[5::50] = 0.25
    x[8::50, v // 2:] = -np.inf
    check(pkg, x, np.random.default_rng(v).integers(0, v, m), top)


@pytest.mark.parametrize("v", [70, 5000, 152064])
@pytest.mark.parametrize("low", [-np.inf, "lowest"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_rows(pkg, v, low, dtype):
    """Rows with few tokens left, fewer than asked for, one, or none at all."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    x = logits(5, v, 3, dtype).clone()
    rng = np.random.default_rng(v)
    t = []
    for r, keep in enumerate((60, 7, 1, 0, 25)):
        idx = rng.choice(v, keep, replace=False)
        row = torch.full((v,), low, dtype=dtype)
        row[idx] = x[r, idx]
        x[r] = row
        t.append(int(idx[0]) if keep else 5)
    check(pkg, x, t, 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_values_before_ordinary_ones(pkg, dtype):
    """What a thread reads first is the type's lowest value (or far below the rest), what it reads later is not."""
    x = logits(4, 20000, 14, dtype).clone()
    x[0, :8192] = torch.finfo(dtype).min
    x[1, :8192] = -1e6
    x[2, ::2] = torch.finfo(dtype).min
    x[3, 3000:] = torch.finfo(dtype).min
    check(pkg, x, [9000, 9000, 1, 7], 20)


def test_a_masked_target(pkg):
    x = logits(2, 300, 4, torch.bfloat16).clone()
    x[0, 17] = -np.inf
    check(pkg, x, [17, 17], 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_index(pkg, dtype):
    v = 20000
    x = torch.zeros((6, v), dtype=dtype)
    x[1] = -3.5
    x[2, 5000:] = 1.0                                             # a block of equals
    x[3, ::7] = 2.0                                               # equals everywhere
    x[4] = (torch.arange(v) % 5).to(dtype)
    x[5, 19990:] = 4.0                                            # fewer equals than asked, at the end
    check(pkg, x, [0, 1, 2, 3, 4, 5], 32)


def test_one_column_holds_all_the_large_values(pkg):
    """Large values a fixed distance apart, which one thread of a CTA would see all of."""
    for step in (256, 512, 2048, 4096, 1024, 8):
        x = logits(2, 100000, 6, torch.float32, scale=1.0).clone()
        n = x[:, ::step].shape[1]
        x[:, ::step] = 100 + torch.randperm(n, generator=torch.Generator().manual_seed(step)).float() / n
        check(pkg, x, [0, step], 32)


@pytest.mark.parametrize("shift", [-3e38, -1e30, 1e5, 1e30, 3e38])
def test_far_from_zero(pkg, shift):
    x = (logits(2, 700, 8, torch.float32) + shift).float()
    check(pkg, x, [3, 699], 4)


def test_wide_range(pkg):
    x = logits(2, 3000, 9, torch.float32, scale=1e4)
    check(pkg, x, [3, 2999], 8)
    x = x.clone()
    x[0, 5], x[0, 6] = 3.4e38, -3.4e38                            # the difference passes the range of fp32
    check(pkg, x, [5, 9], 8)


def test_targets_outside_the_vocabulary(pkg):
    x = logits(4, 500, 10, torch.bfloat16)
    r = check(pkg, x, [-1, 3, -100, 499], 2)
    assert float(r.logprobs[0]) == 0 and float(r.logprobs[2]) == 0
    check(pkg, x, [500, 3, 4, 10 ** 6], 2, err=16)


def test_nan_rows_stay_in_bounds_and_alone(pkg):
    x = logits(4, 6000, 11, torch.bfloat16).to(DEV)
    clean = pkg.token_logprobs(x, torch.zeros(4, dtype=torch.int32, device=DEV), 20)
    x[1, 100:4000] = float("nan")
    x[2, 7] = float("inf")
    r = pkg.token_logprobs(x, torch.zeros(4, dtype=torch.int32, device=DEV), 20)
    assert bool(((r.top_ids >= -1) & (r.top_ids < 6000)).all())
    for row in (0, 3):
        assert torch.equal(r.top_ids[row], clean.top_ids[row]) and torch.equal(r.logprobs[row], clean.logprobs[row])
    x[1] = float("nan")
    pkg.token_logprobs(x, torch.zeros(4, dtype=torch.int32, device=DEV), 20)
    torch.cuda.synchronize()


def test_guards_streams_and_graph(pkg):
    x = logits(9, 5001, 12, torch.bfloat16).to(DEV)
    t = torch.arange(9, dtype=torch.int32, device=DEV)
    want = pkg.token_logprobs(x, t, 7)
    bufs = [guarded_empty(s, dt, DEV) for s, dt in (((9,), torch.float32), ((9,), torch.float32),
                                                   ((9, 7), torch.int32), ((9, 7), torch.float32))]
    pkg.token_logprobs(x, t, 7, *(b[0] for b in bufs))
    for (view, raw), w in zip(bufs, want):
        assert torch.equal(view, w) and guard_intact(raw, w.numel() * 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkg.token_logprobs(x, t, 7, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = pkg.token_logprobs(x, t, 7)
    x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    again = pkg.token_logprobs(x, t, 7)
    assert all(torch.equal(a, b) for a, b in zip(r, again))
