"""GPU tests of fp8bs_sample_tokens with fp32 logits whose steps are as large as
the temperature's window: a token one step below the largest weighs 2^-2.9 to 2^-115
of it, and the window ends within a step or two.

top_p lies halfway into the mass of a token of at least 2^-10 of all, random numbers
2^-16 from a border: far from what masses are off by (below 2^-18).
"""
import math

import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROWS = 12


def rows_near(largest, v, rng):
    """Rows whose largest is `largest`, with a few tokens 0 to 3 steps below it; the rest of a row far below."""
    m = np.float32(largest)
    x = (m - np.abs(m) * rng.uniform(0.1, 1.0, (ROWS, v))).astype(np.float32)
    steps = [m]
    for _ in range(3):
        steps.append(np.nextafter(steps[-1], np.float32(-np.inf)))
    for r in range(ROWS):
        at = rng.permutation(v)[:1 + 3 * r]
        x[r, at] = [steps[i] for i in rng.integers(0, 4, len(at))]
        x[r, at[0]] = m
    return x


@pytest.mark.parametrize("v", [900, 20011])
@pytest.mark.parametrize("largest", [7.3, 12.0, 20.0, -1.5, 1000.25, 3e-5, 2e38])
def test_temperatures_of_a_step(largest, v):
    pkg = lib_or_skip()
    rng = np.random.default_rng(v + int(abs(math.log2(abs(largest)))))
    ulp = float(np.nextafter(np.float32(abs(largest)), np.float32(np.inf)) - np.float32(abs(largest)))
    for share in (80, 63, 44, 30, 20, 8, 2):
        t = np.full(ROWS, ulp / share).astype(np.float32)
        if t[0] > 1e30:
            continue
        x = rows_near(largest, v, rng)
        top_k = rng.integers(1, 40, ROWS).astype(np.int32)
        settings, want = dict(top_p=[], both=[]), dict(top_p=[], top_k=[], both=[])
        u = rng.random((ROWS, 2)).astype(np.float32)
        for r in range(ROWS):
            x64 = x[r].astype(np.float64)
            for kind, k in (("top_p", 0), ("both", int(top_k[r]))):
                kept, w = ref.kept_tokens(x64, float(t[r]), k)
                mass = np.cumsum(w[kept])
                n = int(rng.integers(0, (w[kept] >= 2.0 ** -10 * mass[-1]).sum()))
                settings[kind].append(np.float32((mass[n] - 0.5 * w[kept][n]) / mass[-1]))
            while True:
                got = [ref.sample(x64, float(u[r, 0]), float(u[r, 1]), float(t[r]), **kw)
                       for kw in (dict(top_p=float(settings["top_p"][r])), dict(top_k=int(top_k[r])),
                                  dict(top_p=float(settings["both"][r]), top_k=int(top_k[r])))]
                if min(g[2] for g in got) >= 2.0 ** -16:
                    break
                u[r] = rng.random(2)
            for kind, g in zip(("top_p", "top_k", "both"), got):
                want[kind].append(g[:2])
        dev = {n: torch.from_numpy(np.asarray(a)).to(DEV) for n, a in dict(x=x, u=u, t=t, k=top_k, **settings).items()}
        for kind, kw in (("top_p", dict(top_p=dev["top_p"])), ("top_k", dict(top_k=dev["k"])),
                         ("both", dict(top_p=dev["both"], top_k=dev["k"]))):
            got = pkg.sample_tokens(dev["x"], dev["u"], dev["t"], **kw)
            assert got.tokens.tolist() == [w[0] for w in want[kind]], (share, kind)
            lp = np.array([w[1] for w in want[kind]])
            # two fp32 rounded once and logf, 2^-22 of |log p| + log W <= 14 each way; W within 2^-19
            assert np.all(np.abs(got.logprobs.cpu().double().numpy() - lp) <= 2.0 ** -19 + 2.0 ** -22 * (np.abs(lp) + 28))
    assert pkg.check_device_error() == 0
