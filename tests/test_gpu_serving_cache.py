"""What the serving step (examples/serving_step.py) leaves in the cache:
decoded token by token and given as one prompt, the same tokens have the same
first-layer keys and values.

The two runs quantize x and x', the same projection by GEMV kernels of
different row counts: bf16 of fp32 sums in another order, |x - x'| <= 2^-7 of
the group's amax (two half steps, 2^-9 each, and as much again for the sums).
With den = scale * s of a group, a stored value is within den of x: the widest
step between codes is 2, and den >= amax / 6.4 (half an e4m3 step, 2^-4) leaves
at most 0.4 beyond the last code.  So |v - v'| <= den + den' + 2^-7 6.4 max(den,
den').  Another token's keys are amax, 6 den, and more away somewhere.
"""
import pytest
import torch

from test_gpu_serving_step import PROMPTS, example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def first_layer(m, b, n):
    """Values [2, n, hkv, d] of K and V of request b's tokens, and their groups' dens [2, n, hkv, d / 16]."""
    import fp8_block_scaled_02_gb300 as fp8bs
    pos = torch.arange(n, device="cuda")
    slots = m.table[b].long()[pos // m.page] * m.page + pos % m.page
    values = torch.stack(fp8bs.kv4_gather(*m.caches[0], slots.to(torch.int32), m.scale, m.scale)).float()
    dens = []
    for c in m.caches[0]:
        tile = c[slots // m.page, :, slots % m.page // 16]                            # [n, hkv, 9 d]
        at = 8 * m.d + (slots % 16)[:, None] * (m.d // 16) + torch.arange(m.d // 16, device="cuda")
        sc = tile.gather(2, at[:, None].expand(-1, m.hkv, -1)).view(torch.float8_e4m3fn).float()
        dens.append(sc * m.scale)
    return slots, values, torch.stack(dens)


def test_decoding_writes_what_the_prompt_does(example):  # noqa: F811
    m = example.Decoder()
    first = m.prompt(PROMPTS)
    steps = [t for t, _, _ in m.decode(first, 20)]
    full = [p + [int(first[b])] + [int(t[b]) for t in steps[:-1]] for b, p in enumerate(PROMPTS)]
    again = example.Decoder()
    again.prompt(full)
    used = []
    for b, p in enumerate(full):
        slots, v, den = first_layer(m, b, len(p))
        _, v2, den2 = first_layer(again, b, len(p))
        used.append(slots)
        bound = (den + den2 + 2.0 ** -7 * 6.4 * torch.maximum(den, den2)).repeat_interleave(16, -1)
        # gathered values are bf16: half a step, 2^-9, of each
        assert bool(((v - v2).abs() <= bound + 2.0 ** -9 * (v.abs() + v2.abs())).all())
        assert float(v.abs().amax()) > 1 and bool((den > 0).all())
        other = full[(b + 1) % len(full)]                        # and not what another request holds
        _, v3, _ = first_layer(again, (b + 1) % len(full), len(other))
        n = min(len(p), len(other))
        assert not bool(((v[:, :n] - v3[:, :n]).abs() <= bound[:, :n]).all())
    used = torch.cat(used)
    assert used.unique().numel() == used.numel()                  # no slot twice
