"""Pins of the plain references the serving-step operators are tested against
(CPU only): the 4-bit format against torch's casts, closed forms and
brute force; attention against torch's softmax; the plan's invariants; the
log probabilities against torch; and that attention's bound rejects planted
mistakes."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from oracle import tolerance


def bf16_bits(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_e4m3_values_are_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.E4M3, t)


def test_nearest_is_torchs_cast_and_brute_force():
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.uniform(0, 448, 5000), 10.0 ** rng.uniform(-5, 2.6, 5000), ref.E4M3,
                        (ref.E4M3[1:] + ref.E4M3[:-1]) / 2]).astype(np.float32)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest(v, ref.E4M3), t)
    v = np.concatenate([rng.uniform(0, 8, 4000), ref.E2M1, (ref.E2M1[1:] + ref.E2M1[:-1]) / 2])
    d = np.abs(v[:, None] - ref.E2M1[None])
    for x, got, row in zip(v, ref.nearest(v, ref.E2M1), d):
        best = np.flatnonzero(row == row.min())
        assert got in best and (len(best) == 1 or got % 2 == 0), x


def test_bf16_rounding_is_torchs():
    v = np.random.default_rng(2).standard_normal(4000).astype(np.float32)
    assert np.array_equal(ref.f32_to_bf16_bits(v), bf16_bits(v))


def test_grid_values_are_kept_exactly():
    """Values code * scale * s with amax at 6 scale come back unchanged."""
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (40, 2, 64))
    codes[..., ::16] = 7                                     # every group reaches 6
    sc = rng.integers(8, 120, (40, 2, 4))
    s = np.float32(0.25)
    x = ref.E2M1_SIGNED[codes] * np.repeat(ref.E4M3[sc], 16, axis=-1) * s
    got, gsc = ref.encode(bf16_bits(x), s)
    assert np.array_equal(gsc, sc)
    assert np.array_equal(ref.E2M1_SIGNED[got], ref.E2M1_SIGNED[codes])


def test_encode_error_is_half_a_step():
    rng = np.random.default_rng(4)
    bits = bf16_bits(rng.standard_normal((200, 1, 128)))
    x = ref.bf16_to_f64(bits)
    s = np.float32(5.5 / 2688)
    codes, sc = ref.encode(bits, s)
    step = np.repeat(ref.E4M3[sc], 16, axis=-1) * float(s)
    err = np.abs(ref.E2M1_SIGNED[codes] * step - x)
    # half the widest step (4 .. 6) of the scale, and what a scale rounded down by half an e4m3 step cuts off
    assert np.all(err <= step * (1 + 6 * 2.0 ** -4) * (1 + 1e-6))
    assert 0.05 < np.linalg.norm(err) / np.linalg.norm(x) < 0.12


def test_append_then_decode_places_tokens():
    rng = np.random.default_rng(5)
    bits = bf16_bits(rng.standard_normal((9, 2, 64)))
    slots = np.array([31, 0, 15, 16, -1, 47, 33, 48, 7])     # -1 and 48 store nothing
    cache = rng.integers(0, 100, (3, 2, 1, 9 * 64), dtype=np.uint8)
    out = ref.append(bits, slots, 0.01, cache)
    codes, sc = ref.encode(bits, 0.01)
    x = ref.decode(out)
    for t, s in enumerate(slots):
        if 0 <= s < 48:
            want = ref.E2M1_SIGNED[codes[t]] * np.repeat(ref.E4M3[sc[t]], 16, axis=-1)
            assert np.array_equal(x[s], want)
    untouched = sorted(set(range(48)) - set(slots.tolist()))
    assert np.array_equal(x[untouched], ref.decode(cache)[untouched])


def case(lens, hq, hkv, d, seed):
    rng = np.random.default_rng(seed)
    nb = sum(-(-n // 16) for n in lens) + 1
    caches = []
    for _ in range(2):
        bits = bf16_bits(rng.standard_normal((nb * 16, hkv, d)))
        caches.append(ref.append(bits, np.arange(nb * 16), 0.002, np.zeros((nb, hkv, 1, 9 * d), dtype=np.uint8)))
    table = np.zeros((len(lens), max(-(-n // 16) for n in lens)), dtype=np.int64)
    perm, at = rng.permutation(nb), 0
    for b, n in enumerate(lens):
        table[b, :-(-n // 16)] = perm[at:at - (-n // 16)]
        at -= -n // 16
    return rng, caches, table


@pytest.mark.parametrize("window", [0, 3, 100])
def test_attention_is_torchs(window):
    lens, qls = [20, 5, 33], [1, 3, 2]
    rng, (kc, vc), table = case(lens, 6, 2, 64, 6)
    cu = np.concatenate([[0], np.cumsum(qls)])
    q = bf16_bits(rng.standard_normal((6, 6, 64)))
    o, lse, _ = ref.attention(q, cu, kc, vc, 0.002, 0.002, table, lens, 0.125, window)
    k, v = (torch.from_numpy(ref.decode(c) * float(np.float32(0.002))) for c in (kc, vc))
    x = torch.from_numpy(ref.bf16_to_f64(q))
    for b, n in enumerate(lens):
        pos = np.arange(n)
        idx = table[b, pos // 16] * 16 + pos % 16
        kk, vv = (t[idx].repeat_interleave(3, dim=1).transpose(0, 1) for t in (k, v))
        s = (x[cu[b]:cu[b + 1]].transpose(0, 1) @ kk.transpose(1, 2)) * 0.125
        p = torch.arange(n - qls[b], n)[:, None]
        dead = torch.arange(n)[None] > p
        if window:
            dead |= torch.arange(n)[None] <= p - window
        s = s.masked_fill(dead, -torch.inf)
        assert np.allclose(o[cu[b]:cu[b + 1]], (torch.softmax(s, -1) @ vv).transpose(0, 1).numpy(), atol=1e-12)
        assert np.allclose(lse[cu[b]:cu[b + 1]], torch.logsumexp(s, -1).T.numpy(), atol=1e-12)


def test_attention_bound_rejects_mistakes():
    lens = [40]
    rng, (kc, vc), table = case(lens, 8, 2, 128, 7)
    q = bf16_bits(rng.standard_normal((1, 8, 128)) * 1.5)
    s, sm = np.float32(0.002), 128 ** -0.5
    o, lse, mag = ref.attention(q, [0, 1], kc, vc, s, s, table, lens, sm)
    vmax = np.abs(ref.decode(vc)).max() * float(s)

    def passes(o2):
        got = ref.bf16_to_f64(ref.f32_to_bf16_bits(o2.astype(np.float32)))
        return np.all(np.abs(got - o) <= tolerance.kv_attention_bound(got, o, vmax))

    assert passes(o)
    nib = lambda c: np.concatenate([(c[..., :1024] >> 4) | (c[..., :1024] << 4), c[..., 1024:]], axis=-1).astype(np.uint8)
    shift = lambda c: np.concatenate([c[..., :1024], np.roll(c[..., 1024:], 1, axis=-1)], axis=-1)
    for bad in (ref.attention(q, [0, 1], kc, vc, s, s, table, [39], sm)[0],                # last token dropped
                ref.attention(q, [0, 1], kc, vc, s, s, table, lens, sm, 39)[0],            # first token dropped
                ref.attention(q, [0, 1], kc, vc, s, s, table[:, ::-1], lens, sm)[0],       # blocks in another order
                ref.attention(q, [0, 1], kc, nib(vc), s, s, table, lens, sm)[0],           # nibbles swapped
                ref.attention(q, [0, 1], shift(kc), vc, s, s, table, lens, sm)[0],         # next group's scale
                ref.attention(q, [0, 1], kc, shift(vc), s, s, table, lens, sm)[0],
                ref.attention(q, [0, 1], kc, vc, s * s, s, table, lens, sm)[0],
                o[:, ::-1]):                                                               # heads in another order
        assert not passes(bad)
    lse2 = ref.attention(q, [0, 1], kc, vc, s, s, table, [39], sm)[1]
    assert np.any(np.abs(lse2 - lse) > ref.lse_bound(lse, mag, 128))


def test_empty_rows():
    rng, (kc, vc), table = case([2], 2, 1, 64, 8)
    q = bf16_bits(rng.standard_normal((4, 2, 64)))
    o, lse, _ = ref.attention(q, [0, 4], kc, vc, 1.0, 1.0, table, [2], 0.1)
    assert np.all(o[:2] == 0) and np.all(lse[:2] == -np.inf) and np.all(np.isfinite(lse[2:]))


def test_plan_invariants():
    rng = np.random.default_rng(9)
    for page in (1, 16, 50):
        ctx, new = rng.integers(0, 120, 30).tolist(), rng.integers(0, 60, 30).tolist()
        held = [-(-c // page) for c in ctx]
        perm = rng.permutation(8000)
        table = np.full((30, 200), -1)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = perm[at:at + h]
            at += h
        p, err = ref.plan(ctx, new, table, perm[at:].tolist(), 0, page, 8000, sum(new))
        assert err == 0
        assert len(set(p["slots"].tolist())) == sum(new)              # no two tokens share a slot
        ends = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        used = np.concatenate([p["table"][b, :e] for b, e in enumerate(ends)])
        assert len(set(used.tolist())) == len(used) and used.min() >= 0
        assert int(p["free_head"][0]) == sum(ends) - sum(held)
        for j, (r, q, s) in enumerate(zip(p["requests"], p["positions"], p["slots"])):
            assert p["cu_new"][r] <= j < p["cu_new"][r + 1] and q == ctx[r] + j - p["cu_new"][r]
            assert s == p["table"][r, q // page] * page + q % page


def test_plan_refusals():
    table = [[5, -1], [6, -1], [-1, -1]]
    p, err = ref.plan([16, 8, 0], [1, 1, 4], table, [1], 0, 16, 8, 6)
    assert err == 32 and p["seq_lens"].tolist() == [17, 9, 0] and p["slots"].tolist() == [16, 104, -1, -1, -1, -1]
    assert p["requests"].tolist() == [0, 1, 2, 2, 2, 2] and p["free_head"].tolist() == [1]
    p, err = ref.plan([16, 32, -1], [1, 1, 4], table, [1, 2], 0, 16, 8, 6)
    assert err == 16 and p["seq_lens"].tolist() == [17, 32, 0]


def test_logprobs_are_torchs():
    x = torch.randn((5, 300), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    x[2, 10:] = -torch.inf
    w, _ = ref.logprobs(x.numpy(), [0, 1, 2, 299, -1], 12)
    lsm = torch.log_softmax(x, 1)
    assert np.allclose(w["logprobs"], [lsm[0, 0], lsm[1, 1], lsm[2, 2], lsm[3, 299], 0])
    p = lsm.exp()
    assert np.allclose(w["entropy"], -torch.where(p > 0, p * lsm, 0.0).sum(1).numpy())
    v, i = torch.sort(lsm, dim=1, descending=True, stable=True)
    assert np.array_equal(w["top_ids"], i[:, :12].numpy()) and np.allclose(w["top_logprobs"], v[:, :12].numpy())
    w, _ = ref.logprobs(np.full((1, 50), -3.4e38), [7], 3)
    assert np.allclose(w["logprobs"], -np.log(50)) and w["top_ids"].tolist() == [[0, 1, 2]]
