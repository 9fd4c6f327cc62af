"""GPU tests of the 4-bit paged KV cache: the append and the gather bit for
bit, attention within the FP8 cache's bound.

Attention's tolerance: the output is a convex combination of exactly decoded
values, so every error scales with max|V|: fp32 scores and softmax (relative
about 1e-6), the weights as f16 (half a step, 2^-11, each; at most 2^-11
max|V| in all), fp32 sums, then one bf16 rounding (half a step):
|o - o64| <= 2^-10 max|V| + 1/2 ulp_bf16.  lse: serving_reference.lse_bound.
"""
import numpy as np
import pytest
import torch

import serving_reference as ref
from fp8_block_scaled_02_gb300 import inputs
from gpu_helpers import bits, guard_intact, guarded_empty, lib_or_skip
from oracle import tolerance
from oracle.tolerance import bf16_bits_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
KS, VS = np.float32(5.5 / 2688), np.float32(6.25 / 2688)
COUNTERS = 1280                                                   # FP4KV_WORKSPACE_COUNTER_BYTES


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def scales():
    return torch.tensor([KS], device=DEV), torch.tensor([VS], device=DEV)


def normal(shape, seed, scale=1.0):
    return inputs.gaussian_bf16((int(np.prod(shape[:-1])), shape[-1]), scale, seed).view(*shape)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("t,hkv,d,page", [(1, 1, 64, 16), (1, 8, 128, 16), (5, 2, 128, 48), (33, 8, 64, 32),
                                          (257, 3, 128, 256), (17, 8, 128, 64)])
def test_append_is_bit_exact(pkg, t, hkv, d, page):
    nb = t // page + 3
    rng = np.random.default_rng(t + d)
    k, v = normal((t, hkv, d), 1 + t), normal((t, hkv, d), 2 + t, 3.0)
    slots = rng.choice(nb * page, size=t, replace=False).astype(np.int32)
    k0, v0 = (rng.integers(0, 256, (nb, hkv, page // 16, 9 * d), dtype=np.uint8) for _ in range(2))
    kc, vc = torch.from_numpy(k0.copy()).to(DEV), torch.from_numpy(v0.copy()).to(DEV)
    ks, vs = scales()
    pkg.kv4_append(k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), ks, vs, kc, vc)
    assert np.array_equal(kc.cpu().numpy(), ref.append(bits(k), slots, KS, k0))
    assert np.array_equal(vc.cpu().numpy(), ref.append(bits(v), slots, VS, v0))
    assert pkg.check_device_error() == 0


def hard_rows(d):
    """Groups whose rounding is decided by a hair: zeros, one element, amax at
    every e4m3 border, quotients on and beside the e2m1 midpoints, subnormals,
    the largest bf16 values."""
    rng = np.random.default_rng(4)
    rows = [np.zeros(16), -np.zeros(16), np.full(16, 2.0 ** -133), np.full(16, -3.38e38)]
    for e in range(-20, 20):
        rows.append(np.concatenate([[6.0], [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], -np.arange(8.0)]) * 2.0 ** e)
    for _ in range(600):
        x = rng.standard_normal(16) * 10.0 ** rng.uniform(-6, 4)
        rows.append(np.where(rng.random(16) < 0.3, 0, x))
    rows += [np.zeros(16)] * (-len(rows) % (d // 16))
    return torch.tensor(np.array(rows).reshape(-1, 1, d), dtype=torch.float32).to(torch.bfloat16)


@pytest.mark.parametrize("scale", [KS, np.float32(1.0), np.float32(1e-30), np.float32(1e-42), np.float32(3e35)])
def test_append_hard_groups(pkg, scale):
    d, page = 128, 16
    x = hard_rows(d)
    t = len(x)
    nb = t // page + 1
    slots = np.arange(t, dtype=np.int32)
    zero = np.zeros((nb, 1, 1, 9 * d), dtype=np.uint8)
    kc, vc = torch.from_numpy(zero.copy()).to(DEV), torch.from_numpy(zero.copy()).to(DEV)
    s = torch.tensor([scale], device=DEV)
    pkg.kv4_append(x.to(DEV), (-x).to(DEV), torch.from_numpy(slots).to(DEV), s, s, kc, vc)
    assert np.array_equal(kc.cpu().numpy(), ref.append(bits(x), slots, scale, zero))
    assert np.array_equal(vc.cpu().numpy(), ref.append(bits(-x), slots, scale, zero))


def test_append_of_projection_slices_and_skipped_slots(pkg):
    t, hq, hkv, d, page, nb = 37, 4, 2, 128, 16, 6
    qkv = normal((t, (hq + 2 * hkv) * d), 5).to(DEV)
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    slots = np.random.default_rng(6).permutation(nb * page)[:t].astype(np.int32)
    slots[3] = -1
    zero = np.zeros((nb, hkv, 1, 9 * d), dtype=np.uint8)
    kc, vc = torch.from_numpy(zero.copy()).to(DEV), torch.from_numpy(zero.copy()).to(DEV)
    ks, vs = scales()
    pkg.kv4_append(k, v, torch.from_numpy(slots).to(DEV), ks, vs, kc, vc)
    assert np.array_equal(kc.cpu().numpy(), ref.append(bits(k.contiguous()), slots, KS, zero))
    assert np.array_equal(vc.cpu().numpy(), ref.append(bits(v.contiguous()), slots, VS, zero))
    assert pkg.check_device_error() == 0                          # -1 is not an error
    slots[5], slots[7] = nb * page, -2
    pkg.kv4_append(k, v, torch.from_numpy(slots).to(DEV), ks, vs, kc.zero_(), vc)
    assert np.array_equal(kc.cpu().numpy(), ref.append(bits(k.contiguous()), slots, KS, zero))
    assert pkg.check_device_error() == 16


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("t,hkv,d,page", [(1, 1, 64, 16), (9, 8, 128, 16), (301, 2, 64, 48), (64, 8, 128, 128)])
def test_gather_is_bit_exact(pkg, t, hkv, d, page):
    nb = t // page + 3
    rng = np.random.default_rng(t)
    k0, v0 = (rng.integers(0, 256, (nb, hkv, page // 16, 9 * d), dtype=np.uint8) for _ in range(2))
    for c in (k0, v0):                                            # any code, any finite scale
        c[..., 8 * d:] = rng.integers(0, 0x7F, c[..., 8 * d:].shape)
    slots = rng.integers(0, nb * page, t).astype(np.int32)
    if t > 8:
        slots[2] = -1
    ks, vs = scales()
    outs = [guarded_empty((t, hkv, d), torch.bfloat16, DEV) for _ in range(2)]
    k, v = pkg.kv4_gather(torch.from_numpy(k0).to(DEV), torch.from_numpy(v0).to(DEV), torch.from_numpy(slots).to(DEV),
                          ks, vs, k=outs[0][0], v=outs[1][0])
    for got, c, s in ((k, k0, KS), (v, v0, VS)):
        g, w = bits(got), ref.gather_bits(c, slots, s)
        assert np.array_equal(np.where(g == 0x8000, 0, g), np.where(w == 0x8000, 0, w))
    assert all(guard_intact(raw, t * hkv * d * 2) for _, raw in outs)
    assert pkg.check_device_error() == 0


def test_gather_out_of_range_slots_give_zeros(pkg):
    kc = torch.full((2, 1, 1, 1152), 0x33, dtype=torch.uint8, device=DEV)
    ks, vs = scales()
    k, v = pkg.kv4_gather(kc, kc.clone(), torch.tensor([32, -2, 31], dtype=torch.int32, device=DEV), ks, vs)
    assert pkg.check_device_error() == 16
    assert float(k[:2].float().abs().max()) == 0 and float(v[2].float().abs().min()) > 0


# --------------------------------------------------------------- attention
def layer(lens, hkv, d, page, seed, extra=2):
    """Caches the reference wrote for normal keys and values, scattered blocks."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    nb = sum(need) + extra
    kc, vc = (rng.integers(0, 256, (nb, hkv, page // 16, 9 * d), dtype=np.uint8) for _ in range(2))
    for c in (kc, vc):                                            # what old tenants left: NaN scales among it
        c[..., 8 * d:] = rng.choice([0x7F, 0xFF, 0x20, 0x7E], c[..., 8 * d:].shape)
    perm = rng.permutation(nb)
    table = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        pos = np.arange(lens[b])
        slots = (table[b, pos // page] * page + pos % page).astype(np.int32)
        x = normal((2, max(lens[b], 1), hkv * d), seed + 7 * b + 1).view(2, -1, hkv, d)[:, :lens[b]]
        codes = [ref.append(bits(x[0]), slots, KS, kc), ref.append(bits(x[1] + 0.25), slots, VS, vc)]
        kc, vc = codes
    return kc, vc, table


def attend(pkg, q, kc, vc, table, lens, sm, max_len=None, **kw):
    ks, vs = scales()
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    ws = pkg.kv4_workspace(kc.shape[3] // 9, DEV)
    ws[COUNTERS:] = 0xA5
    if kw.get("cu_q") is not None:
        kw["cu_q"] = t(np.asarray(kw["cu_q"], dtype=np.int32))
    r = pkg.kv4_decode_attention(q.to(DEV), t(kc), t(vc), ks, vs, t(table), t(np.asarray(lens, dtype=np.int32)),
                                 max(max(lens), 1) if max_len is None else max_len, sm, ws, return_lse=True, **kw)
    assert int(ws[:COUNTERS].max()) == 0                          # as the next call needs them
    return r


def check(o, lse, q, cu, kc, vc, table, lens, sm, window=0, err=0, pkg=None):
    w, wl, mag = ref.attention(bits(q), cu, kc, vc, KS, VS, table, lens, sm, window)
    got, gl = bf16_bits_to_f64(bits(o.cpu())), lse.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        vmax = 0.0
        x = np.abs(ref.decode(vc)) * float(VS)
        for b, n in enumerate(lens):
            pos = np.arange(max(n, 0))
            blk = table[b, pos // (vc.shape[2] * 16)]
            ok = (blk >= 0) & (blk < vc.shape[0])
            if ok.any():
                vmax = max(vmax, x[(blk * vc.shape[2] * 16 + pos % (vc.shape[2] * 16))[ok]].max())
    assert np.all(np.isfinite(got))
    e = np.abs(got - w)
    bound = tolerance.kv_attention_bound(got, w, vmax)
    assert np.all(e <= bound), (e.max(), (e / bound).max())
    assert np.array_equal(np.isfinite(gl), np.isfinite(wl))
    fin = np.isfinite(wl)
    assert np.all(gl[~fin] == -np.inf)
    assert np.all(np.abs(gl[fin] - wl[fin]) <= ref.lse_bound(wl, mag, q.shape[2])[fin])
    assert pkg is None or pkg.check_device_error() == err


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [31], [33], [100], [1000], [3, 70, 0, 257]])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (16, 2, 128), (5, 1, 64), (14, 2, 128), (32, 2, 128),
                                      (40, 1, 128), (48, 2, 64)])
def test_attention_small(pkg, lens, hq, hkv, d):
    kc, vc, table = layer(lens, hkv, d, 16, len(lens) + hq)
    q = normal((len(lens), hq, d), hq)
    sm = d ** -0.5
    o, lse = attend(pkg, q, kc, vc, table, lens, sm)
    check(o, lse, q, list(range(len(lens) + 1)), kc, vc, table, lens, sm, pkg=pkg)


@pytest.mark.parametrize("page", [32, 48, 64, 256, 1024])
def test_attention_page_sizes(pkg, page):
    lens = [700, 65, 1, 1025]
    kc, vc, table = layer(lens, 4, 128, page, page)
    q = normal((4, 16, 128), page)
    o, lse = attend(pkg, q, kc, vc, table, lens, 0.0883)
    check(o, lse, q, range(5), kc, vc, table, lens, 0.0883, pkg=pkg)


@pytest.mark.parametrize("window", [0, 1, 5, 16, 17, 100, 5000])
@pytest.mark.parametrize("hq,hkv,d,qls", [(8, 2, 128, [1, 1, 1]), (8, 8, 64, [4, 1, 3]), (20, 4, 128, [0, 5, 2]),
                                          (32, 2, 128, [7, 7, 1]), (4, 1, 64, [40, 3, 0])])
def test_attention_several_query_tokens_and_windows(pkg, hq, hkv, d, qls, window):
    lens = [130, 47, 3]
    kc, vc, table = layer(lens, hkv, d, 16, sum(qls) + window)
    cu = np.concatenate([[0], np.cumsum(qls)])
    q = normal((int(cu[-1]), hq, d), window)
    sm = d ** -0.5
    o, lse = attend(pkg, q, kc, vc, table, lens, sm, cu_q=cu, max_q=max(qls), window=window)
    check(o, lse, q, cu, kc, vc, table, lens, sm, window, pkg=pkg)


def test_rows_without_keys(pkg):
    """More query tokens than cached ones: the first rows see nothing."""
    lens, cu = [2, 0, 20], [0, 5, 8, 11]
    kc, vc, table = layer(lens, 2, 128, 16, 3)
    q = normal((11, 8, 128), 3)
    o, lse = attend(pkg, q, kc, vc, table, lens, 0.1, cu_q=cu, max_q=5)
    check(o, lse, q, cu, kc, vc, table, lens, 0.1, pkg=pkg)
    assert float(o[:3].float().abs().max()) == 0 and float(o[5:8].float().abs().max()) == 0


def test_q_from_a_projection_and_guards(pkg):
    lens, hq, hkv, d = [300, 41], 8, 2, 128
    kc, vc, table = layer(lens, hkv, d, 16, 21)
    qkv = normal((2, (hq + 2 * hkv) * d), 22).to(DEV)
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    out, raw = guarded_empty((2, hq, d), torch.bfloat16, DEV)
    lse, lraw = guarded_empty((2, hq), torch.float32, DEV)
    o, l2 = attend(pkg, q, kc, vc, table, lens, 0.1, out=out, lse=lse)
    check(o, l2, q.contiguous(), range(3), kc, vc, table, lens, 0.1, pkg=pkg)
    assert guard_intact(raw, 2 * hq * d * 2) and guard_intact(lraw, 2 * hq * 4)


@pytest.mark.parametrize("big", [1e-30, 1e30])
def test_q_of_any_size(pkg, big):
    lens = [50]
    kc, vc, table = layer(lens, 1, 128, 16, 23)
    q = (normal((1, 8, 128), 24).float() * big).to(torch.bfloat16)
    sm = 0.1 / big
    o, lse = attend(pkg, q, kc, vc, table, lens, sm)
    check(o, lse, q, range(2), kc, vc, table, lens, sm, pkg=pkg)


def test_peaked_scores(pkg):
    """A few keys take all the weight; scores far below the maximum vanish."""
    lens = [513, 40]
    kc, vc, table = layer(lens, 2, 128, 16, 25)
    q = normal((2, 16, 128), 26, 30.0)
    o, lse = attend(pkg, q, kc, vc, table, lens, 0.3)
    check(o, lse, q, range(3), kc, vc, table, lens, 0.3, pkg=pkg)


@pytest.mark.parametrize("batch,length,hq,hkv", [(1, 16384, 32, 8), (8, 4096, 32, 8), (2, 1023, 16, 16), (1, 6000, 8, 1)])
def test_attention_longer(pkg, batch, length, hq, hkv):
    lens = [length] * batch
    kc, vc, table = layer(lens[:1], hkv, 128, 16, batch, extra=0)
    table = np.repeat(table, batch, axis=0)                       # a shared prefix
    q = normal((batch, hq, 128), batch)
    sm = 128 ** -0.5
    o, lse = attend(pkg, q, kc, vc, table, lens, sm)
    check(o, lse, q, range(batch + 1), kc, vc, table, lens, sm, pkg=pkg)


@pytest.mark.parametrize("hq,d,nq", [(8, 128, 1), (4, 64, 1), (16, 128, 1), (6, 128, 4), (8, 64, 3), (8, 128, 4)])
@pytest.mark.parametrize("peaked", [False, True])
def test_one_sequence_over_many_blocks(pkg, hq, d, nq, peaked):
    """One kv head, more parts than a warp has lanes; with peaked scores a few of them hold all the weight."""
    lens = [30011]
    kc, vc, table = layer(lens, 1, d, 64, 41, extra=0)
    q = normal((nq, hq, d), 42, 30.0 if peaked else 1.0)
    sm = 0.3 if peaked else d ** -0.5
    o, lse = attend(pkg, q, kc, vc, table, lens, sm, cu_q=[0, nq], max_q=nq)
    check(o, lse, q, [0, nq], kc, vc, table, lens, sm, pkg=pkg)


def test_many_sequences(pkg):
    rng = np.random.default_rng(30)
    lens = [int(v) for v in rng.integers(0, 300, 300)]
    kc, vc, table = layer(lens[:12], 8, 64, 16, 31)
    lens = [n for _ in range(25) for n in lens[:12]]
    table = np.tile(table, (25, 1))
    q = normal((300, 16, 64), 32)
    o, lse = attend(pkg, q, kc, vc, table, lens, 0.125)
    check(o, lse, q, range(301), kc, vc, table, lens, 0.125, pkg=pkg)


def test_a_bound_far_above_the_lengths(pkg):
    lens = [77, 3]
    kc, vc, table = layer(lens, 2, 128, 16, 33)
    table = np.pad(table, ((0, 0), (0, 3000)), constant_values=-1)
    q = normal((2, 8, 128), 34)
    o, lse = attend(pkg, q, kc, vc, table, lens, 0.1, max_len=48000)
    check(o, lse, q, range(3), kc, vc, table, lens, 0.1, pkg=pkg)


def test_repeat_is_deterministic(pkg):
    lens = [3000, 2000, 10]
    kc, vc, table = layer(lens, 2, 128, 16, 35)
    q = normal((3, 8, 128), 36)
    a, la = attend(pkg, q, kc, vc, table, lens, 0.09)
    b, lb = attend(pkg, q, kc, vc, table, lens, 0.09)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


def test_bad_pages_and_lengths_are_left_out_and_reported(pkg):
    lens = [90, 40]
    kc, vc, table = layer(lens, 2, 128, 16, 37)
    table[0, 2], table[0, 4], table[1, 0] = 10 ** 6, -7, kc.shape[0]
    q = normal((2, 8, 128), 38)
    o, lse = attend(pkg, q, kc, vc, table, lens, 0.1)
    check(o, lse, q, range(3), kc, vc, table, lens, 0.1, err=16, pkg=pkg)
    kc, vc, table = layer(lens, 2, 128, 16, 37)
    o, lse = attend(pkg, q, kc, vc, table, [90, -4], 0.1)
    check(o, lse, q, range(3), kc, vc, table, [90, 0], 0.1, err=16, pkg=pkg)
    o, lse = attend(pkg, q, kc, vc, table, [10 ** 9, 40], 0.1, max_len=90)
    check(o, lse, q, range(3), kc, vc, table, [90, 40], 0.1, err=16, pkg=pkg)


def test_bad_query_ranges_are_skipped_and_reported(pkg):
    lens = [50, 40, 30]
    kc, vc, table = layer(lens, 2, 128, 16, 39)
    q = normal((6, 8, 128), 40)
    for cu in ([0, 2, 9, 12], [0, 2, 1, 3], [-3, -1, 1, 3], [0, 6, 6, 6]):
        out = torch.full((6, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        attend(pkg, q, kc, vc, table, lens, 0.1, cu_q=cu, max_q=3, out=out)
        assert pkg.check_device_error() == 16
        live = {r for b in range(3) if 0 <= cu[b] <= cu[b + 1] <= 6 and cu[b + 1] - cu[b] <= 3
                for r in range(cu[b], cu[b + 1])}
        for r in range(6):
            assert bool((out[r] == 7).all()) == (r not in live)


def test_streams_and_graph(pkg):
    lens = [600, 33]
    kc, vc, table = layer(lens, 2, 128, 16, 41)
    q = normal((2, 8, 128), 42)
    t = lambda a: torch.from_numpy(a).to(DEV)
    ks, vs = scales()
    args = [q.to(DEV), t(kc), t(vc), ks, vs, t(table), t(np.asarray(lens, dtype=np.int32)), 600, 0.1,
            pkg.kv4_workspace(128, DEV)]
    want = pkg.kv4_decode_attention(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkg.kv4_decode_attention(*args, stream=s)
    s.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = pkg.kv4_decode_attention(*args)
    args[6].copy_(t(np.asarray([17, 600][::-1], dtype=np.int32)))  # same lengths bound, other lengths
    args[6].copy_(t(np.asarray([300, 20], dtype=np.int32)))
    g.replay()
    torch.cuda.synchronize()
    o64, _, _ = ref.attention(bits(q), range(3), kc, vc, KS, VS, table, [300, 20], 0.1)
    vmax = np.nanmax(np.abs(ref.decode(vc)[:, :, :])) * float(VS)
    e = np.abs(bf16_bits_to_f64(bits(o.cpu())) - o64)
    assert np.all(e <= tolerance.kv_attention_bound(o64, o64, min(vmax, 12.0)) + 2.0 ** -9 * np.abs(o64))


def test_long_cache_offsets_pass_32_bits(pkg):
    """Blocks beyond 2^32 bytes of a cache: 4.9 GB each for K and V."""
    hkv, d, page = 32, 128, 256
    nb = (2 ** 32 + 2 ** 29) // (hkv * page // 16 * 9 * d)
    kc = torch.zeros((nb, hkv, page // 16, 9 * d), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks, vs = scales()
    n = 2 * page + 5
    table = np.array([[nb - 1, 0, nb - 2]], dtype=np.int32)
    pos = np.arange(n)
    slots = (table[0, pos // page] * page + pos % page).astype(np.int32)
    k, v = normal((n, hkv, d), 50), normal((n, hkv, d), 51)
    pkg.kv4_append(k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), ks, vs, kc, vc)
    small = np.zeros((3, hkv, page // 16, 9 * d), dtype=np.uint8)
    order = [nb - 1, 0, nb - 2]
    kc_s, vc_s = (ref.append(bits(x), pos.astype(np.int32), s, small) for x, s in ((k, KS), (v, VS)))
    for i, blk in enumerate(order):
        assert np.array_equal(kc[blk].cpu().numpy(), kc_s[i]) and np.array_equal(vc[blk].cpu().numpy(), vc_s[i])
    gk, _ = pkg.kv4_gather(kc, vc, torch.from_numpy(slots).to(DEV), ks, vs)
    w = ref.gather_bits(kc_s, pos, KS)
    assert np.array_equal(bits(gk.cpu()) & 0x7FFF, w & 0x7FFF)
    q = normal((1, hkv, d), 52)
    o, lse = pkg.kv4_decode_attention(q.to(DEV), kc, vc, ks, vs, torch.from_numpy(table).to(DEV),
                                      torch.tensor([n], dtype=torch.int32, device=DEV), n, 0.1,
                                      pkg.kv4_workspace(d, DEV), return_lse=True)
    check(o, lse, q, range(2), kc_s, vc_s, np.arange(3, dtype=np.int32)[None], [n], 0.1, pkg=pkg)
