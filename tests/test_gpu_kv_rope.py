"""GPU tests of fp8kv_rope_append and fp4kv_rope_append: the caches bit for
bit, q within its roundings.

q: a product with r, one with the weight and one each with cos and sin round
by half a step (2^-24) each, the difference once more; the sum of D squares
adds 8 of a lane and log2 of the lanes one after the other, fewer than 14
roundings, which r halves; r itself one: 5 + 7 + 1 < 14 half steps of |n1 c| +
|n2 s|, then one bf16 rounding, half a step of the result (2^-8 of it at most).
"""
import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import bits, guard_intact, guarded_empty, lib_or_skip
from oracle.tolerance import bf16_bits_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def table(positions, rot):
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def inputs_of(t, hq, hkv, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((t, (hq + 2 * hkv) * d), generator=g) * scale).to(torch.bfloat16)
    return qkv


def slices(qkv, hq, hkv, d):
    return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
            qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))


def weights(d, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)


def empty_cache(bits_, nb, page, hkv, d, fill=0):
    shape = (nb, hkv, page // 16, 9 * d) if bits_ == 4 else (nb, page, hkv, d)
    return np.full(shape, fill, dtype=np.uint8)


def run(pkg, bits_, qkv, hq, hkv, d, pos, slots, tab, page, nb, qw=None, kw=None, interleaved=False, eps=EPS, ks=None,
        vs=None, err=0, **kw_args):
    """One call and its comparison.  Returns q."""
    top = 2688.0 if bits_ == 4 else 448.0
    ks = np.float32(8 / top) if ks is None else ks
    vs = np.float32(6 / top) if vs is None else vs
    q, k, v = slices(qkv.to(DEV), hq, hkv, d)
    k0, v0 = empty_cache(bits_, nb, page, hkv, d, 3), empty_cache(bits_, nb, page, hkv, d, 5)
    kc, vc = torch.from_numpy(k0.copy()).to(DEV), torch.from_numpy(v0.copy()).to(DEV)
    before = torch.full((len(pos), hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    out, raw = guarded_empty((len(pos), hq, d), torch.bfloat16, DEV)
    out.copy_(before)
    fn = pkg.kv4_rope_append if bits_ == 4 else pkg.kv_rope_append
    got = fn(q, k, v, torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(slots, dtype=torch.int32, device=DEV),
             torch.from_numpy(tab).to(DEV), torch.tensor([ks], device=DEV), torch.tensor([vs], device=DEV), kc, vc,
             q_norm=None if qw is None else qw.to(DEV), k_norm=None if kw is None else kw.to(DEV), eps=eps,
             interleaved=interleaved, out=out, **kw_args)
    assert got is out and guard_intact(raw, out.numel() * 2)
    pos, slots = np.asarray(pos), np.asarray(slots)
    live = (pos >= 0) & (pos < len(tab))
    at = np.where(live, pos, 0)
    half = tab.shape[1] // 2
    cos, sin = tab[at, :half], tab[at, half:]
    qb, kb, vb = (bits(x.contiguous().cpu()) for x in (q, k, v))
    store = ref.store4 if bits_ == 4 else ref.store8
    kept = np.where(live, slots, -1)
    k_want = store(ref.turned(kb, None if kw is None else bits(kw), eps, cos, sin, interleaved), kept, ks, k0)
    v_want = store(bf16_bits_to_f64(vb), kept, vs, v0)
    assert np.array_equal(kc.cpu().numpy(), k_want)
    assert np.array_equal(vc.cpu().numpy(), v_want)
    want = ref.turned(qb, None if qw is None else bits(qw), eps, cos, sin, interleaved, rounded=False)
    size = ref.turned(qb & 0x7FFF, None if qw is None else bits(qw) & 0x7FFF, eps, np.abs(cos), np.abs(sin), interleaved,
                      rounded=False)
    size = np.maximum(np.abs(size), np.abs(want))
    if not interleaved:                                         # |n1 c| + |n2 s| of either of a pair
        size[..., :half] = np.maximum(size[..., :half], size[..., half:2 * half])
        size[..., half:2 * half] = size[..., :half]
    else:
        size[..., 0:2 * half:2] = np.maximum(size[..., 0:2 * half:2], size[..., 1:2 * half:2])
        size[..., 1:2 * half:2] = size[..., 0:2 * half:2]
    have = bf16_bits_to_f64(bits(out.cpu()))
    tol = 14 * 2.0 ** -24 * size + 2.0 ** -8 * (np.abs(want) + 14 * 2.0 ** -24 * size) + 2.0 ** -133
    assert np.all(np.abs(have - want)[live] <= tol[live]), np.max((np.abs(have - want) - tol)[live])
    assert np.all(have[~live] == 7.0)                          # rows of no position are left as they were
    assert pkg.check_device_error() == err
    return out


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("bits_,t,hq,hkv,d,page,rot,interleaved", [
    (4, 1, 1, 1, 64, 16, 64, False), (4, 1, 32, 8, 128, 16, 128, False), (4, 7, 5, 5, 128, 48, 128, True),
    (4, 33, 16, 2, 64, 32, 32, False), (4, 65, 40, 8, 128, 64, 96, False), (4, 3, 65, 1, 128, 16, 16, True),
    (8, 1, 32, 8, 128, 16, 128, False), (8, 9, 3, 3, 128, 16, 112, False), (8, 130, 64, 8, 128, 32, 64, True),
    (8, 31, 12, 4, 128, 48, 48, False)])
def test_matches_the_definition(pkg, bits_, t, hq, hkv, d, page, rot, interleaved, norm):
    rng = np.random.default_rng(t + hq)
    nb = t // page + 2
    slots = rng.permutation(nb * page)[:t]
    pos = rng.integers(0, 5000, t)
    run(pkg, bits_, inputs_of(t, hq, hkv, d, t + d), hq, hkv, d, pos, slots, table(5000, rot), page, nb,
        weights(d, 1) if norm else None, weights(d, 2) if norm else None, interleaved)


@pytest.mark.parametrize("bits_", [4, 8])
def test_many_tokens(pkg, bits_):
    """More than a wave of the largest CTAs; only k normed."""
    t, hq, hkv, d, page = 2999, 8, 2, 128, 16
    slots = np.random.default_rng(0).permutation(t + 100)[:t]
    run(pkg, bits_, inputs_of(t, hq, hkv, d, 3), hq, hkv, d, np.arange(t) + 1000, slots, table(4096, d), page,
        (t + 100) // page + 1, None, weights(d, 4))


@pytest.mark.parametrize("bits_", [4, 8])
def test_padding_and_bad_places(pkg, bits_):
    t, hq, hkv, d, page, nb = 9, 4, 2, 128, 16, 3
    x = inputs_of(t, hq, hkv, d, 5)
    tab = table(64, d)
    pos, slots = np.arange(t), np.arange(t) + 4
    pos[8], slots[8] = -1, -1                                   # padding
    slots[2] = -1                                               # not stored, but rotated
    run(pkg, bits_, x, hq, hkv, d, pos, slots, tab, page, nb, weights(d, 1), weights(d, 2))
    for where, what in ((pos, 64), (pos, -2), (slots, nb * page), (slots, -2)):
        kept = where[4]
        where[4] = what
        run(pkg, bits_, x, hq, hkv, d, pos, slots, tab, page, nb, weights(d, 1), weights(d, 2), err=16)
        where[4] = kept


@pytest.mark.parametrize("bits_", [4, 8])
@pytest.mark.parametrize("scale,s", [(1e-20, 1e-22), (3e4, 100.0), (1e-30, 1e-30), (1e8, 1e5)])
def test_far_scales(pkg, bits_, scale, s):
    t, hq, hkv, d, page = 20, 2, 2, 128, 16
    x = inputs_of(t, hq, hkv, d, 6, scale)
    for w in (None, weights(d, 3)):
        run(pkg, bits_, x, hq, hkv, d, np.arange(t), np.arange(t), table(32, d), page, 2, w, w, ks=np.float32(s),
            vs=np.float32(s))


@pytest.mark.parametrize("bits_", [4, 8])
def test_zero_heads_and_uneven_ones(pkg, bits_):
    """Heads of zeros; of one element; whose squares differ by 2^40 and cancel nothing."""
    t, hq, hkv, d, page = 16, 2, 2, 128, 16
    x = inputs_of(t, hq, hkv, d, 7)
    x[0] = 0
    x[1] = 0
    x[1, ::d] = 3.0
    x[2:8] *= torch.tensor(2.0) ** torch.randint(-20, 20, x[2:8].shape, generator=torch.Generator().manual_seed(1))
    run(pkg, bits_, x, hq, hkv, d, np.arange(t), np.arange(t), table(32, d), page, 1, weights(d, 1), weights(d, 2))


@pytest.mark.parametrize("bits_", [4, 8])
def test_nan_stays_in_its_head(pkg, bits_):
    t, hq, hkv, d, page = 6, 4, 2, 128, 16
    x = inputs_of(t, hq, hkv, d, 8)
    args = (hq, hkv, d, np.arange(t), np.arange(t), table(32, d), page, 1)
    fn = pkg.kv4_rope_append if bits_ == 4 else pkg.kv_rope_append

    def caches(x):
        q, k, v = slices(x.to(DEV), hq, hkv, d)
        kc, vc = (torch.from_numpy(empty_cache(bits_, 1, page, hkv, d)).to(DEV) for _ in range(2))
        i = torch.arange(t, dtype=torch.int32, device=DEV)
        s = torch.tensor([0.01], device=DEV)
        w = weights(d, 1).to(DEV)
        o = fn(q, k, v, i, i, torch.from_numpy(table(32, d)).to(DEV), s, s, kc, vc, q_norm=w, k_norm=w)
        return o, kc, vc
    clean = caches(x)
    x = x.clone()
    x[3, d + 5] = float("nan")                                  # query head 1 of token 3
    x[4, hq * d + 7] = float("nan")                             # key head 0 of token 4
    x[5, (hq + hkv) * d + d + 9] = float("nan")                 # value head 1 of token 5
    o, kc, vc = caches(x)
    assert bool(torch.isnan(o[3, 1]).all())
    o[3, 1] = clean[0][3, 1]
    assert torch.equal(o, clean[0])
    if bits_ == 4:
        s = torch.tensor([0.01], device=DEV)
        i = torch.arange(t, dtype=torch.int32, device=DEV)
        k, v = pkg.kv4_gather(kc, vc, i, s, s)
        ck, cv = pkg.kv4_gather(clean[1], clean[2], i, s, s)
        group = v[5, 1, :16]
    else:
        k, v, ck, cv = (c.view(torch.float8_e4m3fn)[0].float() for c in (kc, vc, clean[1], clean[2]))
        group = v[5, 1, 9:10]
    assert bool(torch.isnan(k[4, 0]).all()) and bool(torch.isnan(group).all())
    k[4, 0], group[:] = ck[4, 0], cv[5, 1, :16] if bits_ == 4 else cv[5, 1, 9:10]
    assert torch.equal(k[:t], ck[:t]) and torch.equal(v[:t], cv[:t])
    assert pkg.check_device_error() == 0 and args


def test_q_in_place_and_empty(pkg):
    t, hq, hkv, d, page = 50, 8, 2, 128, 16
    x = inputs_of(t, hq, hkv, d, 9).to(DEV)
    q, k, v = (y.contiguous() for y in slices(x, hq, hkv, d))
    tab = torch.from_numpy(table(64, d)).to(DEV)
    i = torch.arange(t, dtype=torch.int32, device=DEV)
    s = torch.tensor([0.01], device=DEV)
    kc, vc = (torch.zeros((4, page, hkv, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    w = weights(d, 1).to(DEV)
    for pairs in (False, True):
        want = pkg.kv_rope_append(q, k, v, i, i, tab, s, s, kc, vc, q_norm=w, interleaved=pairs)
        mine = q.clone()
        assert pkg.kv_rope_append(mine, k, v, i, i, tab, s, s, kc, vc, q_norm=w, interleaved=pairs, out=mine) is mine
        assert torch.equal(mine, want)
    none = pkg.kv_rope_append(q[:0], k[:0], v[:0], i[:0], i[:0], tab, s, s, kc, vc)
    assert none.shape == (0, hq, d) and pkg.check_device_error() == 0


@pytest.mark.parametrize("bits_", [4, 8])
def test_agrees_with_the_append_without_rotation(pkg, bits_):
    """At position 0 nothing turns: without a norm the caches are those of the plain appends."""
    t, hq, hkv, d, page, nb = 40, 4, 4, 128, 16, 4
    q, k, v = slices(inputs_of(t, hq, hkv, d, 10).to(DEV), hq, hkv, d)
    i = torch.arange(t, dtype=torch.int32, device=DEV)
    tab = torch.from_numpy(table(1, d)).to(DEV)
    s = torch.tensor([0.01], device=DEV)
    a, b, c, e = (torch.from_numpy(empty_cache(bits_, nb, page, hkv, d)).to(DEV) for _ in range(4))
    if bits_ == 4:
        out = pkg.kv4_rope_append(q, k, v, torch.zeros_like(i), i, tab, s, s, a, b)
        pkg.kv4_append(k, v, i, s, s, c, e)
    else:
        out = pkg.kv_rope_append(q, k, v, torch.zeros_like(i), i, tab, s, s, a, b)
        pkg.kv_append(k.contiguous(), i, s, c)
        pkg.kv_append(v.contiguous(), i, s, e)
    assert torch.equal(out, q) and torch.equal(b, e)
    zero = 0x7F7F if bits_ == 8 else None                       # 0 - (-0) and the like may change a zero's sign
    if zero:
        a, c = (torch.where((x & 0x7F) == 0, torch.zeros_like(x), x) for x in (a, c))
    assert torch.equal(a, c)


def test_graph_and_streams(pkg):
    t, hq, hkv, d, page, nb = 70, 8, 2, 128, 16, 6
    x = inputs_of(t, hq, hkv, d, 11).to(DEV)
    q, k, v = slices(x, hq, hkv, d)
    i = torch.arange(t, dtype=torch.int32, device=DEV)
    tab = torch.from_numpy(table(128, d)).to(DEV)
    s = torch.tensor([0.003], device=DEV)
    shape = pkg.kv4_cache_shape(nb, page, hkv, d)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    w = weights(d, 1).to(DEV)

    def call(**kw):
        return pkg.kv4_rope_append(q, k, v, i, i, tab, s, s, kc, vc, q_norm=w, k_norm=w, **kw)
    want = call()
    kept = kc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    kc.zero_()
    graph.replay()
    assert torch.equal(got, want) and torch.equal(kc, kept)
    x.mul_(2.0)                                                 # new inputs in the same place
    graph.replay()
    assert torch.equal(kc, torch.zeros_like(kc).copy_(kc)) and torch.equal(got, call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kc.zero_()
    torch.cuda.synchronize()
    other = call(stream=side)
    side.synchronize()
    assert torch.equal(other, got)
    assert pkg.check_device_error() == 0
