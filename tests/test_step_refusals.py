"""What the entry points between a step's linears and its attention refuse,
before anything is launched (CPU only): norm and rotation into the caches,
routing and combination, sampling.  The binding by exceptions, the C ABI by
its status."""
import ctypes

import pytest
import torch

import fp8_block_scaled_02_gb300 as fp8bs

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def L():
    from fp8_block_scaled_02_gb300 import build
    build.build()
    return fp8bs.lib()


def t(shape, dtype=I32, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


C8, C4 = (6, 16, 2, 128), (6, 2, 1, 1152)       # 6 blocks of 16 tokens, 2 kv heads of 128


def rope8(cache=C8, fn=None, **kw):
    a = dict(q=t((4, 8, 128), BF), k=t((4, 2, 128), BF), v=t((4, 2, 128), BF), positions=t(4), slots=t(4),
             cos_sin=t((50, 64), F32), k_scale=t(1, F32), v_scale=t(1, F32), k_cache=t(cache, U8), v_cache=t(cache, U8))
    a.update(kw)
    return (fn or fp8bs.kv_rope_append)(**a)


def rope4(**kw):
    return rope8(C4, fp8bs.kv4_rope_append, **kw)


def route(**kw):
    return fp8bs.moe_route(**dict(dict(logits=t((3, 16), F32), topk=2), **kw))


def combine(**kw):
    return fp8bs.moe_combine(**dict(dict(y=t((3, 2, 64), BF), weights=t((3, 2), F32)), **kw))


def sample(**kw):
    return fp8bs.sample_tokens(**dict(dict(logits=t((3, 50), BF), u=t((3, 2), F32)), **kw))


@pytest.mark.parametrize("call", [
    *[lambda kw=kw, f=f: f(**kw()) for f in (rope8, rope4) for kw in (
        lambda: dict(q=t((4, 1024), BF)), lambda: dict(q=t((3, 8, 128), BF)), lambda: dict(q=t((4, 8, 64), BF)),
        lambda: dict(k=t((4, 256), BF)), lambda: dict(k=t((4, 3, 128), BF)), lambda: dict(v=t((4, 1, 128), BF)),
        lambda: dict(positions=t(3)), lambda: dict(slots=t(5)), lambda: dict(cos_sin=t(64, F32)),
        lambda: dict(k_scale=t(2, F32)), lambda: dict(v_scale=t(0, F32)), lambda: dict(q_norm=t(64, BF)),
        lambda: dict(k_norm=t(129, BF)), lambda: dict(out=t((4, 8, 127), BF)), lambda: dict(k_cache=t((6, 16, 1, 128), U8)),
        lambda: dict(v_cache=t((5, 16, 2, 128), U8)))],
    lambda: rope8(k_cache=t(C4, U8)), lambda: rope4(k_cache=t(C8, U8)), lambda: rope4(v_cache=t((6, 2, 2, 1152), U8)),
    lambda: route(logits=t(16, F32)), lambda: route(topk=0), lambda: route(topk=17), lambda: route(scoring="relu"),
    lambda: route(bias=t(15, F32)), lambda: route(ids=t((3, 3))), lambda: route(weights=t((2, 2), F32)),
    lambda: route(logits=torch.as_strided(t(64, F32), (3, 16), (8, 1))),
    lambda: combine(y=t((3, 128), BF)), lambda: combine(weights=t((3, 3), F32)), lambda: combine(ids=t((2, 2)), num_experts=4),
    lambda: combine(ids=t((3, 2))), lambda: sample(u=t((2, 3), F32)),
    lambda: combine(residual=t((3, 63), BF)), lambda: combine(residual=t(64, BF)), lambda: combine(out=t((2, 64), BF)),
    lambda: sample(logits=t(50, BF)), lambda: sample(u=t((3, 1), F32)), lambda: sample(temperature=t(2, F32)),
    lambda: sample(top_k=t(4)), lambda: sample(top_p=t(1, F32)), lambda: sample(min_p=t(1, F32)),
    lambda: sample(tokens=t(2)), lambda: sample(logprobs=t(4, F32)),
    lambda: sample(logits=torch.as_strided(t(200, BF), (3, 50), (49, 1))),
])
def test_sizes_that_disagree_raise_value_error(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [rope8, rope4, route, combine, sample])
def test_right_sizes_on_the_cpu_are_refused_as_not_cuda(call):
    with pytest.raises(TypeError, match="CUDA"):
        call()


@pytest.mark.parametrize("call", [
    lambda: rope8(q=t((4, 8, 128), F32)), lambda: rope4(positions=t(4, torch.int64)), lambda: rope8(cos_sin=t((50, 64), BF)),
    lambda: rope8(k_norm=t(128, F32)), lambda: rope4(q_norm=1.0), lambda: route(bias=0.0), lambda: combine(residual=1),
    lambda: sample(top_k=40), lambda: sample(min_p=0.1), lambda: sample(tokens=[0, 0, 0]), lambda: route(logits=t((3, 16), torch.float16)), lambda: route(bias=t(16, BF)),
    lambda: combine(weights=t((3, 2), BF)), lambda: combine(ids=t((3, 2), torch.int64), num_experts=4), lambda: sample(temperature=0.7),
    lambda: sample(top_k=t(3, torch.int64)), lambda: sample(top_p=t(3, torch.float64)), lambda: sample(u=t((3, 2), BF)),
    lambda: combine(y=t((3, 4, 64), BF)[:, ::2]), lambda: sample(logits=t((3, 100), BF)[:, ::2]),
    lambda: rope8(q=t((4, 16, 128), BF)[:, ::2]),
])
def test_other_types_and_layouts_raise(call):
    with pytest.raises((TypeError, ValueError)):
        call()


def test_tensors_on_different_devices_raise():
    for call in (lambda: rope4(slots=t(4, I32, "meta")), lambda: route(bias=t(16, F32, "meta")),
                 lambda: combine(ids=t((3, 2), I32, "meta"), num_experts=4), lambda: sample(top_p=t(3, F32, "meta"))):
        with pytest.raises(ValueError, match="is on"):
            call()


P = ctypes.c_void_p


def caller(fn, ok):
    def call(**kw):
        assert set(kw) <= set(ok), set(kw) - set(ok)
        return fn(*dict(ok, **kw).values(), None)
    return call


@pytest.mark.parametrize("four_bit", [False, True])
def test_rope_status(L, four_bit):
    p = {n: P(0x10000 * i) for i, n in enumerate(("q", "k", "v", "pos", "slots", "cs", "qw", "kw", "out", "ks", "vs", "kc",
                                                  "vc"), 1)}
    ok = dict(q=p["q"], qst=1536, k=p["k"], kst=1536, v=p["v"], vst=1536, n=4, hq=8, hkv=2, d=128, pos=p["pos"],
              slots=p["slots"], cs=p["cs"], mp=50, rot=64, il=0, qw=p["qw"], kw=p["kw"], eps=ctypes.c_float(1e-6),
              out=p["out"], ks=p["ks"], vs=p["vs"], kc=p["kc"], vc=p["vc"])
    ok.update(dict(page=16, nb=6) if four_bit else dict(ns=96))
    call = caller(L.fp4kv_rope_append if four_bit else L.fp8kv_rope_append, ok)
    bad = [dict(n=-1), dict(n=2 ** 31), dict(hq=0), dict(hq=65536), dict(hkv=0), dict(hkv=4096), dict(d=96), dict(d=256),
           dict(mp=0), dict(mp=2 ** 31), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(qst=-8),
           dict(kst=2 ** 40), dict(vst=-1), dict(n=2 ** 30, hq=1024)]
    bad += [dict(eps=ctypes.c_float(v)) for v in (-1e-6, float("nan"), float("inf"))]
    bad += [dict(page=24), dict(page=8), dict(nb=0), dict(nb=2 ** 28), dict(d=64, rot=80)] if four_bit else \
        [dict(ns=0), dict(ns=2 ** 31), dict(d=64)]
    for kw in bad:
        assert call(**kw) == -2, kw
    assert call(n=0, q=None, kc=None) == 0
    for name in ("q", "k", "v", "pos", "slots", "cs", "out", "ks", "vs", "kc", "vc"):
        assert call(**{name: None}) == -1, name
    for name in p:
        assert call(**{name: P(0x10002)}) == -4, name
    for name in ("q", "k", "v", "cs", "qw", "kw", "out", "kc", "vc"):
        assert call(**{name: P(0x10008)}) == -4, name
    for name in ("qst", "kst", "vst"):
        assert call(**{name: 1540}) == -4, name


def test_moe_route_status(L):
    ok = dict(x=P(0x10000), f32=1, st=64, m=3, e=64, k=4, sc=0, bias=P(0x20000), g=8, tg=2, gt=2, rn=1,
              scale=ctypes.c_float(1), ids=P(0x30000), w=P(0x40000))
    call = caller(L.fp8bs_moe_route, ok)
    for kw in (dict(m=-1), dict(m=2 ** 31), dict(e=0), dict(e=1025, st=1025, g=1, tg=1), dict(k=0), dict(k=33), dict(k=17),
               dict(st=63), dict(st=-64), dict(st=2 ** 40), dict(g=0), dict(g=7), dict(g=64), dict(tg=0), dict(tg=9),
               dict(gt=0), dict(gt=3), dict(g=32, tg=4, gt=3), dict(sc=2), dict(sc=-1), dict(m=2 ** 29),
               dict(scale=ctypes.c_float(float("nan"))), dict(scale=ctypes.c_float(float("inf")))):
        assert call(**kw) == -2, kw
    assert call(m=0, x=None, ids=None) == 0
    for name in ("x", "ids", "w"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "bias", "ids", "w"):
        assert call(**{name: P(0x10002)}) == -4, name
    assert call(f32=0, x=P(0x10001)) == -4


def test_moe_combine_status(L):
    ok = dict(y=P(0x10000), w=P(0x20000), ids=P(0x30000), e=8, res=P(0x40000), m=3, k=2, n=64, out=P(0x50000))
    call = caller(L.fp8bs_moe_combine, ok)
    for kw in (dict(m=-1), dict(m=2 ** 31), dict(k=0), dict(k=1025), dict(n=0), dict(n=2 ** 31), dict(e=-1), dict(e=2 ** 31),
               dict(m=2 ** 30, n=8192), dict(m=2 ** 30, n=1025, k=1), dict(m=2 ** 30, k=4)):
        assert call(**kw) == -2, kw
    assert call(m=0, y=None, out=None) == 0
    for name in ("y", "w", "out"):
        assert call(**{name: None}) == -1, name
    for name in ("y", "w", "ids", "res", "out"):
        assert call(**{name: P(0x10001)}) == -4, name
    assert call(w=P(0x10002)) == call(ids=P(0x10002)) == -4


def test_sample_tokens_status(L):
    ok = dict(x=P(0x10000), f32=0, st=50, m=3, v=50, u=P(0x20000), t=P(0x30000), tk=P(0x40000), tp=P(0x50000), mp=P(0x60000),
              tok=P(0x70000), lp=P(0x80000))
    call = caller(L.fp8bs_sample_tokens, ok)
    for kw in (dict(m=-1), dict(m=2 ** 28), dict(v=0), dict(v=2 ** 20 + 1, st=2 ** 21), dict(st=49), dict(st=-50),
               dict(st=2 ** 40)):
        assert call(**kw) == -2, kw
    assert call(m=0, x=None, u=None, tok=None) == 0
    for name in ("x", "u", "tok"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "u", "t", "tk", "tp", "mp", "tok", "lp"):
        assert call(**{name: P(0x10001)}) == -4, name
    assert call(f32=1, x=P(0x10002)) == -4
