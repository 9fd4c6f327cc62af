"""The serving-step entry points refuse what does not fit, before anything is
launched (CPU only): the binding by exceptions, the C ABI by its status."""
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


C = (6, 2, 1, 1152)            # 6 blocks of 16 tokens, 2 kv heads of 128


def plan(**kw):
    a = dict(ctx_lens=t(3), new_lens=t(3), block_table=t((3, 4)), free_blocks=t(5), free_head=t(1), page_size=16,
             num_blocks=20, num_tokens=7)
    a.update(kw)
    return fp8bs.kv_plan(**a)


def append(**kw):
    a = dict(k=t((4, 2, 128), BF), v=t((4, 2, 128), BF), slots=t(4), k_scale=t(1, F32), v_scale=t(1, F32),
             k_cache=t(C, U8), v_cache=t(C, U8))
    a.update(kw)
    return fp8bs.kv4_append(**a)


def gather(**kw):
    a = dict(k_cache=t(C, U8), v_cache=t(C, U8), slots=t(4), k_scale=t(1, F32), v_scale=t(1, F32))
    a.update(kw)
    return fp8bs.kv4_gather(**a)


def attend(**kw):
    a = dict(q=t((3, 8, 128), BF), k_cache=t(C, U8), v_cache=t(C, U8), k_scale=t(1, F32), v_scale=t(1, F32),
             block_table=t((3, 4)), seq_lens=t(3), max_seq_len=64, sm_scale=0.1, workspace=t(16, U8))
    a.update(kw)
    return fp8bs.kv4_decode_attention(**a)


def logprobs(**kw):
    a = dict(logits=t((3, 50), BF), targets=t(3), top=4)
    a.update(kw)
    return fp8bs.token_logprobs(**a)


@pytest.mark.parametrize("call", [
    lambda: plan(new_lens=t(2)), lambda: plan(block_table=t((2, 4))), lambda: plan(block_table=t(12)),
    lambda: plan(free_head=t(2)), lambda: plan(seq_lens=t(4)), lambda: plan(cu_new=t(3)), lambda: plan(slots=t(6)),
    lambda: plan(positions=t(8)), lambda: plan(requests=t(1)), lambda: plan(free_head_out=t(0)),
    lambda: append(v=t((4, 2, 64), BF)), lambda: append(k=t((4, 256), BF)), lambda: append(slots=t(5)),
    lambda: append(k_cache=t((6, 2, 1, 1151), U8)), lambda: append(v_cache=t((5, 2, 1, 1152), U8)),
    lambda: append(k_cache=t((6, 1, 1, 1152), U8)), lambda: append(k_scale=t(2, F32)),
    lambda: gather(k_cache=t((6, 2, 1, 1151), U8)), lambda: gather(v_cache=t((6, 2, 1, 576), U8)),
    lambda: gather(k=t((4, 2, 64), BF)), lambda: gather(v=t((3, 2, 128), BF)), lambda: gather(v_scale=t(0, F32)),
    lambda: attend(q=t((2, 8, 128), BF)), lambda: attend(q=t((3, 1024), BF)), lambda: attend(q=t((3, 8, 64), BF)),
    lambda: attend(block_table=t((2, 4))), lambda: attend(cu_q=t(3)), lambda: attend(out=t((3, 8, 127), BF)),
    lambda: attend(lse=t((3, 7), F32)), lambda: attend(v_cache=t((6, 2, 2, 1152), U8)),
    lambda: logprobs(logits=t(50, BF)), lambda: logprobs(targets=t(2)), lambda: logprobs(entropy=t(4, F32)),
    lambda: logprobs(top_ids=t((3, 5))), lambda: logprobs(top_logprobs=t((3, 3), F32)),
    lambda: fp8bs.kv4_cache_shape(4, 24, 2, 128),
])
def test_sizes_that_disagree_raise_value_error(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [plan, append, gather, attend, logprobs])
def test_right_sizes_on_the_cpu_are_refused_as_not_cuda(call):
    with pytest.raises(TypeError, match="CUDA"):
        call()


def test_tensors_on_different_devices_raise():
    with pytest.raises(ValueError, match="is on"):
        attend(workspace=t(16, U8, "meta"))
    with pytest.raises(ValueError, match="is on"):
        plan(free_blocks=t(5, I32, "meta"))


def test_row_strides():
    x = t((4, 6, 128), BF)
    assert fp8bs._row_stride(x[:, 2:4]) == 768 and fp8bs._row_stride(x[:1, 2:4]) == 256
    assert fp8bs._row_stride(x[:0]) == 0
    a = fp8bs._Args().need("x", x[:, 2:4], BF, rows=True)
    assert a.items[0][3]


P = ctypes.c_void_p


def test_kv_plan_status(L):
    ok = dict(ctx=P(0x10000), new=P(0x20000), b=3, table=P(0x30000), mb=4, free=P(0x40000), nf=5, head=P(0x50000),
              page=16, nb=20, t=7, seq=P(0x60000), cu=P(0x70000), slots=P(0x80000), pos=P(0x90000), req=P(0xA0000),
              out=P(0xB0000))

    def call(**kw):
        assert set(kw) <= set(ok)
        return L.fp8bs_kv_plan(*dict(ok, **kw).values(), None)
    assert call(b=-1) == call(b=16385) == call(mb=0) == call(nf=-1) == call(t=-1) == -2
    assert call(page=0) == call(page=65537) == call(nb=0) == call(nb=2 ** 28) == call(mb=2 ** 28) == -2
    for name in ("ctx", "new", "table", "free", "head", "seq", "cu", "slots", "pos", "req", "out"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P(0x10002)}) == -4, name


def test_kv4_status(L):
    p = {n: P(0x10000 * i) for i, n in enumerate(("k", "v", "slots", "ks", "vs", "kc", "vc", "ko", "vo"), 1)}

    def append_(k=p["k"], kst=256, v=p["v"], vst=256, n=4, h=2, d=128, slots=p["slots"], ks=p["ks"], vs=p["vs"],
                kc=p["kc"], vc=p["vc"], page=16, nb=6):
        return L.fp4kv_append(k, kst, v, vst, n, h, d, slots, ks, vs, kc, vc, page, nb, None)

    def gather_(kc=p["kc"], vc=p["vc"], slots=p["slots"], n=4, h=2, d=128, page=16, nb=6, ks=p["ks"], vs=p["vs"],
                ko=p["ko"], vo=p["vo"]):
        return L.fp4kv_gather(kc, vc, slots, n, h, d, page, nb, ks, vs, ko, vo, None)
    for f in (append_, gather_):
        assert f(n=-1) == f(h=0) == f(h=4096) == f(d=96) == f(page=8) == f(page=24) == f(page=8192) == -2
        assert f(nb=0) == f(nb=2 ** 28) == -2
        assert f(n=0, slots=None) == 0
        for name in ("slots", "ks", "vs", "kc", "vc"):
            assert f(**{name: None}) == -1, name
            assert f(**{name: P(0x10002)}) == -4, name
        assert f(kc=P(0x10008)) == f(vc=P(0x10008)) == -4
    assert append_(kst=-8) == append_(vst=2 ** 40) == -2
    assert append_(k=None) == append_(v=None) == gather_(ko=None) == gather_(vo=None) == -1
    assert append_(k=P(0x10008)) == append_(kst=260) == append_(vst=257) == gather_(ko=P(0x10008)) == -4


def test_kv4_attention_status(L):
    need = L.fp4kv_attention_ws_bytes(128)
    assert need > 0 and L.fp4kv_attention_ws_bytes(64) > 0 and L.fp4kv_attention_ws_bytes(96) == -2
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.kv4_workspace(80)
    ok = dict(q=P(0x10000), qst=1024, cu=None, t=3, mq=1, kc=P(0x20000), vc=P(0x30000), ks=P(0x40000), vs=P(0x50000),
              bt=P(0x60000), mb=4, lens=P(0x70000), b=3, hq=8, hkv=2, d=128, page=16, nb=6, ml=64, w=0,
              sm=ctypes.c_float(0.1), out=P(0x80000), lse=P(0x90000), ws=P(0xA0000), wsb=need)

    def call(**kw):
        assert set(kw) <= set(ok)
        return L.fp4kv_decode_attention(*dict(ok, **kw).values(), None)
    for kw in (dict(d=96), dict(page=24), dict(hq=7), dict(hq=0), dict(b=-1), dict(b=65536), dict(t=-1), dict(mq=0),
               dict(mq=65536), dict(t=4), dict(mq=2), dict(mb=0), dict(ml=65), dict(ml=-1), dict(w=-1), dict(qst=-8),
               dict(sm=ctypes.c_float(float("nan"))), dict(sm=ctypes.c_float(float("inf"))), dict(wsb=need - 1)):
        assert call(**kw) == -2, kw
    assert call(b=0, t=0, q=None) == 0
    for name in ("q", "kc", "vc", "ks", "vs", "bt", "lens", "out", "ws"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P(0x10002)}) == -4, name
    assert call(qst=1025) == call(lse=P(0x10002)) == call(cu=P(0x10002)) == call(out=P(0x10008)) == -4


def test_token_logprobs_status(L):
    ok = dict(x=P(0x10000), f32=0, st=50, m=3, v=50, tg=P(0x20000), k=4, lp=P(0x30000), en=P(0x40000), ids=P(0x50000),
              tops=P(0x60000))

    def call(**kw):
        assert set(kw) <= set(ok)
        return L.fp8bs_token_logprobs(*dict(ok, **kw).values(), None)
    assert call(m=-1) == call(v=0) == call(st=49) == call(k=-1) == call(k=33) == call(k=20, v=19) == -2
    assert call(m=0, x=None) == 0
    for name in ("x", "tg", "lp", "en", "ids", "tops"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P(0x10001)}) == -4, name
    assert call(f32=1, x=P(0x10002)) == -4
