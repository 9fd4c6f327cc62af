"""Rows that repeat or overlap in what the serving-step calls read: the row
stride that reaches the library (CPU), and the results (GPU).

token_logprobs reads rows a stride apart; logits.expand(M, V), several
targets under one row of logits, has the stride 0.  kv4_append and
kv4_decode_attention take one row for every token in the same way.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

import fp8_block_scaled_02_gb300 as fp8bs
import serving_reference as ref

DEV = "cuda"
BF = torch.bfloat16
P = ctypes.c_void_p


@pytest.fixture
def recorded(monkeypatch):
    """The arguments that would reach the library, without a GPU."""
    calls = []
    monkeypatch.setattr(fp8bs, "_checked", lambda *specs: torch.device("cpu"))
    monkeypatch.setattr(fp8bs, "_call", lambda device, what, fn, args, stream=None: calls.append(args))
    return calls


@pytest.mark.parametrize("logits,stride", [
    (torch.zeros((4, 1000), dtype=BF), 1000),
    (torch.zeros((4, 1008), dtype=BF)[:, :1000], 1008),
    (torch.zeros((1, 1000), dtype=BF).expand(4, 1000), 0),
    (torch.zeros(1000).expand(7, 1000), 0),
    (torch.zeros((9, 1000), dtype=BF)[::2], 2000),
    (torch.zeros((1, 1000), dtype=BF), 1000),
    (torch.zeros(1500, dtype=BF).as_strided((1, 1000), (3, 1)), 1000),    # one row has no next one
    (torch.zeros((0, 1000), dtype=BF), 1000),
])
def test_the_row_stride_of_logits(recorded, logits, stride):
    fp8bs.token_logprobs(logits, torch.zeros(logits.shape[0], dtype=torch.int32), 2)
    assert recorded[0][2] == stride


@pytest.mark.parametrize("stride", [1, 100, 999])
def test_overlapping_rows_of_logits_are_refused(stride):
    logits = torch.zeros(4000, dtype=BF).as_strided((4, 1000), (stride, 1))
    with pytest.raises(ValueError, match="overlap"):
        fp8bs.token_logprobs(logits, torch.zeros(4, dtype=torch.int32), 2)


def test_row_strides_at_the_c_entry():
    if not os.path.exists(fp8bs.LIB_PATH):
        pytest.skip("libfp8bs.so has not been built")
    lib = fp8bs.lib()

    def call(stride, x=0x10001):  # misaligned: refused for that once the sizes have passed
        return lib.fp8bs_token_logprobs(P(x), 0, stride, 3, 50, P(0x20000), 4, P(0x30000), P(0x40000), P(0x50000),
                                        P(0x60000), None)
    assert call(-1) == call(1) == call(49) == -2
    assert call(0) == call(50) == call(51) == -4


# --------------------------------------------------------------------- GPU
@pytest.fixture(scope="module")
def pkg():
    from gpu_helpers import lib_or_skip
    return lib_or_skip()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("m,v,top", [(2, 1000, 5), (5, 33, 32), (700, 3001, 4), (4, 152064, 20)])
def test_one_row_of_logits_for_many_targets(pkg, m, v, top, dtype):
    """Every row's result is that of the row alone, written out."""
    row = (torch.randn((1, v + 3), generator=torch.Generator().manual_seed(v)) * 2).to(dtype).to(DEV)[:, 1:v + 1]
    targets = torch.arange(m, dtype=torch.int32, device=DEV) % v
    got = pkg.token_logprobs(row.expand(m, v), targets, top)
    want = pkg.token_logprobs(row.repeat(m, 1), targets, top)
    assert torch.equal(got.top_ids, want.top_ids)
    # l = sum 2^d in fp32: a thread of the smallest CTA, 128 threads, adds V / 128 terms, the merges fewer than 64 (half
    # a step, 2^-24, each); a term is off by an exp2 (2^-22) and by the roundings of d, 2^-24 and 2^-25 of |d|, whose
    # mean under the weights is below 17 log2 e (at most 152064 tokens): r in all, then two roundings of the result
    r = (v / 128 + 64) * 2.0 ** -24 + 2.0 ** -22 + 25 * 2.0 ** -23
    x = row[0].double()
    logp = x - torch.logsumexp(x, 0)
    assert torch.equal(got.top_ids[0].long(), torch.sort(x, descending=True, stable=True).indices[:top])
    lp = logp[targets.long()]
    bound = r + 2.0 ** -22 * (lp.abs() + 12)
    assert bool(((got.logprobs.double() - lp).abs() <= bound).all())
    assert bool(((want.logprobs.double() - lp).abs() <= bound).all())
    assert all(torch.equal(got.entropy[i], got.entropy[0]) for i in (m // 2, m - 1))
    assert pkg.check_device_error() == 0


@pytest.mark.gpu
def test_one_key_and_query_for_every_token(pkg):
    t, hq, hkv, d, page, nb = 5, 8, 2, 128, 16, 3
    g = torch.Generator().manual_seed(1)
    k, v, q = ((torch.randn((1, h, d), generator=g)).to(BF) for h in (hkv, hkv, hq))
    s = np.float32(5.5 / 2688)
    scale = torch.tensor([s], device=DEV)
    zero = np.zeros((nb, hkv, 1, 9 * d), dtype=np.uint8)
    kc, vc = torch.from_numpy(zero.copy()).to(DEV), torch.from_numpy(zero.copy()).to(DEV)
    slots = np.array([3, 40, 17, 0, 31], dtype=np.int32)
    pkg.kv4_append(k.to(DEV).expand(t, hkv, d), v.to(DEV).expand(t, hkv, d), torch.from_numpy(slots).to(DEV), scale,
                   scale, kc, vc)
    from gpu_helpers import bits
    for c, x in ((kc, k), (vc, v)):
        assert np.array_equal(c.cpu().numpy(), ref.append(bits(x.repeat(t, 1, 1)), slots, s, zero))
    table = torch.tensor([[0, 1]] * 3, dtype=torch.int32, device=DEV)
    lens = torch.tensor([30, 4, 17], dtype=torch.int32, device=DEV)
    ws = pkg.kv4_workspace(d, DEV)
    args = (kc, vc, scale, scale, table, lens, 32, 0.1, ws)
    got = pkg.kv4_decode_attention(q.to(DEV).expand(3, hq, d), *args)
    want = pkg.kv4_decode_attention(q.to(DEV).repeat(3, 1, 1), *args)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert pkg.check_device_error() == 0
