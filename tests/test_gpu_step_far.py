"""GPU tests of the step's operators where offsets pass 32 bits: caches, experts' outputs and strided rows of more than
4 GB, compared at their ends with small calls."""
import pytest
import torch

from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


@pytest.mark.parametrize("four_bit", [False, True])
def test_far_slots(pkg, four_bit):
    hkv, d, page, t = 8, 128, 16, 6
    row = hkv * (d * 9 // 16 if four_bit else d)                # bytes of a token
    nb = ((1 << 32) // row + 5 * page) // page
    shape = pkg.kv4_cache_shape(nb, page, hkv, d) if four_bit else (nb, page, hkv, d)
    small = pkg.kv4_cache_shape(6, page, hkv, d) if four_bit else (6, page, hkv, d)
    g = torch.Generator().manual_seed(0)
    qkv = torch.randn((t, 10 * hkv * d), generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([8 * hkv * d, hkv * d, hkv * d], 1))
    a = torch.arange(50)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    tab = torch.cat([a.cos(), a.sin()], 1).to(DEV)
    pos = torch.arange(t, dtype=torch.int32, device=DEV) + 7
    s = torch.tensor([0.002 if four_bit else 0.02], device=DEV)
    fn = pkg.kv4_rope_append if four_bit else pkg.kv_rope_append
    near = torch.tensor([0, 17, 35, 50, 81, 95], dtype=torch.int32, device=DEV)     # blocks 0, 1, 2, 3, 5, 5
    blocks = torch.tensor([0, 1, nb - 4, nb - 3, nb - 2, nb - 1], device=DEV)
    far = (blocks[near // page] * page + near % page).to(torch.int32)
    big, little = ([torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)] for n in (shape, small))
    assert big[0].numel() > 1 << 32
    one = fn(q, k, v, pos, far, tab, s, s, *big)
    two = fn(q, k, v, pos, near, tab, s, s, *little)
    assert torch.equal(one, two)
    for b, w in zip(big, little):
        assert torch.equal(b[blocks], w) and int(torch.count_nonzero(w)) > 0
        b[blocks] = 0
        assert not bool(b.any())                                # and nothing anywhere else
    assert pkg.check_device_error() == 0


def test_far_outputs_of_experts(pkg):
    m, topk, n = 66000, 8, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    y = torch.empty((m, topk, n), dtype=torch.bfloat16, device=DEV)
    assert y.numel() > 1 << 31
    ends = [0, 1, 65535, 65536, m - 2, m - 1]
    y[ends] = torch.randn((len(ends), topk, n), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.rand((m, topk), generator=g, device=DEV)
    assert torch.equal(pkg.moe_combine(y, w)[ends], pkg.moe_combine(y[ends].contiguous(), w[ends].contiguous()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_far_rows(pkg, dtype):
    v, stride = 5001, (1 << 31) + 24
    x = torch.empty(2 * stride + v, dtype=dtype, device=DEV).as_strided((3, v), (stride, 1))
    g = torch.Generator(device=DEV).manual_seed(2)
    for r in range(3):
        x[r] = torch.randn(v, generator=g, device=DEV).to(dtype)
    near = x.contiguous()
    u = torch.rand((3, 2), generator=g, device=DEV)
    p = torch.full((3,), 0.9, device=DEV)
    for a, b in zip(pkg.sample_tokens(x, u, top_p=p) + pkg.sample_tokens(x, u),
                    pkg.sample_tokens(near, u, top_p=p) + pkg.sample_tokens(near, u)):
        assert torch.equal(a, b)
    for a, b in zip(pkg.moe_route(x[:, :200], 7), pkg.moe_route(near[:, :200], 7)):
        assert torch.equal(a, b)
    assert pkg.check_device_error() == 0
