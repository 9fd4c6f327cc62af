"""GPU tests of a captured fp8kv_rope_append / fp4kv_rope_append replayed on new
inputs, positions and slots in the same places: q and both caches are those of an
eager call on them."""
import pytest
import torch

from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("interleaved", [False, True])
def test_replay_on_new_inputs(bits, interleaved):
    pkg = lib_or_skip()
    t, hq, hkv, d, page, nb = 70, 8, 2, 128, 16, 6
    g = torch.Generator(device=DEV).manual_seed(bits)
    x = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), \
        x[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    pos = torch.arange(t, dtype=torch.int32, device=DEV)
    slots = torch.arange(t, dtype=torch.int32, device=DEV)
    angle = torch.arange(128, device=DEV)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, device=DEV) / d)
    table = torch.cat((torch.cos(angle), torch.sin(angle)), 1).float()
    ks, vs = torch.tensor([0.003], device=DEV), torch.tensor([0.002], device=DEV)
    w = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
    shape = pkg.kv4_cache_shape(nb, page, hkv, d) if bits == 4 else (nb, page, hkv, d)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    fn = pkg.kv4_rope_append if bits == 4 else pkg.kv_rope_append

    def call():
        return fn(q, k, v, pos, slots, table, ks, vs, kc, vc, q_norm=w, k_norm=w, interleaved=interleaved)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    seen = []
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        pos.copy_(torch.randint(0, 128, (t,), generator=g, device=DEV))
        slots.copy_(torch.randperm(nb * page, generator=g, device=DEV)[:t])
        if i == 2:
            pos[3], slots[3], slots[9] = -1, -1, -1             # padding, and a token that is not stored
        got.fill_(7.0)
        kc.zero_(), vc.zero_()
        graph.replay()
        replayed = [y.clone() for y in (got, kc, vc)]
        kc.zero_(), vc.zero_()
        want = call()
        if i == 2:
            want[3] = 7.0                                       # left as it was
        assert torch.equal(replayed[0], want) and torch.equal(replayed[1], kc) and torch.equal(replayed[2], vc)
        for y in replayed:
            assert int((y != 0).sum()) > 0 and not any(y.shape == z.shape and torch.equal(y, z) for z in seen)
        seen += replayed
    assert pkg.check_device_error() == 0
