"""Loads of the serving-step kernels.  A kernel launched ahead of its
predecessor's end may be on the GPU while what it will read is still being
written; ld.global.nc (__ldg) promises that nothing writes it while the kernel
lives, so these kernels use ordinary loads behind griddepcontrol.wait."""
import os
import re

import numpy as np
import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_02_gb300", "csrc")
DEV = "cuda"


@pytest.mark.parametrize("name", ["kv4.cu", "kvplan.cu", "logprobs.cu"])
def test_no_load_promises_that_its_source_is_constant(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"ld_nc_\w+|__ldg\b|ld\.global\.nc", code)


@pytest.mark.gpu
def test_every_call_sees_what_the_call_before_it_wrote():
    """Plans, appends, gathers and attention back to back on the same buffers, other values every round, with nothing
    but the stream between them."""
    from gpu_helpers import lib_or_skip
    pkg = lib_or_skip()
    b, hkv, d, page, rounds = 64, 4, 128, 16, 40
    g = torch.Generator(device=DEV).manual_seed(0)
    s = torch.tensor([5.5 / 2688], device=DEV)
    shape = pkg.kv4_cache_shape(b * 4, page, hkv, d)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    lens, head = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (b, 1))
    table = torch.full((b, 4), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(b * 4, generator=g, device=DEV).to(torch.int32)
    ones = torch.ones(b, dtype=torch.int32, device=DEV)
    xs = torch.randn((rounds, 2, b, hkv, d), generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn((b, 4 * hkv, d), generator=g, device=DEV).to(torch.bfloat16)
    ws = pkg.kv4_workspace(d, DEV)
    got = []
    torch.cuda.synchronize()
    for r in range(rounds):
        plan = pkg.kv_plan(lens, ones, table, free, head, page, b * 4, b, seq_lens=lens, free_head_out=head)
        pkg.kv4_append(xs[r, 0], xs[r, 1], plan.slots, s, s, kc, vc)
        k, v = pkg.kv4_gather(kc, vc, plan.slots, s, s)
        o = pkg.kv4_decode_attention(q, kc, vc, s, s, table, lens, 64, 0.1, ws)
        got.append((k, v, o))
    # the same with the GPU idle between calls
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pos = torch.arange(rounds, device=DEV)
    slots = table[:, pos // page] * page + pos % page                                # [b, rounds]
    for r in range(rounds):
        sl = slots[:, r].contiguous().to(torch.int32)
        pkg.kv4_append(xs[r, 0], xs[r, 1], sl, s, s, kc2, vc2)
        torch.cuda.synchronize()
        k, v = pkg.kv4_gather(kc2, vc2, sl, s, s)
        torch.cuda.synchronize()
        o = pkg.kv4_decode_attention(q, kc2, vc2, s, s, table, torch.full_like(lens, r + 1), 64, 0.1, ws)
        torch.cuda.synchronize()
        for a, w in zip(got[r], (k, v, o)):
            assert torch.equal(a.view(torch.int16), w.view(torch.int16)), r
    assert lens.tolist() == [rounds] * b and np.array_equal(kc.cpu().numpy(), kc2.cpu().numpy())
    assert pkg.check_device_error() == 0
