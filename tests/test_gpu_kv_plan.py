"""GPU tests of fp8bs_kv_plan against a plain request-by-request plan: every
output is a whole number and has to be equal."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from gpu_helpers import lib_or_skip

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


def make(batch, page, seed, max_ctx=200, max_new=40, spare=30, used=5, num_tokens=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, max_ctx + 1, batch)
    new = np.where(rng.random(batch) < 0.5, 1, rng.integers(0, max_new + 1, batch))
    held, end = -(-ctx // page), -(-(ctx + new) // page)
    nb = int(held.sum()) + used + int((end - held).sum()) + spare
    perm = rng.permutation(nb)
    table = np.full((batch, int(end.max(initial=1)) + 2), -1)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    return dict(ctx=ctx, new=new, table=table, free=perm[at:], head=used, page=page, num_blocks=nb,
                num_tokens=int(new.sum()) if num_tokens is None else num_tokens)


def dev(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def run_and_check(pkg, c, **kw):
    want, err = ref.plan(c["ctx"].tolist(), c["new"].tolist(), c["table"], c["free"].tolist(), c["head"], c["page"],
                         c["num_blocks"], c["num_tokens"])
    table = dev(c["table"])
    p = pkg.kv_plan(dev(c["ctx"]), dev(c["new"]), table, dev(c["free"]), dev([c["head"]]), c["page"], c["num_blocks"],
                    c["num_tokens"], **kw)
    got = dict(p._asdict(), table=table)
    for name, w in want.items():
        assert np.array_equal(got[name].cpu().numpy(), w), name
    assert pkg.check_device_error() == err
    return p


@pytest.mark.parametrize("page", [1, 16, 48, 256])
@pytest.mark.parametrize("batch", [1, 2, 33, 512, 513, 2000])
def test_matches_the_plain_plan(pkg, batch, page):
    run_and_check(pkg, make(batch, page, batch + page))


@pytest.mark.parametrize("new", [1, 3, 4095, 4096, 30011])
def test_one_long_prompt_among_single_tokens(pkg, new):
    c = make(9, 16, new, max_ctx=50, max_new=1)
    c["new"][4] = new
    end = -(-(c["ctx"] + c["new"]) // 16)
    c["table"] = np.pad(c["table"], ((0, 0), (0, int(end.max()))), constant_values=-1)
    c["num_tokens"] = int(c["new"].sum()) + 13                    # a padded token axis
    c["free"] = np.concatenate([c["free"], c["num_blocks"] + np.arange(new // 16 + 2)])
    c["num_blocks"] += new // 16 + 2
    run_and_check(pkg, c)


def test_no_requests_and_no_tokens(pkg):
    c = make(3, 16, 1)
    c.update(ctx=c["ctx"][:0], new=c["new"][:0], table=np.full((0, 4), -1), num_tokens=6)
    run_and_check(pkg, c)
    c = make(5, 16, 2)
    c["new"][:] = 0
    c["num_tokens"] = 0
    run_and_check(pkg, c)


@pytest.mark.parametrize("left", [0, 1, 7, 20])
def test_the_free_list_runs_out(pkg, left):
    c = make(64, 16, 3, used=2)
    c["free"] = c["free"][:2 + left]
    run_and_check(pkg, c)


def test_an_empty_free_list(pkg):
    c = make(4, 16, 4, used=0)
    c["free"] = c["free"][:0]
    run_and_check(pkg, c)


@pytest.mark.parametrize("head", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_a_head_outside_the_list(pkg, head):
    c = make(8, 16, 5)
    c["head"] = head
    run_and_check(pkg, c)


def test_lengths_that_cannot_be_are_refused(pkg):
    c = make(12, 16, 6)
    c["ctx"][2], c["new"][5] = -3, -7
    c["ctx"][7] = c["table"].shape[1] * 16                        # full: one more token does not fit
    c["new"][7] = 1
    c["ctx"][9], c["new"][9] = 2 ** 31 - 1, 2 ** 31 - 1           # the sum passes 32 bits
    c["new"][10] = 1
    run_and_check(pkg, c)


def test_more_tokens_than_the_token_axis_holds(pkg):
    c = make(10, 16, 7)
    c["num_tokens"] = int(c["new"][:6].sum())
    c["new"][6:] = np.maximum(c["new"][6:], 1)
    run_and_check(pkg, c)


def test_bad_block_ids_give_no_slots(pkg):
    c = make(6, 16, 8)
    c["ctx"][:] = 20                                              # the first new token shares an old block
    c["new"][:] = 30
    c["table"] = np.full((6, 6), -1)
    c["table"][:, :2] = np.arange(12).reshape(6, 2)
    c["num_blocks"], c["head"], c["num_tokens"] = 64, 0, 180
    c["free"] = np.arange(20, 60)
    c["table"][1, 1], c["table"][2, 1] = -5, 64
    c["free"][3], c["free"][4] = -2, 10 ** 6
    run_and_check(pkg, c)


def test_in_place_steps(pkg):
    """seq_lens in ctx_lens and the head in itself: several steps in a row."""
    page, batch, nb = 16, 40, 900
    rng = np.random.default_rng(9)
    ctx, table = dev(np.zeros(batch)), dev(np.full((batch, 24), -1))
    free, head = dev(rng.permutation(nb)), dev([0])
    h_ctx, h_table, h_head = np.zeros(batch, dtype=np.int64), np.full((batch, 24), -1), 0
    for step in range(6):
        new = rng.integers(0, 50, batch) if step == 0 else np.ones(batch, dtype=np.int64)
        want, err = ref.plan(h_ctx.tolist(), new.tolist(), h_table, free.cpu().tolist(), h_head, page, nb, 4096)
        p = pkg.kv_plan(ctx, dev(new), table, free, head, page, nb, 4096, seq_lens=ctx, free_head_out=head)
        assert p.seq_lens is ctx and p.free_head is head
        for name, w in want.items():
            got = table if name == "table" else getattr(p, name)
            assert np.array_equal(got.cpu().numpy(), w), (step, name)
        h_ctx, h_table, h_head = want["seq_lens"], want["table"], int(want["free_head"][0])
        assert err == 0 and pkg.check_device_error() == 0


def test_another_stream_and_a_graph(pkg):
    c = make(20, 32, 10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run_and_check(pkg, c, stream=s)
    args = (dev(c["ctx"]), dev(c["new"]), dev(c["table"]), dev(c["free"]), dev([c["head"]]), c["page"],
            c["num_blocks"], c["num_tokens"])
    want = pkg.kv_plan(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = pkg.kv_plan(*args)
    p.slots.fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.slots, want.slots) and torch.equal(p.seq_lens, want.seq_lens)
