"""GPU test of a step's operators run together, as a decoder with experts uses
them: plan, fused projection, norm and rotation into the paged cache,
attention, routing, the experts' products, their combination, lm_head,
sampling.  Every operator against its plain reference on the inputs it was
given; the whole eager, from a graph, and as two decoders on two streams at
once, bit for bit.
"""
import numpy as np
import pytest
import torch

import step_reference as ref
from gpu_helpers import bits, lib_or_skip
from oracle.tolerance import bf16_bits_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HQ, HKV, D, HIDDEN, E, TOPK, VOCAB, PAGE, MAX_LEN = 5, 8, 2, 128, 256, 16, 4, 2500, 16, 64


@pytest.fixture(scope="module")
def pkg():
    return lib_or_skip()


class Decoder:
    """One layer of random weights and the state of B requests."""

    def __init__(self, pkg, four_bit, seed):
        self.pkg, self.four_bit = pkg, four_bit
        g = torch.Generator().manual_seed(seed)

        def weight(n, k):
            return pkg.quantize((torch.randn((n, k), generator=g) * k ** -0.5).to(torch.bfloat16).to(DEV))
        self.embed = torch.randn((VOCAB, HIDDEN), generator=g).to(torch.bfloat16).to(DEV)
        self.qkv, self.out = weight((HQ + 2 * HKV) * D, HIDDEN), weight(HIDDEN, HQ * D)
        pairs = [weight(HIDDEN, HIDDEN) for _ in range(E)]
        self.experts = [torch.stack([p[j] for p in pairs]) for j in (0, 1)]
        self.router = torch.randn((E, HIDDEN), generator=g).to(DEV) * HIDDEN ** -0.5
        self.bias = torch.randn(E, generator=g).to(DEV) * 0.1
        self.head = weight(VOCAB, HIDDEN)
        self.q_norm, self.k_norm = ((1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
        a = torch.arange(MAX_LEN)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).to(DEV)
        self.nb = B * MAX_LEN // PAGE
        shape = pkg.kv4_cache_shape(self.nb, PAGE, HKV, D) if four_bit else (self.nb, PAGE, HKV, D)
        self.kc, self.vc = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.scale = torch.tensor([6.0 / (2688 if four_bit else 448)], device=DEV)
        self.ws = pkg.kv4_workspace(D, DEV)
        self.lens, self.free_head = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (B, 1))
        self.table = torch.full((B, MAX_LEN // PAGE), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(self.nb, generator=g).to(torch.int32).to(DEV)
        self.settings = dict(temperature=torch.tensor([1.0, 0.0, 0.7, 1.5, 1.0], device=DEV),
                             top_k=torch.tensor([0, 0, 50, 0, 20], dtype=torch.int32, device=DEV),
                             top_p=torch.tensor([1.0, 1.0, 0.9, 0.8, 0.95], device=DEV),
                             min_p=torch.tensor([0.0, 0.0, 0.0, 0.02, 0.0], device=DEV))
        self.tokens = torch.randint(0, VOCAB, (B,), generator=g).to(torch.int32).to(DEV)
        self.u = torch.rand((B, 2), generator=g).to(DEV)
        self.state = (self.lens, self.free_head, self.table, self.tokens, self.kc, self.vc)

    def rope(self, qkv, plan):
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        fn = self.pkg.kv4_rope_append if self.four_bit else self.pkg.kv_rope_append
        return fn(q, k, v, plan.positions, plan.slots, self.cos_sin, self.scale, self.scale, self.kc, self.vc,
                  q_norm=self.q_norm, k_norm=self.k_norm, out=torch.zeros((len(qkv), HQ, D), dtype=torch.bfloat16, device=DEV))

    def step(self, new_lens, rows=B, tokens=None, max_q=1, draw=None):
        """A step of `rows` token rows; draws for the rows of `draw` (all without)."""
        pkg = self.pkg
        plan = pkg.kv_plan(self.lens, new_lens, self.table, self.free, self.free_head, PAGE, self.nb, rows,
                           seq_lens=self.lens, free_head_out=self.free_head)
        x = self.embed[(self.tokens if tokens is None else tokens).long()]
        qkv = pkg.gemv(torch.nn.functional.rms_norm(x, (HIDDEN,)), *self.qkv)
        q = self.rope(qkv, plan)
        zeros = torch.zeros((rows, HQ, D), dtype=torch.bfloat16, device=DEV)
        if self.four_bit:
            o = pkg.kv4_decode_attention(q, self.kc, self.vc, self.scale, self.scale, self.table, plan.seq_lens, MAX_LEN,
                                         D ** -0.5, self.ws, cu_q=plan.cu_new, max_q=max_q, out=zeros)
        else:
            o = pkg.kv_decode_attention(q, self.kc, self.vc, self.scale, self.scale, self.table, plan.seq_lens, MAX_LEN,
                                        D ** -0.5, out=zeros)
        x = x + pkg.gemv(o.view(rows, -1), *self.out)
        h = torch.nn.functional.rms_norm(x, (HIDDEN,))
        router = h.float() @ self.router.T
        ids, w = pkg.moe_route(router, TOPK, scoring="sigmoid", bias=self.bias, groups=4, topk_groups=2, group_top=2,
                               scale=1.5)
        y = pkg.moe_gemv(h, ids, *self.experts)
        z = pkg.moe_combine(y, w, ids=ids, num_experts=E, residual=x)
        last = z if draw is None else z[draw]
        logits = pkg.gemv(torch.nn.functional.rms_norm(last, (HIDDEN,)), *self.head)
        got = pkg.sample_tokens(logits, self.u, **self.settings)
        self.tokens.copy_(got.tokens)
        return dict(plan=plan, qkv=qkv, q=q, router=router, ids=ids, w=w, y=y, x=x, z=z, logits=logits,
                    tokens=got.tokens, logprobs=got.logprobs)

    def prompt(self):
        """Prompts of 1 .. 9 tokens (4-bit) and three rows of padding, or of one token."""
        lens = [3, 1, 9, 5, 2] if self.four_bit else [1] * B
        rows = sum(lens) + (3 if self.four_bit else 0)
        tokens = torch.randint(0, VOCAB, (rows,), generator=torch.Generator().manual_seed(1)).to(DEV)
        return self.step(torch.tensor(lens, dtype=torch.int32, device=DEV), rows, tokens, max(lens),
                         (torch.tensor(lens).cumsum(0) - 1).to(DEV))


def check(m, r, cache_before):
    """The step's outputs against the plain references on the inputs each operator had."""
    pos, slots = (t.cpu().numpy() for t in (r["plan"].positions, r["plan"].slots))
    tab = m.cos_sin.cpu().numpy()
    cos, sin = tab[np.maximum(pos, 0), :D // 2], tab[np.maximum(pos, 0), D // 2:]
    qkv = bits(r["qkv"].cpu())
    q, k, v = (np.ascontiguousarray(a).reshape(len(pos), -1, D) for a in np.split(qkv, [HQ * D, (HQ + HKV) * D], 1))
    store = ref.store4 if m.four_bit else ref.store8
    s = np.float32(m.scale.item())
    kept = np.where(pos >= 0, slots, -1)
    turned = ref.turned(k, bits(m.k_norm.cpu()), 1e-6, cos, sin, False)
    assert np.array_equal(store(turned, kept, s, cache_before[0].cpu().numpy()), m.kc.cpu().numpy())
    assert np.array_equal(store(bf16_bits_to_f64(v), kept, s, cache_before[1].cpu().numpy()), m.vc.cpu().numpy())
    want = ref.turned(q, bits(m.q_norm.cpu()), 1e-6, cos, sin, False, rounded=False)
    want[pos < 0] = 0
    # 14 half steps of fp32 of either product, which are at most the head's size, and half a step of bf16
    size = np.abs(want).max() * 2
    assert np.all(np.abs(bf16_bits_to_f64(bits(r["q"].cpu())) - want) <= 2.0 ** -8 * np.abs(want) + 15 * 2.0 ** -24 * size)
    ids, w = ref.route(r["router"].double().cpu().numpy(), TOPK, "sigmoid", m.bias.cpu().numpy(), 4, 2, 2, scale=1.5)
    assert np.array_equal(r["ids"].cpu().numpy(), ids)
    assert np.all(np.abs(r["w"].double().cpu().numpy() - w) <= 2.0 ** -18 * w)
    y, z = r["y"].double().cpu().numpy(), r["z"].double().cpu().numpy()
    w, x = r["w"].double().cpu().numpy(), r["x"].double().cpu().numpy()
    want = ref.combine(y, w, residual=x)
    size = ref.combine(np.abs(y), w, residual=np.abs(x))         # 4 products and 4 sums round, then bf16
    assert np.all(np.abs(z - want) <= 2.0 ** -8 * np.abs(want) + 9 * 2.0 ** -24 * size)
    logits, u = r["logits"].double().cpu().numpy(), m.u.double().cpu().numpy()
    for b in range(B):
        token, lp, near = ref.sample(logits[b], *u[b], **{n: t[b].item() for n, t in m.settings.items()})
        assert near < 1e-6 or (int(r["tokens"][b]) == token and abs(float(r["logprobs"][b]) - lp) < 1e-5)


OUT = ("qkv", "q", "router", "ids", "w", "y", "x", "z", "logits", "tokens", "logprobs")


@pytest.mark.parametrize("four_bit", [True, False])
def test_steps_are_the_references_and_replay(pkg, four_bit):
    m = Decoder(pkg, four_bit, 3)
    before = m.kc.clone(), m.vc.clone()
    r = m.prompt()
    check(m, r, before)
    ones = torch.ones(B, dtype=torch.int32, device=DEV)
    m.step(ones)                                                # warm
    torch.cuda.synchronize()
    kept, u_start = [s.clone() for s in m.state], m.u.clone()
    eager = []
    for _ in range(12):
        before = m.kc.clone(), m.vc.clone()
        r = m.step(ones)
        check(m, r, before)
        eager.append({n: r[n].clone() for n in OUT})
        m.u.copy_((m.u * 7 + 0.13) % 1)
    after = [s.clone() for s in m.state]
    graph = torch.cuda.CUDAGraph()
    u_end = m.u.clone()
    m.u.copy_(u_start)
    for s, was in zip(m.state, kept):
        s.copy_(was)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r = m.step(ones)
        m.u.copy_((m.u * 7 + 0.13) % 1)
    for want in eager:
        graph.replay()
        for n in OUT:
            assert torch.equal(r[n], want[n]), n
    assert torch.equal(m.u, u_end)
    for s, want in zip(m.state, after):
        assert torch.equal(s, want)
    assert pkg.check_device_error() == 0


def test_two_decoders_on_two_streams(pkg):
    """The same steps alone, then at once on two streams and from two graphs that share nothing."""
    ones = torch.ones(B, dtype=torch.int32, device=DEV)

    def alone(four_bit, seed):
        m = Decoder(pkg, four_bit, seed)
        m.prompt()
        return [{n: t.clone() for n, t in m.step(ones).items() if n in OUT} for _ in range(20)]
    want = [alone(True, 3), alone(False, 4)]
    both = [Decoder(pkg, True, 3), Decoder(pkg, False, 4)]
    for m in both:
        m.prompt()
    torch.cuda.synchronize()
    kept = [[s.clone() for s in m.state] for m in both]
    streams, graphs, outs = [torch.cuda.Stream() for _ in both], [], []
    got = [[], []]
    for i in range(20):
        for j, m in enumerate(both):
            with torch.cuda.stream(streams[j]):
                got[j].append({n: t for n, t in m.step(ones).items() if n in OUT})
    torch.cuda.synchronize()
    for j in (0, 1):
        for i in range(20):
            for n in OUT:
                assert torch.equal(got[j][i][n], want[j][i][n]), (j, i, n)
    for m, state in zip(both, kept):
        for s, was in zip(m.state, state):
            s.copy_(was)
    torch.cuda.synchronize()
    for m in both:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(ones))
        graphs.append(g)
    torch.cuda.synchronize()
    for i in range(20):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                graphs[j].replay()
        torch.cuda.synchronize()
        for j in (0, 1):
            for n in OUT:
                assert torch.equal(outs[j][n], want[j][i][n]), (j, i, n)
    assert pkg.check_device_error() == 0


def test_a_refused_request_leaves_its_rows(pkg):
    """A pool too small for one request: its rows of q and the cache stay as they were, the others' do not change."""
    ones = torch.ones(B, dtype=torch.int32, device=DEV)
    full, short = Decoder(pkg, True, 5), Decoder(pkg, True, 5)
    short.free = short.free[:4].contiguous()                    # of five blocks
    a, b = full.step(ones), short.step(ones)
    gone = [int(i) for i in np.flatnonzero(b["plan"].positions.cpu().numpy() < 0)]
    assert len(gone) == 1 and pkg.check_device_error() == 32
    left = [i for i in range(B) if i not in gone]
    assert torch.equal(a["q"][left], b["q"][left]) and torch.all(b["q"][gone] == 0)
    check(short, b, (torch.zeros_like(short.kc), torch.zeros_like(short.vc)))
