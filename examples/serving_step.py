"""A decoder's serving step on the 4-bit paged KV cache, end to end:

    kv_plan               cache blocks and slots for the step's new tokens, from the request lengths
    per layer: gemv       the fused q, k, v projection (block FP8)
               kv4_append the new keys and values, straight from the projection's rows
               kv4_decode_attention   over the paged cache, any number of new tokens per request
               gemv       the output projection
    gemv                  the lm_head
    token_logprobs        the chosen token's log probability, the entropy and the alternatives

Prompts and decoding are the same step: a prompt is a step with several new
tokens per request.  Decode steps are captured once into a CUDA graph; the
plan runs inside it, on lengths and a free list that live on the device.

A request that finds no free blocks is refused for the step: its tokens keep
their rows, with slot -1, but are not in the cache, so what the step computes
in those rows means nothing.  Here its next token is -1 then; decoding gives
it the same token again until blocks have come back, and leaves out a request
that never got its prompt in.
Random weights; run on a GPU:

    python examples/serving_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_02_gb300 as fp8bs  # noqa: E402


class Decoder:
    """Random weights of a small decoder and the state of its requests."""

    def __init__(self, batch=4, layers=2, q_heads=8, kv_heads=2, head_dim=128, vocab=1000, page=16, max_len=512,
                 top=5, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        hidden, self.d = q_heads * head_dim, head_dim
        self.hq, self.hkv, self.page, self.top, self.max_len = q_heads, kv_heads, page, top, max_len
        self.device, self.batch = torch.device(device), batch

        def weight(n, k):
            return fp8bs.quantize((torch.randn((n, k), generator=g) * k ** -0.5).to(torch.bfloat16).to(device))

        self.embed = torch.randn((vocab, hidden), generator=g).to(torch.bfloat16).to(device)
        self.qkv = [weight((q_heads + 2 * kv_heads) * head_dim, hidden) for _ in range(layers)]
        self.out = [weight(hidden, hidden) for _ in range(layers)]
        self.head = weight(vocab, hidden)

        max_blocks = max_len // page
        self.num_blocks = batch * max_blocks
        shape = fp8bs.kv4_cache_shape(self.num_blocks, page, kv_heads, head_dim)
        self.caches = [[torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)] for _ in range(layers)]
        # amax / 2688 of normalised keys and values; a real model keeps the calibrated ones of each layer
        self.scale = torch.tensor([5.0 / 2688], device=device)
        self.workspace = fp8bs.kv4_workspace(head_dim, device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.table = torch.full((batch, max_blocks), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(self.num_blocks, generator=g).to(torch.int32).to(device)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, tokens, new_lens, max_q):
        """tokens [T]: new_lens[b] of each request, one after the other (what
        comes after them is padding).  Returns the plan, the logits [T, vocab],
        the likeliest next tokens [T], -1 where a token has no slot, and the
        TokenLogprobs of them."""
        t, hq, hkv, d = tokens.numel(), self.hq, self.hkv, self.d
        plan = fp8bs.kv_plan(self.lens, new_lens, self.table, self.free, self.free_head, self.page, self.num_blocks, t,
                             seq_lens=self.lens, free_head_out=self.free_head)
        x = self.embed[tokens.long().clamp(min=0)]
        for (wq, sq), (wo, so), (kc, vc) in zip(self.qkv, self.out, self.caches):
            qkv = fp8bs.gemv(torch.nn.functional.rms_norm(x, x.shape[1:]), wq, sq)
            q = qkv[:, :hq * d].unflatten(1, (hq, d))
            k, v = (qkv[:, i * d:(i + hkv) * d].unflatten(1, (hkv, d)) for i in (hq, hq + hkv))
            fp8bs.kv4_append(k, v, plan.slots, self.scale, self.scale, kc, vc)
            o = fp8bs.kv4_decode_attention(q, kc, vc, self.scale, self.scale, self.table, plan.seq_lens, self.max_len,
                                           d ** -0.5, self.workspace, cu_q=plan.cu_new, max_q=max_q,
                                           out=x.new_zeros((t, hq, d)))  # rows of padding are not written
            x = x + fp8bs.gemv(o.view(t, -1), wo, so)
        logits = fp8bs.gemv(torch.nn.functional.rms_norm(x, x.shape[1:]), *self.head)
        best = torch.where(plan.slots >= 0, logits.argmax(dim=1).to(torch.int32), -1)
        return plan, logits, best, fp8bs.token_logprobs(logits, best, self.top)

    def prompt(self, prompts):
        """Runs the requests' prompts (lists of tokens); returns each one's
        next token, -1 for a refused request."""
        lens = [len(p) for p in prompts]
        tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=self.device)
        new = torch.tensor(lens, dtype=torch.int32, device=self.device)
        plan, _, best, _ = self.step(tokens, new, max(lens))
        return best[plan.cu_new[1:].long() - 1].contiguous()

    def decode(self, tokens, steps):
        """Greedy decoding from each request's last token (-1: leave it out),
        every step one replay of a graph.  Yields (next tokens, log
        probabilities, entropies), -1, 0 and 0 for a request that was refused
        or left out."""
        state = [self.lens, self.table, self.free_head]
        tokens = tokens.clone()

        def one():
            live = tokens >= 0
            row = torch.where(live, live.cumsum(0) - 1, live.sum() + (~live).cumsum(0) - 1)  # of each request
            packed = torch.empty_like(tokens)
            packed[row] = tokens
            _, _, best, lp = self.step(packed, live.to(torch.int32), 1)
            best, logprobs, entropy = best[row], lp.logprobs[row], lp.entropy[row]
            done = best >= 0
            tokens.copy_(torch.where(done, best, tokens))
            return best, logprobs, torch.where(done, entropy, 0.0)

        kept = [s.clone() for s in state] + [tokens.clone()]
        one()                                                   # warm up, then put the requests back
        for s, was in zip(state + [tokens], kept):
            s.copy_(was)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = one()
        for _ in range(steps):
            graph.replay()
            yield tuple(t.clone() for t in out)


def main():
    model = Decoder()
    first = model.prompt([[3, 14, 15], [9], [2, 6, 5, 35, 8, 97, 93], list(range(40))])
    for i, (tokens, logprobs, entropy) in enumerate(model.decode(first, 8)):
        print(f"step {i}: tokens {tokens.tolist()}  log p {[round(v, 3) for v in logprobs.tolist()]}  "
              f"entropy {[round(v, 3) for v in entropy.tolist()]}")
    print("lengths", model.lens.tolist(), " blocks in use", int(model.free_head), "of", model.num_blocks)
    assert fp8bs.check_device_error() == 0


if __name__ == "__main__":
    main()
